// mx_format.cuh -- the microscaled 4-bit formats on the device (sm_100a):
// e2m1 elements, one scale per block of 32 (MXFP4, E8M0) or 16 (NVFP4, E4M3),
// and where a scale byte lies in its tile.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mx.h"

namespace qlora {

// Byte of the scale of block `blk` of row `row`: tiles of 128 rows x 4 blocks,
// 512 bytes, row-tile major (kt tiles a row), the layout the tensor core's
// 32-lane x 16-byte scale copies read without rearranging.
__host__ __device__ __forceinline__ int64_t mx_scale_offset(int64_t row, int64_t blk, int64_t kt) {
  return ((row >> 7) * kt + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
}

// Eight floats -> eight e2m1 codes (element j in bits 4j .. 4j+3): nearest,
// ties to the even code, values above 6 saturate.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// E8M0 byte of a block whose largest magnitude has the bits of a non-negative
// finite float: floor(log2 amax) - 2, at least -127, biased by 127 (6 = 1.5 * 2^2
// is the largest level).  Subnormal floats have exponent field 0 and clamp too.
__device__ __forceinline__ uint32_t mx_e8m0(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 2;
  return e > 0 ? static_cast<uint32_t>(e) : 0u;
}
// 2^(127 - byte) for byte <= 253, exact.
__device__ __forceinline__ float mx_e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// The value of an E8M0 byte (255: NaN).
__device__ __forceinline__ float mx_e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// E4M3 byte of a non-negative float <= 448 (ties to even).
__device__ __forceinline__ uint32_t mx_e4m3(float v) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.0f), "f"(v));
  return h & 0xFFu;
}

// The value of an E4M3 byte.
__device__ __forceinline__ float mx_e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// The NVFP4 global scale of magnitudes up to `amax` (bits of a non-negative
// finite float): the smallest power of two g with amax <= 6 * 448 * g
// (2688 = 1.3125 * 2^11), at least 2^-126; 1 for amax = 0.  A power of two, so
// that x / g is exact and every comparison below is the one of exact numbers.
__device__ __forceinline__ float mx_global_scale(uint32_t amax_bits) {
  if (amax_bits == 0u) return 1.0f;
  int e = static_cast<int>(amax_bits >> 23) - 127 - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  if (e < -126) e = -126;
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// 1 / g of a power of two in [2^-126, 2^127).
__device__ __forceinline__ float mx_pow2_inverse(float g) { return __uint_as_float((254u << 23) - __float_as_uint(g)); }

// y gx gw, the value of an accumulator under NVFP4's two global scales (gx a power
// of two from 2^-126 to 2^117, gw any positive float).  Without a rank-r term y is 0
// or between 2^-20 and 2^37 or so, so y gw stays a normal float for gw from 2^-106 to
// 2^91, and times gx is the result; the other order leaves the range on the way (y =
// 2^20 under gx = 2^110 and gw = 2^-14 is 2^116, y gx no float).  A gw beyond is
// brought inside by 2^64, which the result gets back.  No element asks for a case:
// branches in k_mx_pair's epilogue made it slower than the product it runs beside
// (8192^3: 381 us, 243 this way), and code that the end of a short kernel runs for the
// first time has to be fetched.
struct MxRowScale {
  float g, post;
};
__device__ __forceinline__ MxRowScale mx_row_scale(float gw) {
  MxRowScale r;
  r.post = gw < 0x1p-106f ? 0x1p-64f : gw > 0x1p91f ? 0x1p64f : 1.0f;
  r.g = __fmul_rn(gw, gw < 0x1p-106f ? 0x1p64f : gw > 0x1p91f ? 0x1p-64f : 1.0f);
  return r;
}
__device__ __forceinline__ float mx_scaled(float y, float gx, const MxRowScale& r) {
  return __fmul_rn(__fmul_rn(__fmul_rn(y, r.g), gx), r.post);
}

// Pairs of floats (sm_100's f32x2 arithmetic, each half rounded to nearest even
// as the scalar operation is).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// Quotients v / s to within a rounding, from r = 1 / s to within 2^-22: one Newton
// step on the remainder (minus_s = -s).  Where v / s is exactly half way between two levels
// it is representable and the step returns it exactly, so the tie stays a tie;
// every other quotient of an 8-bit by a 4-bit significand is 2^-8 away from one.
// The step turns -0 into +0, so the caller puts the sign back.
__device__ __forceinline__ uint64_t mx_quotient2(uint64_t v, uint64_t minus_s, uint64_t r) {
  const uint64_t q = f32x2_mul(v, r);
  return f32x2_fma(f32x2_fma(q, minus_s, v), r, q);
}

// bf16 bits -> magnitude bits with non-finite values as zero, and whether any was seen.
__device__ __forceinline__ uint32_t mx_finite_mag(uint32_t bits16, bool& bad) {
  const uint32_t m = bits16 & 0x7FFFu;
  if (m >= 0x7F80u) { bad = true; return 0u; }
  return m;
}

}  // namespace qlora
