// mx_encode.cuh -- quantisation of bf16 elements to a microscaled 4-bit format on
// the device: loads, block magnitudes, scale bytes and codes.  Shared by the
// codec (mx_codec.cu) and the product for few tokens (mx_few.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mx.h"
#include "mx_format.cuh"
#include "nf4_device.cuh"

namespace qlora {

// 8 kN consecutive elements of a row, from column c (a multiple of 8; zero past
// cols).  kVec: rows start on 16 bytes (cols % 8 == 0).  Otherwise the 16-byte
// pieces that hold them are loaded and shifted into place; `limit`: elements from
// the row's start to the end of the matrix, past which nothing is read.  kLate: the
// elements may have been written after this kernel began (before its
// griddepcontrol.wait), which the read-only path is not for.
template <bool kLate, typename T>
__device__ __forceinline__ T load_in(const T* p) {
  return kLate ? *p : __ldg(p);
}
template <bool kVec, int kN, bool kLate = false>
__device__ __forceinline__ void load_elems(const uint16_t* row, int64_t c, int64_t cols, int64_t limit, uint4 (&out)[kN]) {
  if constexpr (kVec) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      out[i] = c + 8 * i < cols ? load_in<kLate>(reinterpret_cast<const uint4*>(row + c) + i) : make_uint4(0, 0, 0, 0);
    return;
  }
  const int d = static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7u);    // elements past a 16-byte border
  const uint16_t* at = row + c - d;
  uint32_t w[4 * kN + 4];
#pragma unroll
  for (int i = 0; i <= kN; ++i) {
    uint4 q = make_uint4(0, 0, 0, 0);
    const int64_t e = c - d + 8 * i;                      // first element of the piece, counted from the row's start
    if (e < cols) {
      if (e + 8 <= limit) {
        q = load_in<kLate>(reinterpret_cast<const uint4*>(at) + i);
      } else {
        uint32_t* qw = &q.x;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (e + k < limit) qw[k >> 1] |= static_cast<uint32_t>(load_in<kLate>(at + 8 * i + k)) << (16 * (k & 1));
      }
    }
    w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
  }
  // shift by d elements: 4, 2, then 1 (d is the row's, the same in all lanes of a warp)
  if (d & 4) {
#pragma unroll
    for (int i = 0; i < 4 * kN + 2; ++i) w[i] = w[i + 2];
  }
  if (d & 2) {
#pragma unroll
    for (int i = 0; i < 4 * kN + 1; ++i) w[i] = w[i + 1];
  }
  if (d & 1) {
#pragma unroll
    for (int i = 0; i < 4 * kN; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  if (c + 8 * kN > cols) {                                // the row's end: nothing of the next row
#pragma unroll
    for (int i = 0; i < 4 * kN; ++i) {
      const int64_t left = cols - c - 2 * i;
      w[i] = left >= 2 ? w[i] : (left == 1 ? w[i] & 0xFFFFu : 0u);
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t cols, int64_t limit) {
  uint4 q[1];
  load_elems<kVec, 1>(row, c, cols, limit, q);
  return q[0];
}

// Thirty-two consecutive elements: what one thread encodes, one MXFP4 block or
// two NVFP4 blocks, so that no block is shared between threads.
struct Elems32 {
  uint4 q[4];
};
template <bool kVec, bool kLate = false>
__device__ __forceinline__ Elems32 load32(const uint16_t* row, int64_t c, int64_t cols, int64_t limit) {
  Elems32 e;
  load_elems<kVec, 4, kLate>(row, c, cols, limit, e.q);
  return e;
}

// Per 16-bit half: the larger magnitude.
__device__ __forceinline__ uint32_t mag_max2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t mag16(const uint4& a, const uint4& b) {
  uint32_t m = a.x & 0x7FFF7FFFu;
  m = mag_max2(m, a.y); m = mag_max2(m, a.z); m = mag_max2(m, a.w);
  m = mag_max2(m, b.x); m = mag_max2(m, b.y); m = mag_max2(m, b.z); m = mag_max2(m, b.w);
  return m;
}
__device__ __forceinline__ uint32_t wider_half(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// Largest finite magnitude (bf16 bits) of what mag16 saw or, where that holds
// values that are not finite, of the elements again without them.
__device__ __forceinline__ uint32_t finite_mag(uint32_t m, const uint4& q) {
  uint32_t top = wider_half(m);
  if (top >= 0x7F80u) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    bool bad = false;
    top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(mx_finite_mag(w[i], bad), mx_finite_mag(w[i] >> 16, bad)));
  }
  return top;
}
__device__ __forceinline__ uint32_t finite_mag8(const uint4& q) {
  uint32_t m = q.x & 0x7FFF7FFFu;
  m = mag_max2(m, q.y); m = mag_max2(m, q.z); m = mag_max2(m, q.w);
  return finite_mag(m, q);
}

// Scale byte of a block with the largest magnitude `mag` (bf16 bits).
template <int kFmt>
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag, float inv_g) {
  if (kFmt == kMxFp4) return mag >= 0x7F80u ? 255u : mx_e8m0(mag << 16);
  // v / 6 as mx_quotient2 has it: exact where it is half way between two E4M3 values
  const float v = __fmul_rn(__uint_as_float(mag << 16), inv_g), r = 1.0f / 6.0f, q = __fmul_rn(v, r);
  return mag >= 0x7F80u ? 0x7Fu : mx_e4m3(__fmaf_rn(__fmaf_rn(-6.0f, q, v), r, q));
}

// Multiplier (MXFP4), or scale and its reciprocal (NVFP4), of a block's elements.
struct BlockScale {
  float s, r;
  bool zero;                 // every code is 0: NaN scale or (NVFP4) scale 0
};
template <int kFmt>
__device__ __forceinline__ BlockScale block_scale(uint32_t sb) {
  BlockScale b;
  if (kFmt == kMxFp4) {
    b.zero = sb == 255u;
    b.s = b.r = mx_e8m0_inverse(b.zero ? 127u : sb);
  } else {
    b.zero = sb == 0x7Fu || sb == 0u;
    b.s = mx_e4m3_value(b.zero ? 0x38u : sb);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b.r) : "f"(b.s));      // the quotient's step makes up for its error
  }
  return b;
}
template <int kFmt>
__device__ __forceinline__ uint32_t encode8(float (&v)[8], const BlockScale& b, float inv_g) {
  const uint64_t s = f32x2(kFmt == kMxFp4 ? b.s : -b.s, kFmt == kMxFp4 ? b.s : -b.s), r = f32x2(b.r, b.r);
  const uint64_t ig = f32x2(inv_g, inv_g);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t x = f32x2(v[i], v[i + 1]);
    float lo, hi;
    if (kFmt == kMxFp4) {
      f32x2_split(f32x2_mul(x, s), lo, hi);
      v[i] = lo;
      v[i + 1] = hi;
    } else {
      f32x2_split(mx_quotient2(f32x2_mul(x, ig), s, r), lo, hi);
      v[i] = copysignf(lo, v[i]);
      v[i + 1] = copysignf(hi, v[i + 1]);
    }
  }
  const uint32_t c = mx_codes8(v);
  return b.zero ? 0u : c;
}
__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Codes of 32 elements and their scale byte (MXFP4), or two of them (NVFP4, the
// earlier block's in the low byte).
template <int kFmt>
__device__ __forceinline__ uint4 encode32(const Elems32& e, float inv_g, uint32_t& scales) {
  uint4 out;
  uint32_t* o = &out.x;
  float v[8];
  if (kFmt == kMxFp4) {
    scales = scale_byte<kFmt>(wider_half(__vmaxu2(mag16(e.q[0], e.q[1]), mag16(e.q[2], e.q[3]))), inv_g);
    const BlockScale b = block_scale<kFmt>(scales);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unpack8(e.q[i], v);
      o[i] = encode8<kFmt>(v, b, inv_g);
    }
  } else {
    scales = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t sb = scale_byte<kFmt>(wider_half(mag16(e.q[2 * h], e.q[2 * h + 1])), inv_g);
      const BlockScale b = block_scale<kFmt>(sb);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unpack8(e.q[2 * h + i], v);
        o[2 * h + i] = encode8<kFmt>(v, b, inv_g);
      }
      scales |= sb << (8 * h);
    }
  }
  return out;
}

}  // namespace qlora
