// mx_codec.cu -- microscaled 4-bit floating point: quantisation of a bf16
// matrix (also of its transpose) and dequantisation (sm_100a).
//
// A row is cut into blocks along the contraction index; a block's elements are
// e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and sign) times one scale:
//   MXFP4  32 elements, E8M0 scale 2^E, E = max(-127, floor(log2 amax) - 2);
//          code = e2m1(x / 2^E).
//   NVFP4  16 elements, E4M3 scale S and a float g for the whole tensor (or one
//          per row): g = the smallest power of two with amax_all <= 6 * 448 g;
//          S = e4m3((amax / g) / 6), code = e2m1((x / g) / S), 0 where S = 0.
// e2m1() and e4m3() round to nearest, ties to even.  Divisions by powers of two
// are exact; the other two cannot cross a rounding border in 32 bits (a bf16
// numerator over 6 or over a 4-bit significand is exactly on the border or
// 2^-9 away from it), so codes and scales are those of exact arithmetic.  A block with
// a value that is not finite gets the scale NaN; other blocks do not see it.
//
// Every pass is bound by memory: 2 bytes in, 0.5 + 1/32 (1/16) out per element.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mx.h"
#include "mx_format.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// Eight consecutive elements of a row, from column c (zero past cols).
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t cols) {
  if (c >= cols) return make_uint4(0, 0, 0, 0);
  if constexpr (kVec) return __ldg(reinterpret_cast<const uint4*>(row + c));   // cols % 8 == 0
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) w[i >> 1] |= static_cast<uint32_t>(__ldg(row + c + i)) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest finite magnitude of eight bf16 values (bits), and whether any is not finite.
__device__ __forceinline__ uint32_t mag8(const uint4& q, bool& bad) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = max(m, w[i] & 0x7FFFu);
    m = max(m, (w[i] >> 16) & 0x7FFFu);
  }
  if (m >= 0x7F80u) {                      // rare: look again, without the values that are not finite
    bad = true;
    m = 0;
    bool b = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = max(m, mx_finite_mag(w[i], b));
      m = max(m, mx_finite_mag(w[i] >> 16, b));
    }
  }
  return m;
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// The scale byte of a block (magnitude bits of bf16) and its eight codes per thread.
template <int kFmt>
__device__ __forceinline__ uint32_t scale_byte(uint32_t mag, bool bad, float inv_g) {
  if (kFmt == kMxFp4) return bad ? 255u : mx_e8m0(mag << 16);
  return bad ? 0x7Fu : mx_e4m3(__fdiv_rn(__fmul_rn(__uint_as_float(mag << 16), inv_g), 6.0f));
}

template <int kFmt>
__device__ __forceinline__ uint32_t encode8(float (&v)[8], uint32_t sb, bool bad, float inv_g) {
  if (bad) return 0u;
  if (kFmt == kMxFp4) {
    const float inv = mx_e8m0_inverse(sb);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], inv);
  } else {
    if (sb == 0u) return 0u;
    const float s = e4m3_to_f32(sb), r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx_quotient(__fmul_rn(v[i], inv_g), s, r);
  }
  return mx_codes8(v);
}

// A warp's 256 consecutive elements (eight per lane, from column c): codes and
// scales to memory.  Lanes of a block share its scale; the four bytes of a
// scale tile's row leave as one word.
template <int kFmt>
__device__ __forceinline__ void emit256(const MxQuantArgs& a, int64_t row, int64_t c, const uint4& q, float inv_g) {
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = mx_block(kFmt) / 8;                 // lanes of a block
  bool bad = false;
  uint32_t mag = mag8(q, bad);
  uint32_t key = bad ? (0x10000u | mag) : mag;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, key, o);
    key = max(key & 0xFFFFu, other & 0xFFFFu) | ((key | other) & 0x10000u);
  }
  bad = (key >> 16) != 0;
  mag = key & 0xFFFFu;
  const uint32_t sb = scale_byte<kFmt>(mag, bad, inv_g);
  float v[8];
  unpack8(q, v);
  const uint32_t codes = encode8<kFmt>(v, sb, bad, inv_g);
  uint32_t word = sb << (8 * ((lane / kLanes) & 3));
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, kLanes);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * kLanes);
  if (row < a.rows && c < a.pitch * 2) *reinterpret_cast<uint32_t*>(a.codes + row * a.pitch + (c >> 1)) = codes;
  const int64_t kt = c / (4 * mx_block(kFmt));
  if ((lane & (4 * kLanes - 1)) == 0 && kt < a.kt)
    *reinterpret_cast<uint32_t*>(a.scales + mx_scale_offset(row, kt * 4, a.kt)) = word;
}

// Largest of the partial maxima, in every thread.
__device__ uint32_t reduce_amax(const uint32_t* partials, int n) {
  __shared__ uint32_t s_max[kThreads / 32];
  uint32_t m = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) m = max(m, __ldcg(partials + i));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_max[i]);
  __syncthreads();
  return m;
}

__global__ void __launch_bounds__(kThreads) k_mx_amax(const uint16_t* in, int64_t numel, uint32_t* partials) {
  __shared__ uint32_t s_max[kThreads / 32];
  const int64_t nvec = numel / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  uint32_t m = 0;
  bool bad = false;
#pragma unroll 4
  for (int64_t i = first; i < nvec; i += stride) m = max(m, mag8(__ldg(reinterpret_cast<const uint4*>(in) + i), bad));
  if (first < numel - nvec * 8) m = max(m, mx_finite_mag(in[nvec * 8 + first], bad));
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_max[i]);
    partials[blockIdx.x] = m;
  }
}

// One warp per 1024 elements of a row (four loads in flight per lane).
template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) k_mx_quant(const MxQuantArgs a) {
  float inv_g = 1.0f;
  if (kFmt == kNvFp4) {
    const float g = mx_global_scale(reduce_amax(a.amax, a.amax_n) << 16);
    inv_g = mx_pow2_inverse(g);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.global_scale[0] = g;
  }
  const int lane = threadIdx.x & 31;
  const int64_t segs = (a.kt * 4 * mx_block(kFmt) + 1023) / 1024;
  const int64_t units = segs * a.tile_rows;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int64_t row = u / segs, c0 = (u - row * segs) * 1024 + lane * 8;
    const uint16_t* src = a.in + row * a.cols;
    uint4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = row < a.rows ? load8<kVec>(src, c0 + j * 256, a.cols) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) emit256<kFmt>(a, row, c0 + j * 256, q[j], inv_g);
  }
}

// NVFP4 with a global scale per row: one CTA per row.  The first 8192 elements
// stay in registers between the row's maximum and its codes; the rest of a
// longer row is read again (from L2).
template <bool kVec>
__global__ void __launch_bounds__(kThreads) k_mx_quant_rows(const MxQuantArgs a) {
  __shared__ uint32_t s_max[kThreads / 32];
  constexpr int kHeld = 4;
  const int64_t row = blockIdx.x;
  const uint16_t* src = a.in + row * a.cols;
  const int64_t span = a.kt * 64;
  const int64_t c0 = threadIdx.x * 8;
  uint4 held[kHeld];
  uint32_t m = 0;
  bool bad = false;
  if (row < a.rows) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) held[j] = load8<kVec>(src, c0 + j * (kThreads * 8), a.cols);
#pragma unroll
    for (int j = 0; j < kHeld; ++j) m = max(m, mag8(held[j], bad));
#pragma unroll 4
    for (int64_t c = c0 + kHeld * (kThreads * 8); c < a.cols; c += kThreads * 8)
      m = max(m, mag8(load8<kVec>(src, c, a.cols), bad));
  } else {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) held[j] = make_uint4(0, 0, 0, 0);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_max[i]);
  const float g = mx_global_scale(m << 16);
  const float inv_g = mx_pow2_inverse(g);
  if (threadIdx.x == 0 && row < a.rows) a.global_scale[row] = g;
  // whole warps step together: emit256 shuffles
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if ((threadIdx.x & ~31) * 8 + j * (kThreads * 8) < span)
      emit256<kNvFp4>(a, row, c0 + j * (kThreads * 8), held[j], inv_g);
  for (int64_t base = kHeld * (kThreads * 8) + (threadIdx.x & ~31) * 8; base < span; base += kThreads * 8) {
    const int64_t c = base + (threadIdx.x & 31) * 8;
    emit256<kNvFp4>(a, row, c, row < a.rows ? load8<kVec>(src, c, a.cols) : make_uint4(0, 0, 0, 0), inv_g);
  }
}

// The transpose: result row k is column k of the input, blocks run along the
// input's rows n.  A CTA takes 128 n x 64 k: rows of 128 bytes in, a column per
// thread out of shared memory (32 n: one MXFP4 or two NVFP4 blocks, 16 bytes of codes).
constexpr int kTileN = 128, kTileK = 64;

template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) k_mx_quant_t(const MxQuantArgs a) {
  __shared__ uint16_t tile[kTileN][kTileK + 2];
  float inv_g = 1.0f;
  if (kFmt == kNvFp4) {
    const float g = mx_global_scale(reduce_amax(a.amax, a.amax_n) << 16);
    inv_g = mx_pow2_inverse(g);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.global_scale[0] = g;
  }
  const int64_t n_tiles = (a.kt * 4 * mx_block(kFmt) + kTileN - 1) / kTileN;
  const int64_t k_tiles = (a.tile_rows + kTileK - 1) / kTileK;
  for (int64_t u = blockIdx.x; u < n_tiles * k_tiles; u += gridDim.x) {
    const int64_t k0 = u % k_tiles * kTileK, n0 = u / k_tiles * kTileN;
    uint4 q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + (threadIdx.x >> 3) + 32 * j;
      q[j] = n < a.in_rows ? load8<kVec>(a.in + n * a.in_cols, k0 + (threadIdx.x & 7) * 8, a.in_cols)
                           : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();                       // the tile's readers of the unit before are done
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(&tile[(threadIdx.x >> 3) + 32 * j][(threadIdx.x & 7) * 8]);
      dst[0] = q[j].x; dst[1] = q[j].y; dst[2] = q[j].z; dst[3] = q[j].w;
    }
    __syncthreads();
    const int kl = threadIdx.x & 63, nb = (threadIdx.x >> 6) * 32;
    const int64_t k = k0 + kl, n = n0 + nb;
    uint4 out;
    uint32_t* ow = &out.x;
    uint32_t sbytes = 0;
    uint32_t mag = 0;
    bool bad = false;
    constexpr int kBlk = mx_block(kFmt);
#pragma unroll
    for (int b = 0; b < 32 / kBlk; ++b) {
      mag = 0;
      bad = false;
#pragma unroll
      for (int i = 0; i < kBlk; ++i) mag = max(mag, mx_finite_mag(tile[nb + b * kBlk + i][kl], bad));
      const uint32_t sb = scale_byte<kFmt>(mag, bad, inv_g);
      sbytes |= sb << (8 * b);
#pragma unroll
      for (int g8 = 0; g8 < kBlk / 8; ++g8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bf16_lo(tile[nb + b * kBlk + g8 * 8 + i][kl]);
        ow[b * (kBlk / 8) + g8] = encode8<kFmt>(v, sb, bad, inv_g);
      }
    }
    if (k < a.rows && n < a.pitch * 2) *reinterpret_cast<uint4*>(a.codes + k * a.pitch + (n >> 1)) = out;
    const int64_t blk = n / kBlk;
    if (k < a.tile_rows && blk < a.kt * 4) {
      uint8_t* dst = a.scales + mx_scale_offset(k, blk, a.kt);
      if (kFmt == kMxFp4) *dst = static_cast<uint8_t>(sbytes);
      else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(sbytes);
    }
  }
}

// Eight codes (one 32-bit word, element j in bits 4j) times their scale -> bf16.
template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads)
k_mx_dequant(const uint8_t* codes, const uint8_t* scales, const float* gs, int per_row, int64_t rows, int64_t cols,
             int64_t pitch, int64_t kt, uint16_t* out) {
  const int64_t per = (cols + 7) / 8;
  const int64_t units = rows * per;
  const float g0 = (kFmt == kNvFp4 && !per_row) ? __ldg(gs) : 1.0f;
#pragma unroll 4
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < units;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = u / per, c = (u - row * per) * 8;
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + row * pitch + (c >> 1)));
    const uint32_t sb = __ldg(scales + mx_scale_offset(row, c / mx_block(kFmt), kt));
    float s;
    if (kFmt == kMxFp4) s = mx_e8m0_value(sb);
    else s = e4m3_to_f32(sb);
    const float g = kFmt == kNvFp4 ? (per_row ? __ldg(gs + row) : g0) : 1.0f;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t code = (w >> (8 * i + 4 * h)) & 15u;
        const uint32_t m = code & 7u;                           // 0, 1/2, then (1 + m0/2) 2^(e-1)
        const uint32_t bits = m < 2u ? (m ? 0x3F000000u : 0u) : (((m >> 1) + 126u) << 23) | ((m & 1u) << 22);
        f[h] = __fmul_rn(__fmul_rn(__uint_as_float(bits | ((code & 8u) << 28)), s), g);
      }
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[0], f[1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    if constexpr (kVec) {
      *reinterpret_cast<uint4*>(out + row * cols + c) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) out[row * cols + c + i] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
    }
  }
}

int grid_of(int64_t want, int num_sms, int per_sm) {
  const int64_t cap = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
}

template <int kFmt, bool kVec>
cudaError_t quant_t(bool transpose, const MxQuantArgs& a, int num_sms, cudaStream_t stream) {
  if (transpose) {
    const int64_t units = (a.kt * 4 * mx_block(kFmt) + kTileN - 1) / kTileN * ((a.tile_rows + kTileK - 1) / kTileK);
    k_mx_quant_t<kFmt, kVec><<<grid_of(units, num_sms, 8), kThreads, 0, stream>>>(a);
  } else if (kFmt == kNvFp4 && a.per_row) {
    k_mx_quant_rows<kVec><<<static_cast<unsigned>(a.tile_rows), kThreads, 0, stream>>>(a);
  } else {
    const int64_t segs = (a.kt * 4 * mx_block(kFmt) + 1023) / 1024;
    const int64_t ctas = (segs * a.tile_rows + kThreads / 32 - 1) / (kThreads / 32);
    k_mx_quant<kFmt, kVec><<<grid_of(ctas, num_sms, 8), kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_amax(const uint16_t* in, int64_t numel, uint32_t* partials, int grid, cudaStream_t stream) {
  k_mx_amax<<<grid, kThreads, 0, stream>>>(in, numel, partials);
  return cudaGetLastError();
}

cudaError_t launch_mx_quant(int fmt, bool transpose, const MxQuantArgs& a, int num_sms, cudaStream_t stream) {
  const bool vec = a.in_cols % 8 == 0;          // rows start on 16 bytes
  if (fmt == kMxFp4)
    return vec ? quant_t<kMxFp4, true>(transpose, a, num_sms, stream) : quant_t<kMxFp4, false>(transpose, a, num_sms, stream);
  return vec ? quant_t<kNvFp4, true>(transpose, a, num_sms, stream) : quant_t<kNvFp4, false>(transpose, a, num_sms, stream);
}

cudaError_t launch_mx_dequant(int fmt, const uint8_t* codes, const uint8_t* scales, const float* global_scale,
                              int per_row, int64_t rows, int64_t cols, int64_t pitch, int64_t kt, uint16_t* out,
                              int num_sms, cudaStream_t stream) {
  const int64_t units = rows * ((cols + 7) / 8);
  const int grid = grid_of((units + kThreads - 1) / kThreads, num_sms, 8);
  const bool vec = cols % 8 == 0;
#define QLORA_MX_DEQUANT(F, V) \
  k_mx_dequant<F, V><<<grid, kThreads, 0, stream>>>(codes, scales, global_scale, per_row, rows, cols, pitch, kt, out)
  if (fmt == kMxFp4) {
    if (vec) QLORA_MX_DEQUANT(kMxFp4, true); else QLORA_MX_DEQUANT(kMxFp4, false);
  } else {
    if (vec) QLORA_MX_DEQUANT(kNvFp4, true); else QLORA_MX_DEQUANT(kNvFp4, false);
  }
#undef QLORA_MX_DEQUANT
  return cudaGetLastError();
}

}  // namespace qlora
