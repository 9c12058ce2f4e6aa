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
// 2^-8 away from it), so codes and scales are those of exact arithmetic.  A block with
// a value that is not finite gets the scale NaN; other blocks do not see it.
//
// Bytes per element: 2 in, 0.5 + 1/32 (1/16) out.  MXFP4 is bound by them (8192 x
// 8192: 30 us, 5.6 TB/s), NVFP4 by instruction issue beside them (62 us with a pass
// for the maximum; transposed 70; dequantised 33).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mx.h"
#include "mx_encode.cuh"
#include "mx_format.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// A warp's 1024 consecutive elements (32 per lane, from column c): codes and
// scales to memory.  The four bytes of a scale tile's row leave as one word.
template <int kFmt>
__device__ __forceinline__ void emit1024(const MxQuantArgs& a, int64_t row, int64_t c, const Elems32& e, float inv_g) {
  const int lane = threadIdx.x & 31;
  uint32_t scales;
  const uint4 out = encode32<kFmt>(e, inv_g, scales);
  uint32_t word;
  if (kFmt == kMxFp4) {
    word = scales << (8 * (lane & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
  } else {
    word = scales << (16 * (lane & 1));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
  }
  if (row < a.rows && c < a.pitch * 2) *reinterpret_cast<uint4*>(a.codes + row * a.pitch + (c >> 1)) = out;
  constexpr int kTileElems = 4 * mx_block(kFmt);
  const int64_t kt = c / kTileElems;
  if ((lane & (kTileElems / 32 - 1)) == 0 && kt < a.kt)
    *reinterpret_cast<uint32_t*>(a.scales + mx_scale_offset(row, kt * 4, a.kt)) = word;
}

// Largest finite magnitude of elements first, first + stride, ... (8 at a time).
__device__ __forceinline__ uint32_t scan_amax(const uint16_t* in, int64_t numel, int64_t first, int64_t stride) {
  const int64_t nvec = numel / 8;
  uint32_t m = 0;
  bool bad = false;
  constexpr int kBatch = 8;                  // loads in flight per thread
  int64_t i = first;
  for (; i + (kBatch - 1) * stride < nvec; i += kBatch * stride) {
    uint4 q[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) q[j] = __ldg(reinterpret_cast<const uint4*>(in) + i + j * stride);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) m = max(m, finite_mag8(q[j]));
  }
  for (; i < nvec; i += stride) m = max(m, finite_mag8(__ldg(reinterpret_cast<const uint4*>(in) + i)));
  if (first < numel - nvec * 8) m = max(m, mx_finite_mag(in[nvec * 8 + first], bad));
  return m;
}

// Largest magnitude of the whole matrix, in every thread: of the partial maxima
// or, for a small matrix (amax_n = 0), found by every CTA for itself, which is
// faster than a launch.
__device__ uint32_t reduce_amax(const MxQuantArgs& a) {
  __shared__ uint32_t s_max[kThreads / 32];
  uint32_t m = 0;
  if (a.amax_n == 0) m = scan_amax(a.in, a.in_rows * a.in_cols, threadIdx.x, kThreads);
  else
    for (int i = threadIdx.x; i < a.amax_n; i += kThreads) m = max(m, __ldcg(a.amax + i));
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
  uint32_t m = scan_amax(in, numel, static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x,
                         static_cast<int64_t>(gridDim.x) * kThreads);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, s_max[i]);
    partials[blockIdx.x] = m;
  }
}

// What a kernel that reads the result may do meanwhile: start, and wait for this
// grid before it reads.  Its counters are cleared here.
__device__ __forceinline__ void open_dependents(const MxQuantArgs& a) {
  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      for (int i = threadIdx.x; i < a.zero_n[j]; i += blockDim.x) a.zero[j][i] = 0u;
}

// Units (row, segment) of a row-major walk with a fixed stride, without a
// division per step.
struct Walk {
  int64_t row, seg, step_rows, step_segs, segs;
  __device__ Walk(int64_t first, int64_t stride, int64_t per_row)
      : row(first / per_row), seg(first - row * per_row), step_rows(stride / per_row),
        step_segs(stride - step_rows * per_row), segs(per_row) {}
  __device__ void next() {
    row += step_rows;
    seg += step_segs;
    if (seg >= segs) { seg -= segs; ++row; }
  }
};

// One warp per 1024 elements of a row.  With a global scale the rows go from the
// last to the first: the maximum's pass has just left the last ones in L2.
template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) k_mx_quant(const MxQuantArgs a) {
  open_dependents(a);
  float inv_g = 1.0f;
  if (kFmt == kNvFp4) {
    const float g = mx_global_scale(reduce_amax(a) << 16);
    inv_g = mx_pow2_inverse(g);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.global_scale[0] = g;
  }
  const int lane = threadIdx.x & 31;
  for (Walk w(static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5),
              static_cast<int64_t>(gridDim.x) * (kThreads / 32), (a.kt * 4 * mx_block(kFmt) + 1023) / 1024);
       w.row < a.tile_rows; w.next()) {
    const int64_t row = kFmt == kNvFp4 ? a.tile_rows - 1 - w.row : w.row, c = w.seg * 1024 + lane * 32;
    Elems32 e{};
    if (row < a.rows) e = load32<kVec>(a.in + row * a.cols, c, a.cols, (a.rows - row) * a.cols);
    emit1024<kFmt>(a, row, c, e, inv_g);
  }
}

// NVFP4 with a global scale per row: one CTA per row.  The first
// kRowThreads * 32 * kHeld elements stay in registers between the row's maximum
// and its codes; the rest of the row is read again (from L2).
template <bool kVec, int kRowThreads, int kHeld>
__global__ void __launch_bounds__(kRowThreads) k_mx_quant_rows(const MxQuantArgs a) {
  open_dependents(a);
  __shared__ uint32_t s_max[32];
  constexpr int kStep = kRowThreads * 32;
  const int64_t row = blockIdx.x;
  const uint16_t* src = a.in + row * a.cols;
  const int64_t limit = (a.rows - row) * a.cols;
  const int64_t span = a.kt * 64;
  const int64_t c0 = threadIdx.x * 32, w0 = (threadIdx.x & ~31) * 32;
  Elems32 held[kHeld > 0 ? kHeld : 1];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    held[j] = Elems32{};
    if (row < a.rows) held[j] = load32<kVec>(src, c0 + j * kStep, a.cols, limit);
  }
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, finite_mag8(held[j].q[i]));
  if (row < a.rows)
    for (int64_t c = kHeld * kStep + threadIdx.x * 8; c < a.cols; c += 8 * kRowThreads * 8) {
      uint4 q[8];                            // eight loads in flight (zero past the row)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = load8<kVec>(src, c + j * kRowThreads * 8, a.cols, limit);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, finite_mag8(q[j]));
    }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xFFFFFFFFu, s_max[threadIdx.x & (kRowThreads / 32 - 1)]);
  const float g = mx_global_scale(m << 16);
  const float inv_g = mx_pow2_inverse(g);
  if (threadIdx.x == 0 && row < a.rows) a.global_scale[row] = g;
  // whole warps step together: emit1024 shuffles
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (w0 + j * kStep < span) emit1024<kNvFp4>(a, row, c0 + j * kStep, held[j], inv_g);
  for (int64_t b = kHeld * kStep; w0 + b < span; b += kStep) {
    Elems32 e{};
    if (row < a.rows) e = load32<kVec>(src, c0 + b, a.cols, limit);
    emit1024<kNvFp4>(a, row, c0 + b, e, inv_g);
  }
}

// The transpose: result row k is column k of the input, blocks run along the
// input's rows n.  A CTA takes 256 n x 64 k: rows of 128 bytes in; a thread then
// takes 32 n of two neighbouring columns out of shared memory, whose magnitudes
// it compares as pairs of 16 bits.
constexpr int kTileN = 256, kTileK = 64;

template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads) k_mx_quant_t(const MxQuantArgs a) {
  __shared__ uint32_t tile[kTileN][kTileK / 2 + 1];
  float inv_g = 1.0f;
  if (kFmt == kNvFp4) {
    const float g = mx_global_scale(reduce_amax(a) << 16);
    inv_g = mx_pow2_inverse(g);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.global_scale[0] = g;
  }
  const int64_t n_tiles = (a.kt * 4 * mx_block(kFmt) + kTileN - 1) / kTileN;
  const int64_t k_tiles = (a.tile_rows + kTileK - 1) / kTileK;
  for (Walk w(blockIdx.x, gridDim.x, k_tiles); w.row < n_tiles; w.next()) {
    const int64_t k0 = w.seg * kTileK, n0 = (kFmt == kNvFp4 ? n_tiles - 1 - w.row : w.row) * kTileN;
    uint4 q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t n = n0 + (threadIdx.x >> 3) + 32 * j;
      q[j] = n < a.in_rows ? load8<kVec>(a.in + n * a.in_cols, k0 + (threadIdx.x & 7) * 8, a.in_cols,
                                           (a.in_rows - n) * a.in_cols)
                           : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();                       // the tile's readers of the unit before are done
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t* dst = &tile[(threadIdx.x >> 3) + 32 * j][(threadIdx.x & 7) * 4];
      dst[0] = q[j].x; dst[1] = q[j].y; dst[2] = q[j].z; dst[3] = q[j].w;
    }
    __syncthreads();
    const int kp = threadIdx.x & 31, nb = (threadIdx.x >> 5) * 32;
    const int64_t k = k0 + 2 * kp, n = n0 + nb;
    uint32_t e[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) e[i] = tile[nb + i][kp];
    constexpr int kBlk = mx_block(kFmt);
    uint4 out[2];
    uint32_t sbytes[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 32 / kBlk; ++b) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kBlk; ++i) m = mag_max2(m, e[b * kBlk + i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sb = scale_byte<kFmt>(h ? m >> 16 : m & 0xFFFFu, inv_g);
        const BlockScale bs = block_scale<kFmt>(sb);
        sbytes[h] |= sb << (8 * b);
#pragma unroll
        for (int g8 = 0; g8 < kBlk / 8; ++g8) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x = e[b * kBlk + g8 * 8 + i];
            v[i] = h ? bf16_hi(x) : bf16_lo(x);
          }
          (&out[h].x)[b * (kBlk / 8) + g8] = encode8<kFmt>(v, bs, inv_g);
        }
      }
    }
    const int64_t blk = n / kBlk;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (k + h < a.rows && n < a.pitch * 2) *reinterpret_cast<uint4*>(a.codes + (k + h) * a.pitch + (n >> 1)) = out[h];
      if (k + h < a.tile_rows && blk < a.kt * 4) {
        uint8_t* dst = a.scales + mx_scale_offset(k + h, blk, a.kt);
        if (kFmt == kMxFp4) *dst = static_cast<uint8_t>(sbytes[h]);
        else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(sbytes[h]);
      }
    }
  }
}

// Eight codes (element j in bits 4j .. 4j+3) -> four pairs of halves, exact.
__device__ __forceinline__ void mx_levels8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// v g for a g that is no power of two, as floats that rounding to bf16 takes where the
// exact products go: only a product that fp32 rounds onto a tie of bf16 can go
// wrong, and is moved one step towards the exact one.  Its remainder is exact where
// the product's last bit, 2^-33 g at least, is a float; below, the 6 and 24 bits are
// multiplied in doubles and cut off, the last bit standing for all that follows.
constexpr float kForeignLeast = 0x1p-116f;
__device__ __forceinline__ void mx_times_foreign8(float (&v)[8], float g) {
  bool tie = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) tie |= (__float_as_uint(__fmul_rn(v[i], g)) & 0xFFFFu) == 0x8000u;
  if (!tie) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], g);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = __fmul_rn(v[i], g), left = __fmaf_rn(v[i], g, -p);
    const uint32_t u = __float_as_uint(p);
    const uint32_t step = static_cast<uint32_t>((static_cast<int32_t>(u ^ __float_as_uint(left)) >> 31) | 1);
    v[i] = left != 0.0f && (u & 0xFFFFu) == 0x8000u ? __uint_as_float(u + step) : p;
  }
}
__device__ __forceinline__ void mx_times_tiny8(float (&v)[8], float g) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double p = static_cast<double>(v[i]) * static_cast<double>(g);
    const float f = __double2float_rz(p);
    v[i] = static_cast<double>(f) == p ? f : __uint_as_float(__float_as_uint(f) | 1u);
  }
}

// Codes times their scale -> bf16; one warp per 1024 elements of a row.  The global
// scales that the encoder writes are powers of two, whose product in fp32 is exact
// wherever bf16 can tell.
template <int kFmt, bool kVec>
__global__ void __launch_bounds__(kThreads)
k_mx_dequant(const uint8_t* codes, const uint8_t* scales, const float* gs, int per_row, int64_t rows, int64_t cols,
             int64_t pitch, int64_t kt, uint16_t* out) {
  __shared__ uint4 s_out[kThreads];          // a warp's 256 values on their way to a row that starts anywhere
  const int lane = threadIdx.x & 31;
  const float g0 = (kFmt == kNvFp4 && !per_row) ? __ldg(gs) : 1.0f;
  for (Walk w(static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5),
              static_cast<int64_t>(gridDim.x) * (kThreads / 32), (cols + 1023) / 1024);
       w.row < rows; w.next()) {
    const int64_t c0 = w.seg * 1024 + lane * 8;
    const float g = kFmt == kNvFp4 ? (per_row ? __ldg(gs + w.row) : g0) : 1.0f;
    const bool foreign = kFmt == kNvFp4 && (__float_as_uint(g) & 0x7FFFFFu) != 0u;
    uint32_t word[4], sb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + j * 256;
      word[j] = sb[j] = 0;
      if (c < cols) {
        word[j] = __ldg(reinterpret_cast<const uint32_t*>(codes + w.row * pitch + (c >> 1)));
        sb[j] = __ldg(scales + mx_scale_offset(w.row, c / mx_block(kFmt), kt));
      }
    }
    auto store = [&](auto times_g) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + j * 256;
        if (kVec && c >= cols) continue;
        const float s = kFmt == kMxFp4 ? mx_e8m0_value(sb[j]) : mx_e4m3_value(sb[j]);
        uint32_t h[4], o[4];
        mx_levels8(word[j], h);
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
          v[2 * i] = __fmul_rn(f.x, s);
          v[2 * i + 1] = __fmul_rn(f.y, s);
        }
        times_g(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          o[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        if constexpr (kVec) {
          *reinterpret_cast<uint4*>(out + w.row * cols + c) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          // 32 neighbouring values a store
          uint4* mine = s_out + (threadIdx.x & ~31);
          __syncwarp();
          mine[lane] = make_uint4(o[0], o[1], o[2], o[3]);
          __syncwarp();
          const int64_t first = w.seg * 1024 + j * 256;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (first + i * 32 + lane < cols)
              out[w.row * cols + first + i * 32 + lane] = reinterpret_cast<const uint16_t*>(mine)[i * 32 + lane];
        }
      }
    };
    // one branch for all of a warp's 1024 values: inside the loop it costs 12%
    if constexpr (kFmt == kMxFp4) {
      store([](float (&)[8]) {});
    } else if (!foreign) {
      store([&](float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], g);
      });
    } else if (g >= kForeignLeast) {
      store([&](float (&v)[8]) { mx_times_foreign8(v, g); });
    } else {
      store([&](float (&v)[8]) { mx_times_tiny8(v, g); });
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
    // Many rows: small CTAs that read a long row twice, the second time from L2, so
    // that an SM has several rows in all phases at once (8192 rows of 22016: 119 us;
    // held in the registers of 1024 threads 208 us).  Few rows: as many threads as
    // hold the row (16 rows of 22016: 4.7 us; the small CTAs 9 us).
    const unsigned grid = static_cast<unsigned>(a.tile_rows);
    if (a.cols <= 4096) k_mx_quant_rows<kVec, 128, 1><<<grid, 128, 0, stream>>>(a);
    else if (a.tile_rows >= 4 * static_cast<int64_t>(num_sms)) k_mx_quant_rows<kVec, 128, 0><<<grid, 128, 0, stream>>>(a);
    else if (a.cols <= 8192) k_mx_quant_rows<kVec, 256, 1><<<grid, 256, 0, stream>>>(a);
    else if (a.cols <= 16384) k_mx_quant_rows<kVec, 512, 1><<<grid, 512, 0, stream>>>(a);
    else k_mx_quant_rows<kVec, 1024, 1><<<grid, 1024, 0, stream>>>(a);
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
  const int64_t units = rows * ((cols + 1023) / 1024);
  const int grid = grid_of((units + kThreads / 32 - 1) / (kThreads / 32), num_sms, 8);
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
