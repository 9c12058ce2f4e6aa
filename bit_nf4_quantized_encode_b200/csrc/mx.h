// mx.h -- launch interfaces of the microscaled 4-bit kernels: quantise and
// dequantise (mx_codec.cu), the product for a token or a few (mx_few.cu), few
// (mx_stream.cu) and many (mx_pair.cu), X A^T beside it (mx_xa.cu) and the
// mixture-of-experts layer for a few tokens (mx_moe.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qlora {

enum : int { kMxFp4 = 0, kNvFp4 = 1 };

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == kMxFp4 ? 32 : 16; }
// Bytes of one row of codes: two codes a byte, whole 16-byte pieces (32 codes).
inline int64_t mx_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
// Scale tiles (128 rows x 4 blocks, 512 bytes) along a row.
inline int64_t mx_tiles_k(int fmt, int64_t cols) {
  const int64_t per = 4 * mx_block(fmt);
  return (cols + per - 1) / per;
}
inline int64_t mx_scale_bytes(int fmt, int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * mx_tiles_k(fmt, cols) * 512;
}

// CTAs of the amax pass of an NVFP4 tensor quantised with one global scale
// (one partial maximum each).
constexpr int kMxAmaxGrid = 1184;
// Up to this many elements every CTA of the quantiser finds the maximum itself.  In
// us of the GPU, one launch and two: 16384 elements 3.0 and 4.7, 65536 4.7 and 4.6,
// 100000 6.8 and 5.6, 131072 7.6 and 5.2, 262144 20 and 6.3; from the binding, where
// the second launch and its work buffer cost the host 5: 8 and 13, 8 and 13, 8 and 15,
// 10 and 13, 23 and 13.  The limit is the calls'; a graph of many such quantisations
// loses 2.4 us each at its upper end.
constexpr int64_t kMxSmallElements = 131072;

struct MxQuantArgs {
  const uint16_t* in;        // bf16 [in_rows, in_cols], contiguous
  int64_t in_rows, in_cols;
  uint8_t* codes;            // [rows][pitch] of the result
  uint8_t* scales;
  float* global_scale;       // NVFP4: [1], or [rows] when per_row
  int64_t rows, cols;        // of the result: (in_rows, in_cols), or swapped
  int64_t pitch, kt;
  int64_t tile_rows;         // rows whose scale bytes are written: rows, or rows padded to 128
  int per_row;
  uint32_t* amax;            // NVFP4, one global scale: partial maxima [amax_n]
  int amax_n;                // 0: none, a small matrix
  uint32_t* zero[2];         // words cleared on the way (the counters of later kernels)
  int zero_n[2];
};

cudaError_t launch_mx_amax(const uint16_t* in, int64_t numel, uint32_t* partials, int grid, cudaStream_t stream);
cudaError_t launch_mx_quant(int fmt, bool transpose, const MxQuantArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_mx_dequant(int fmt, const uint8_t* codes, const uint8_t* scales, const float* global_scale,
                              int per_row, int64_t rows, int64_t cols, int64_t pitch, int64_t kt, uint16_t* out,
                              int num_sms, cudaStream_t stream);

// The product D[token, row] = sum_k x[token, k] w[row, k] of two microscaled
// operands plus a rank-r bf16 term, on the tensor cores' block-scaled
// instructions.
struct MxGemmArgs {
  const uint8_t* w_scales;   // scale tiles of the weight [rows, k]
  const uint8_t* x_scales;   // and of the activations [m, k]
  int64_t kt;                // scale tiles along k (the same for both)
  const float* w_global;     // NVFP4: [1] or [rows]
  int w_per_row;
  const float* x_global;     // NVFP4: [m]
  int64_t rows, m, k;
  int ksteps;                // ceil(k / 256)
  int lora_steps;            // 64 ranks each of the rank-r term (0: none), its activations in two bf16 parts
  int lora_mn;               // its weight-side operand: 0 [rows, r], 1 [r, rows] (rows contiguous)
  uint16_t* out;             // bf16 [m, rows]
  int m_tiles, t_tiles;      // tiles of rows (128, of a pair 256) and of tokens
  // pairs: row tiles swept across all token tiles before the next group
  int m_group;
  // streams: partial tiles [runs][2][m][128] and a counter (zero) per 32 rows
  float* slots;
  uint32_t* counters;
  uint32_t* err;
};
// Tensor maps: w / x the codes as uint8 [rows or m][pitch], 128B swizzle, box
// {128, 128} / {128, x rows}; w_scales / x_scales the scale tiles as 32-bit
// words [row tiles * kt][128], box {128, 2 (MXFP4) or 4} (pairs only); lora_w
// bf16, box {64, 128} ([rows, r]) or {64, 64} ([r, rows]); lora_x bf16
// [m, 128 lora_steps] (after 64 ranks' first parts their second ones), box {64, x rows}.
struct MxMaps {
  CUtensorMap w, x, w_scales, x_scales, lora_w, lora_x;
};
// Few tokens (mx_stream.cu): one tile of 16, 32 or 64 tokens (x rows the same).
constexpr int kMxMaxRuns = 256;             // CTAs at most: the work buffer's slots are sized by it
cudaError_t launch_mx_stream(int fmt, int token_tile, const MxGemmArgs& a, const MxMaps& m, int num_sms,
                             cudaStream_t stream);
// Many tokens (mx_pair.cu): tiles of 256 rows x 256 or 128 tokens (x rows half of it).
cudaError_t launch_mx_pair(int fmt, int token_tile, const MxGemmArgs& a, const MxMaps& m, int num_sms,
                           cudaStream_t stream);

// At most 16 tokens, quantised by the product itself (mx_few.cu).
struct MxFewArgs {
  const uint16_t* x;         // bf16 [m, k]
  int vec;                   // k % 8 == 0: rows start on 16 bytes
  const uint8_t* w_scales;
  int64_t kt;
  const float* w_global;     // NVFP4: [1] or [rows]
  int w_per_row;
  int64_t rows, k;
  int m, ksteps, lora_steps;
  uint16_t* out;             // bf16 [m, rows]
  int chunks, units, stage_bytes, stages;   // set by the launch
  uint32_t* err;
};
// Every CTA reads the tokens (2 bytes an element, from L2) and keeps them: limits
// of their number and of their shared memory.
constexpr int64_t kMxFewElements = 16384;
constexpr size_t kMxFewShared = 132 * 1024;
// Token tile (8 or 16), or 0 where the tokens are too many or mx_stream.cu is faster.
int mx_few_tile(int fmt, int64_t rows, int64_t m, int64_t k, int lora_steps, int num_sms);
// Maps: w codes box {128, 32}; lora_w [rows, r] box {64, 32}; lora_x box {64, token_tile}.
cudaError_t launch_mx_few(int fmt, int token_tile, const MxFewArgs& a, const MxMaps& m, int num_sms, cudaStream_t stream);

// X A^T for at most 64 tokens (mx_xa.cu), as run_rank_xa gives it for more.
struct MxXaArgs {
  const uint16_t* x;         // bf16 [m, k]
  const uint16_t* a;         // bf16 [r, k]
  int64_t k;                 // a multiple of 64
  int m, r, rpad;
  float s;
  float* xa;                 // fp32 [m, r] or null
  uint16_t* sxa;             // bf16 [m, 2 rpad]: s X A^T [/ (g all_div)], zero from column r, in two
                             // parts (RankProblem::out_parts)
  const float* all_div;      // [1]: divide by it and the token's NVFP4 global scale g; or null
  // the first kernel of its call starts when all before it has ended, a later one
  // beside the one before
  int first;
};
cudaError_t launch_mx_xa(const MxXaArgs& a, cudaStream_t stream);

// Mixture-of-experts layer for at most 16 tokens (mx_moe.cu).
constexpr int kMoeMaxExperts = 256, kMoeMaxTopK = 16, kMoeMaxTokens = 16;

// An expert in use: its tokens (bit t) and, four bits per token, which of the
// token's choices it is.
struct MoeExpert {
  int32_t id;
  uint32_t tokens;
  uint64_t slots;
};

struct MxMoeArgs {
  const uint16_t* x;          // bf16 [m, hidden]
  const uint16_t* router;     // bf16 [experts, hidden]
  const uint8_t* w13_scales;  // of [experts * 2 inner, hidden]
  const uint8_t* w2_scales;   // of [experts * hidden, inner]
  int64_t hidden, inner;      // multiples of 128
  int m, experts, top_k;
  uint16_t* y;                // bf16 [m, hidden]
  int32_t* ids;               // [m, top_k]
  float* probs;               // [m, top_k]
  // work space
  uint8_t* x_codes;           // [m][hidden / 2]
  uint8_t* x_scales;          // one row tile
  uint8_t* h_codes;           // [used][16][inner / 2]
  uint8_t* h_scales;          // [used] row tiles
  float* slots;               // [runs][2][2 m][128]
  MoeExpert* list;            // [used]
  int* n_used;
  uint32_t* counters;         // the down tiles' [hidden / 32], the up tiles' [used * inner / 32]
  uint32_t* up_counters;
  int n_counters;
  uint32_t* err;
};
// Maps: w13 / w2 / x / h codes as uint8, 128B swizzle, box {128, 128} for the
// weights and {128, 16} for x [m rows] and h [16 * max_used rows].
cudaError_t launch_mx_moe(const MxMoeArgs& a, const CUtensorMap& w13, const CUtensorMap& x, const CUtensorMap& w2,
                          const CUtensorMap& h, int max_used, int num_sms, cudaStream_t stream);

}  // namespace qlora
