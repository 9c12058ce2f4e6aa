// mx.h -- launch interfaces of the microscaled 4-bit kernels: quantise and
// dequantise (mx_codec.cu), the product (mx_gemm.cu) and the
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
  int amax_n;
};

cudaError_t launch_mx_amax(const uint16_t* in, int64_t numel, uint32_t* partials, int grid, cudaStream_t stream);
cudaError_t launch_mx_quant(int fmt, bool transpose, const MxQuantArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_mx_dequant(int fmt, const uint8_t* codes, const uint8_t* scales, const float* global_scale,
                              int per_row, int64_t rows, int64_t cols, int64_t pitch, int64_t kt, uint16_t* out,
                              int num_sms, cudaStream_t stream);

}  // namespace qlora
