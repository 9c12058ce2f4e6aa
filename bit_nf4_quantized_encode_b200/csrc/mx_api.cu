// mx_api.cu -- the C entry points of the microscaled 4-bit formats (declared in
// include/qlora.h): argument validation, work-buffer layout, tensor maps and
// launch sequences.  The kernels are in mx_codec.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "mx.h"
#include "qlora.h"

namespace qlora {
namespace {

// Sizes above this would overflow a grid or a TMA coordinate after padding.
constexpr int64_t kMxMaxDim = kMaxDim - 256;

// Descriptor checks before any launch, in the order: NULL, shape, format, then
// (for a non-empty matrix) NULL buffers and alignment.
qlora_status check_mx(const qlora_mx_tensor* t) {
  if (!t) return QLORA_ERR_NULL;
  if (t->rows < 0 || t->cols < 0 || t->rows > kMxMaxDim || t->cols > kMxMaxDim) return QLORA_ERR_SHAPE;
  if (t->format != QLORA_MXFP4 && t->format != QLORA_NVFP4) return QLORA_ERR_UNSUPPORTED;
  if (t->scale_per_row != 0 && (t->format != QLORA_NVFP4 || t->scale_per_row != 1)) return QLORA_ERR_UNSUPPORTED;
  if (t->rows == 0 || t->cols == 0) return QLORA_OK;
  const bool g = t->format == QLORA_NVFP4;
  if (!t->codes || !t->scales || (g && !t->global_scale)) return QLORA_ERR_NULL;
  if (!aligned16(t->codes) || !aligned16(t->scales) || (g && !aligned16(t->global_scale))) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

size_t quantize_workspace(int format, int per_row) {
  return format == QLORA_NVFP4 && !per_row ? round_up(kMxAmaxGrid * sizeof(uint32_t), 256) : 0;
}

}  // namespace
}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status qlora_mx_sizes(int64_t rows, int64_t cols, int32_t format, int32_t scale_per_row, size_t* codes_bytes,
                            size_t* scales_bytes, size_t* global_scale_bytes, size_t* workspace_bytes) {
  if (rows < 0 || cols < 0 || rows > kMxMaxDim || cols > kMxMaxDim) return QLORA_ERR_SHAPE;
  if (format != QLORA_MXFP4 && format != QLORA_NVFP4) return QLORA_ERR_UNSUPPORTED;
  if (scale_per_row != 0 && (format != QLORA_NVFP4 || scale_per_row != 1)) return QLORA_ERR_UNSUPPORTED;
  if (codes_bytes) *codes_bytes = static_cast<size_t>(rows) * mx_pitch(cols);
  if (scales_bytes) *scales_bytes = static_cast<size_t>(mx_scale_bytes(format, rows, cols));
  if (global_scale_bytes)
    *global_scale_bytes = format == QLORA_NVFP4 ? 4 * (scale_per_row ? static_cast<size_t>(rows) : 1) : 0;
  if (workspace_bytes) *workspace_bytes = quantize_workspace(format, scale_per_row);
  return QLORA_OK;
}

qlora_status qlora_mx_quantize(const uint16_t* W, int32_t transpose, const qlora_mx_tensor* out, void* workspace,
                               size_t workspace_bytes, qlora_stream_t stream) {
  qlora_status st = check_mx(out);
  if (st != QLORA_OK) return st;
  if ((transpose != 0 && transpose != 1) || (transpose && out->scale_per_row)) return QLORA_ERR_UNSUPPORTED;
  if (out->rows == 0 || out->cols == 0) return QLORA_OK;
  const size_t need = quantize_workspace(out->format, out->scale_per_row);
  if (!W || (need && !workspace)) return QLORA_ERR_NULL;
  if (!aligned16(W) || (need && !aligned16(workspace))) return QLORA_ERR_ALIGN;
  if (workspace_bytes < need) return QLORA_ERR_WORKSPACE;
  DeviceInfo d;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  MxQuantArgs a{};
  a.in = W;
  a.in_rows = transpose ? out->cols : out->rows;
  a.in_cols = transpose ? out->rows : out->cols;
  a.codes = out->codes;
  a.scales = out->scales;
  a.global_scale = out->global_scale;
  a.rows = out->rows;
  a.cols = out->cols;
  a.pitch = mx_pitch(out->cols);
  a.kt = mx_tiles_k(out->format, out->cols);
  a.tile_rows = (out->rows + 127) / 128 * 128;
  a.per_row = out->scale_per_row;
  if (need) {
    const int64_t numel = out->rows * out->cols;
    const int64_t want = (numel / 8 + 1023) / 1024;      // four vectors a thread
    a.amax = static_cast<uint32_t*>(workspace);
    a.amax_n = static_cast<int>(want < 1 ? 1 : (want > kMxAmaxGrid ? kMxAmaxGrid : want));
    if (counted(launch_mx_amax(W, numel, a.amax, a.amax_n, cs)) != cudaSuccess) return QLORA_ERR_CUDA;
  }
  return counted(launch_mx_quant(out->format, transpose != 0, a, d.num_sms, cs)) == cudaSuccess ? QLORA_OK
                                                                                                  : QLORA_ERR_CUDA;
}

qlora_status qlora_mx_dequantize(const qlora_mx_tensor* W, uint16_t* W_out, qlora_stream_t stream) {
  qlora_status st = check_mx(W);
  if (st != QLORA_OK) return st;
  if (W->rows == 0 || W->cols == 0) return QLORA_OK;
  if (!W_out) return QLORA_ERR_NULL;
  if (!aligned16(W_out)) return QLORA_ERR_ALIGN;
  DeviceInfo d;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  return counted(launch_mx_dequant(W->format, W->codes, W->scales, W->global_scale, W->scale_per_row, W->rows, W->cols,
                                   mx_pitch(W->cols), mx_tiles_k(W->format, W->cols), W_out, d.num_sms,
                                   reinterpret_cast<cudaStream_t>(stream))) == cudaSuccess
             ? QLORA_OK
             : QLORA_ERR_CUDA;
}

}  // extern "C"
