// mx_api.cu -- the C entry points of the microscaled 4-bit formats (declared in
// include/qlora.h): argument validation, work-buffer layout, tensor maps and
// launch sequences.  mx.h names the files of the kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gemm.h"
#include "internal.h"
#include "lora_branch.h"
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

// (rows, cols <= 2^31: the product fits)
size_t quantize_workspace(int format, int per_row, int64_t rows, int64_t cols) {
  return format == QLORA_NVFP4 && !per_row && rows * cols > kMxSmallElements
             ? round_up(kMxAmaxGrid * sizeof(uint32_t), 256)
             : 0;
}

// ------------------------------------------------------------------ linear layer
// Quantised activations [m, k] in a work buffer, from offset `base`.
struct ActLayout {
  size_t codes, scales, global, end;
};
ActLayout act_layout(int format, int64_t m, int64_t k, size_t base) {
  ActLayout l{};
  size_t o = base;
  l.codes = o;  o = round_up(o + static_cast<size_t>(m) * mx_pitch(k), 256);
  l.scales = o; o = round_up(o + static_cast<size_t>(mx_scale_bytes(format, m, k)), 256);
  l.global = o; if (format == QLORA_NVFP4) o = round_up(o + static_cast<size_t>(m) * 4, 256);
  l.end = o;
  return l;
}

// Tokens up to which the product streams the weight (mx_stream.cu) rather than
// tiling the tokens over pairs (mx_pair.cu).
constexpr int64_t kMxStreamTokens = 64;

// The rank contractions' sums leave the tensor core every 512 of the contraction
// (RankProblem::flush).
constexpr int kRankFlush = 8;

// What one product needs beside its operands: a streamed one's counters (one per
// 32 weight rows) and partial tiles.
struct ProductLayout {
  ActLayout act;
  size_t counters, slots, end;
};
ProductLayout product_layout(int format, int64_t rows, int64_t k, int64_t m, size_t base) {
  ProductLayout l{};
  l.act = act_layout(format, m, k, base);
  size_t o = l.act.end;
  l.counters = o;
  l.slots = o;
  if (m <= kMxStreamTokens) {
    o = round_up(o + static_cast<size_t>((rows + 127) / 128) * 16, 256);
    l.slots = o;
    o += size_t{kMxMaxRuns} * 2 * m * 128 * sizeof(float);
  }
  l.end = o;
  return l;
}

// The rank-r activations of a product, two bf16 parts (RankProblem::out_parts).
size_t parts_bytes(int64_t m, const LinearShape& sh) { return static_cast<size_t>(m) * sh.rpad * 4; }

struct MxFwdLayout {
  XaLayout xa;             // of its members only sxa for few tokens
  ProductLayout product;
};
MxFwdLayout mx_fwd_layout(int format, int64_t rows, int64_t cols, int64_t m, int r, const LinearShape& sh) {
  MxFwdLayout l{};
  if (r && m > kMxStreamTokens) l.xa = xa_layout(sh, 2, 0);
  else if (r) l.xa.end = round_up(parts_bytes(m, sh), 256);
  l.product = product_layout(format, rows, cols, m, l.xa.end);
  return l;
}
struct MxBwdLayout {
  BwdLayout lora;
  size_t sg_div;           // NVFP4: s G / (gx gw) for dX
  ProductLayout product;
};
MxBwdLayout mx_bwd_layout(int format, int64_t rows, int64_t cols, int64_t m, int r, const LinearShape& sh) {
  MxBwdLayout l{};
  if (r) l.lora = bwd_layout(sh, 2, false);
  size_t o = round_up(l.lora.total, 256);
  l.sg_div = o;
  if (r && format == QLORA_NVFP4) o = round_up(o + parts_bytes(m, sh), 256);
  l.product = product_layout(format, cols, rows, m, o);
  return l;
}

// Sizes of the layer W [rows, cols] with M tokens and rank r (0: no adapter).
qlora_status mx_layer_shape(int64_t rows, int64_t cols, int64_t M, int32_t r, LinearShape* sh) {
  if (r != 0) return rows > kMxMaxDim || cols > kMxMaxDim || M > kMxMaxDim ? QLORA_ERR_SHAPE
                                                                             : linear_shape(rows, cols, M, r, sh);
  if (rows < 1 || cols < 1 || rows > kMxMaxDim || cols > kMxMaxDim || M < 1 || M > kMxMaxDim) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

// Whether a product's tiles and scale tiles can be counted and addressed in 32 bits.
bool product_fits(int format, int64_t rows, int64_t k, int64_t m) {
  const int64_t kt = mx_tiles_k(format, k), wt = (rows + 127) / 128, xt = (m + 127) / 128;
  return wt * xt <= (int64_t{1} << 28) && wt * kt <= kMxMaxDim && xt * kt <= kMxMaxDim;
}

// Row tiles swept across all token tiles before the next group: about 48 MB of
// weight codes, so that they stay in L2 meanwhile.
int mx_group(int m_tiles, int64_t pitch) {
  int64_t g = (int64_t{48} << 20) / (128 * pitch);
  if (g < 1) g = 1;
  return static_cast<int>(g > m_tiles ? m_tiles : g);
}

// q(X) into the work buffer (NVFP4: a global scale per token).
// Words of the work buffer that later kernels of the call count in ([zero, zero_end)
// bytes, and a streamed product's counters) are cleared on the way: a memset of its
// own takes 4 us in a graph.
cudaError_t quantize_acts(const qlora_mx_tensor* W, const uint16_t* X, int64_t M, uint8_t* ws, const ProductLayout& P,
                          size_t zero, size_t zero_end, const DeviceInfo& d, cudaStream_t cs) {
  const ActLayout& L = P.act;
  MxQuantArgs a{};
  a.in = X;
  a.in_rows = a.rows = a.tile_rows = M;
  a.in_cols = a.cols = W->cols;
  a.codes = ws + L.codes;
  a.scales = ws + L.scales;
  a.global_scale = reinterpret_cast<float*>(ws + L.global);
  a.pitch = mx_pitch(W->cols);
  a.kt = mx_tiles_k(W->format, W->cols);
  a.per_row = W->format == QLORA_NVFP4;
  a.zero[0] = reinterpret_cast<uint32_t*>(ws + zero);
  a.zero_n[0] = static_cast<int>((zero_end - zero) / 4);
  a.zero[1] = reinterpret_cast<uint32_t*>(ws + P.counters);
  a.zero_n[1] = M <= kMxStreamTokens ? static_cast<int>((W->rows + 127) / 128 * 4) : 0;
  return counted(launch_mx_quant(W->format, false, a, d.num_sms, cs));
}

// Token tile of the pair kernel: the one whose waves of tiles over the pairs of
// SMs take less time.
int pair_token_tile(int64_t rows, int64_t m, int num_sms) {
  const int64_t pairs = num_sms / 2, mt = (rows + 255) / 256;
  const int64_t wide = (mt * ((m + 255) / 256) + pairs - 1) / pairs * 2;
  const int64_t narrow = (mt * ((m + 127) / 128) + pairs - 1) / pairs;
  return narrow < wide ? 128 : 256;
}

// Which kernel multiplies, and its token tile.  The backward (not `fwd`) always
// quantises dY in a launch of its own.
enum class MxForm { few, stream, pair };
MxForm product_form(int format, int64_t rows, int64_t k, int64_t m, int lora_steps, bool fwd, int num_sms, int* tile) {
  if (fwd && (*tile = mx_few_tile(format, rows, m, k, lora_steps, num_sms)) != 0) return MxForm::few;
  const bool pair = m > kMxStreamTokens;
  *tile = pair ? pair_token_tile(rows, m, num_sms) : m <= 16 ? 16 : m <= 32 ? 32 : 64;
  return pair ? MxForm::pair : MxForm::stream;
}

// out [M, W->rows] = q(X) deq(W)^T + lora_x lora_w (see mx_stream.cu); lora_x in two
// bf16 parts, [M][2 * 64 lora_steps].
qlora_status run_mx_gemm(const qlora_mx_tensor* W, int64_t M, uint8_t* ws, const ProductLayout& P, const uint16_t* lora_w,
                         bool lora_mn, const uint16_t* lora_x, int r, int lora_steps, uint16_t* out,
                         const DeviceInfo& d, cudaStream_t cs) {
  const ActLayout& L = P.act;
  int bn;
  const bool pair = product_form(W->format, W->rows, W->cols, M, lora_steps, false, d.num_sms, &bn) == MxForm::pair;
  const int box_x = pair ? bn / 2 : bn;
  const int64_t pitch = mx_pitch(W->cols);
  MxGemmArgs a{};
  a.w_scales = W->scales;
  a.x_scales = ws + L.scales;
  a.kt = mx_tiles_k(W->format, W->cols);
  if (W->format == QLORA_NVFP4) {
    a.w_global = W->global_scale;
    a.w_per_row = W->scale_per_row;
    a.x_global = reinterpret_cast<const float*>(ws + L.global);
  }
  a.rows = W->rows;
  a.m = M;
  a.k = W->cols;
  a.ksteps = static_cast<int>((W->cols + 255) / 256);
  a.lora_steps = lora_steps;
  a.lora_mn = lora_mn ? 1 : 0;
  a.out = out;
  const int64_t m_tiles = pair ? (W->rows + 255) / 256 : (W->rows + 127) / 128, t_tiles = (M + bn - 1) / bn;
  const int64_t w_tiles = (W->rows + 127) / 128 * a.kt, x_tiles = (M + 127) / 128 * a.kt;
  a.m_tiles = static_cast<int>(m_tiles);
  a.t_tiles = static_cast<int>(t_tiles);
  a.m_group = mx_group(a.m_tiles, 2 * pitch);
  a.slots = reinterpret_cast<float*>(ws + P.slots);
  a.counters = reinterpret_cast<uint32_t*>(ws + P.counters);
  a.err = d.err;
  MxMaps m;
  const uint64_t up = static_cast<uint64_t>(pitch);
  if (!make_map_u8(&m.w, W->codes, up, static_cast<uint64_t>(W->rows), up, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_u8(&m.x, ws + L.codes, up, static_cast<uint64_t>(M), up, 128, static_cast<uint32_t>(box_x),
                   CU_TENSOR_MAP_SWIZZLE_128B))
    return QLORA_ERR_CUDA;
  if (lora_steps) {
    const uint64_t both = static_cast<uint64_t>(lora_steps) * 128, n = static_cast<uint64_t>(W->rows);
    if (!(lora_mn ? make_map(&m.lora_w, lora_w, n, r, n * 2, 64)
                  : make_map(&m.lora_w, lora_w, r, n, static_cast<uint64_t>(r) * 2, 128)) ||
        !make_map(&m.lora_x, lora_x, both, static_cast<uint64_t>(M), both * 2, static_cast<uint32_t>(box_x)))
      return QLORA_ERR_CUDA;
  } else {
    m.lora_w = m.w;
    m.lora_x = m.x;
  }
  cudaError_t e;
  if (pair) {
    const uint32_t atoms = W->format == QLORA_MXFP4 ? 2 : 4;
    if (!make_map_scales(&m.w_scales, W->scales, static_cast<uint64_t>(w_tiles), atoms) ||
        !make_map_scales(&m.x_scales, a.x_scales, static_cast<uint64_t>(x_tiles), atoms))
      return QLORA_ERR_CUDA;
    e = launch_mx_pair(W->format, bn, a, m, d.num_sms, cs);
  } else {
    e = launch_mx_stream(W->format, bn, a, m, d.num_sms, cs);
  }
  return counted(e) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

// The same with the tokens' quantisation in the product (see mx_few.cu).
qlora_status run_mx_few(const qlora_mx_tensor* W, const uint16_t* X, int64_t M, int tile, const uint16_t* lora_w,
                        const uint16_t* lora_x, int r, int lora_steps, uint16_t* out, const DeviceInfo& d,
                        cudaStream_t cs) {
  MxFewArgs a{};
  a.x = X;
  a.vec = W->cols % 8 == 0;
  a.w_scales = W->scales;
  a.kt = mx_tiles_k(W->format, W->cols);
  if (W->format == QLORA_NVFP4) {
    a.w_global = W->global_scale;
    a.w_per_row = W->scale_per_row;
  }
  a.rows = W->rows;
  a.k = W->cols;
  a.m = static_cast<int>(M);
  a.ksteps = static_cast<int>((W->cols + 255) / 256);
  a.lora_steps = lora_steps;
  a.out = out;
  a.err = d.err;
  MxMaps m;
  const uint64_t up = static_cast<uint64_t>(mx_pitch(W->cols)), n = static_cast<uint64_t>(W->rows);
  if (!make_map_u8(&m.w, W->codes, up, n, up, 128, 32, CU_TENSOR_MAP_SWIZZLE_128B)) return QLORA_ERR_CUDA;
  if (lora_steps) {
    const uint64_t both = static_cast<uint64_t>(lora_steps) * 128;
    if (!make_map(&m.lora_w, lora_w, r, n, static_cast<uint64_t>(r) * 2, 32) ||
        !make_map(&m.lora_x, lora_x, both, static_cast<uint64_t>(M), both * 2, static_cast<uint32_t>(tile)))
      return QLORA_ERR_CUDA;
  } else {
    m.lora_w = m.lora_x = m.w;
  }
  return counted(launch_mx_few(W->format, tile, a, m, d.num_sms, cs)) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

// ------------------------------------------------------------------ mixture of experts
struct MoeLayout {
  size_t x_codes, x_scales, h_codes, h_scales, slots, list, n_used, counters, total;
  int64_t n_counters;
  int max_used;
};
qlora_status moe_layout(int32_t experts, int64_t hidden, int64_t inner, int64_t M, int32_t top_k, MoeLayout* l) {
  if (M < 1 || M > kMoeMaxTokens || experts < 1 || experts > kMoeMaxExperts || top_k < 1 || top_k > kMoeMaxTopK ||
      top_k > experts)
    return QLORA_ERR_SHAPE;
  if (hidden < 128 || inner < 128 || hidden % 128 || inner % 128 || hidden > (1 << 20) || inner > (1 << 20) ||
      experts * 2 * inner > kMxMaxDim || experts * hidden > kMxMaxDim)
    return QLORA_ERR_SHAPE;
  const int64_t pairs = M * top_k;
  l->max_used = static_cast<int>(pairs < experts ? pairs : experts);
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o = round_up(o + n, 256); return at; };
  l->x_codes = take(static_cast<size_t>(M) * hidden / 2);
  l->x_scales = take(static_cast<size_t>(hidden) / 128 * 512);
  l->h_codes = take(static_cast<size_t>(l->max_used) * 16 * inner / 2);
  l->h_scales = take(static_cast<size_t>(l->max_used) * inner / 128 * 512);
  l->slots = take(size_t{kMxMaxRuns} * 2 * 2 * M * 128 * sizeof(float));
  l->list = take(static_cast<size_t>(l->max_used) * sizeof(MoeExpert));
  l->n_used = take(4);
  l->n_counters = hidden / 32 + l->max_used * (inner / 32);
  l->counters = take(static_cast<size_t>(l->n_counters) * 4);
  l->total = o;
  return QLORA_OK;
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
  if (workspace_bytes) *workspace_bytes = quantize_workspace(format, scale_per_row, rows, cols);
  return QLORA_OK;
}

qlora_status qlora_mx_quantize(const uint16_t* W, int32_t transpose, const qlora_mx_tensor* out, void* workspace,
                               size_t workspace_bytes, qlora_stream_t stream) {
  qlora_status st = check_mx(out);
  if (st != QLORA_OK) return st;
  if ((transpose != 0 && transpose != 1) || (transpose && out->scale_per_row)) return QLORA_ERR_UNSUPPORTED;
  if (out->rows == 0 || out->cols == 0) return QLORA_OK;
  const size_t need = quantize_workspace(out->format, out->scale_per_row, out->rows, out->cols);
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

qlora_status qlora_mx_linear_workspace_size(int64_t rows, int64_t cols, int32_t format, int64_t M, int32_t r,
                                            size_t* fwd_bytes, size_t* bwd_bytes) {
  if (format != QLORA_MXFP4 && format != QLORA_NVFP4) return QLORA_ERR_UNSUPPORTED;
  LinearShape sh{};
  const qlora_status st = mx_layer_shape(rows, cols, M, r, &sh);
  if (st != QLORA_OK) return st;
  if (fwd_bytes) *fwd_bytes = mx_fwd_layout(format, rows, cols, M, r, sh).product.end;
  if (bwd_bytes) *bwd_bytes = mx_bwd_layout(format, rows, cols, M, r, sh).product.end;
  return QLORA_OK;
}

qlora_status qlora_mx_linear_fwd(const qlora_mx_tensor* W, const uint16_t* X, int64_t M, const uint16_t* A,
                                 const uint16_t* B, int32_t r, float s, uint16_t* Y, float* XA_out, void* workspace,
                                 size_t workspace_bytes, qlora_stream_t stream) {
  qlora_status st = check_mx(W);
  if (st != QLORA_OK) return st;
  LinearShape sh{};
  if ((st = mx_layer_shape(W->rows, W->cols, M, r, &sh)) != QLORA_OK) return st;
  if (!product_fits(W->format, W->rows, W->cols, M)) return QLORA_ERR_SHAPE;
  if (r && W->scale_per_row) return QLORA_ERR_UNSUPPORTED;
  if (!X || !Y || !workspace || (r && (!A || !B))) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(workspace) ||
      (r && (!aligned16(A) || !aligned16(B) || (XA_out && !aligned16(XA_out)))))
    return QLORA_ERR_ALIGN;
  if (r && !std::isfinite(s)) return QLORA_ERR_SHAPE;
  const MxFwdLayout L = mx_fwd_layout(W->format, W->rows, W->cols, M, r, sh);
  if (workspace_bytes < L.product.end) return QLORA_ERR_WORKSPACE;
  DeviceInfo d;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int few;
  if (product_form(W->format, W->rows, W->cols, M, r ? sh.lora_steps : 0, true, d.num_sms, &few) != MxForm::few) few = 0;
  if (!few && quantize_acts(W, X, M, ws, L.product, L.xa.cnt, L.xa.cnt_end, d, cs) != cudaSuccess) return QLORA_ERR_CUDA;
  const uint16_t* sxa = nullptr;
  if (r) {
    sxa = reinterpret_cast<const uint16_t*>(ws + L.xa.sxa);
    const float* all_div = W->format == QLORA_NVFP4 ? W->global_scale : nullptr;
    if (M > kMxStreamTokens) {
      RankDivide div;
      if (all_div) {
        div.out = reinterpret_cast<uint16_t*>(ws + L.xa.sxa);
        div.row = reinterpret_cast<const float*>(ws + L.product.act.global);
        div.all = all_div;
      }
      if ((st = run_rank_xa(sh, X, A, s, XA_out, ws, L.xa, 2, div, kRankFlush, true, d, cs)) != QLORA_OK) return st;
    } else {
      MxXaArgs xa{};
      xa.x = X;
      xa.a = A;
      xa.k = W->cols;
      xa.m = static_cast<int>(M);
      xa.r = r;
      xa.rpad = sh.rpad;
      xa.s = s;
      xa.xa = XA_out;
      xa.sxa = reinterpret_cast<uint16_t*>(ws + L.xa.sxa);
      xa.all_div = all_div;
      xa.first = few != 0;
      if (counted(launch_mx_xa(xa, cs)) != cudaSuccess) return QLORA_ERR_CUDA;
    }
  }
  if (few) return run_mx_few(W, X, M, few, B, sxa, r, r ? sh.lora_steps : 0, Y, d, cs);
  return run_mx_gemm(W, M, ws, L.product, B, false, sxa, r, r ? sh.lora_steps : 0, Y, d, cs);
}

qlora_status qlora_mx_linear_bwd(const qlora_mx_tensor* WT, const uint16_t* X, const uint16_t* dY, int64_t M,
                                 const uint16_t* A, const uint16_t* B, int32_t r, float s, const float* XA,
                                 uint16_t* dX, float* dA, float* dB, void* workspace, size_t workspace_bytes,
                                 qlora_stream_t stream) {
  qlora_status st = check_mx(WT);
  if (st != QLORA_OK) return st;
  const int64_t rows = WT->cols, cols = WT->rows;          // the layer's W is [rows, cols]
  LinearShape sh{};
  if ((st = mx_layer_shape(rows, cols, M, r, &sh)) != QLORA_OK) return st;
  if (!product_fits(WT->format, cols, rows, M)) return QLORA_ERR_SHAPE;
  if (r && WT->scale_per_row) return QLORA_ERR_UNSUPPORTED;
  if (!dY || !workspace || (!r && !dX) || (r && (!X || !A || !B || !dA || !dB))) return QLORA_ERR_NULL;
  if (!aligned16(dY) || !aligned16(workspace) || (dX && !aligned16(dX)) ||
      (r && (!aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(dA) || !aligned16(dB) ||
             (XA && !aligned16(XA)))))
    return QLORA_ERR_ALIGN;
  if (r && !std::isfinite(s)) return QLORA_ERR_SHAPE;
  MxBwdLayout L = mx_bwd_layout(WT->format, rows, cols, M, r, sh);
  if (workspace_bytes < L.product.end) return QLORA_ERR_WORKSPACE;
  DeviceInfo d;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (dX && quantize_acts(WT, dY, M, ws, L.product, 0, r ? L.lora.clear_end : 0, d, cs) != cudaSuccess) return QLORA_ERR_CUDA;
  const uint16_t* sg = nullptr;
  if (r) {
    // G = dY B and X A^T as the backward over an NF4 weight has them
    RankDivide div;
    sg = reinterpret_cast<const uint16_t*>(ws + L.lora.sg);
    if (dX && WT->format == QLORA_NVFP4) {
      sg = div.out = reinterpret_cast<uint16_t*>(ws + L.sg_div);
      div.row = reinterpret_cast<const float*>(ws + L.product.act.global);
      div.all = WT->global_scale;
    }
    if ((st = run_rank_inputs(sh, X, dY, A, B, s, XA, ws, &L.lora, dX && !div.out, div, kRankFlush, dX != nullptr,
                              d, cs)) != QLORA_OK) return st;
  }
  if (dX && (st = run_mx_gemm(WT, M, ws, L.product, A, true, sg, r, r ? sh.lora_steps : 0, dX, d, cs)) != QLORA_OK) return st;
  return r ? run_lora_grads(sh, X, dY, s, XA, dA, dB, ws, &L.lora, kRankFlush, d, cs) : QLORA_OK;
}

qlora_status qlora_selftest_mx_form(int64_t rows, int64_t cols, int32_t format, int64_t M, int32_t r, int32_t backward,
                                    int32_t num_sms, int32_t* form, int32_t* token_tile) {
  if (format != QLORA_MXFP4 && format != QLORA_NVFP4) return QLORA_ERR_UNSUPPORTED;
  LinearShape sh{};
  const qlora_status st = mx_layer_shape(rows, cols, M, r, &sh);
  if (st != QLORA_OK) return st;
  if (num_sms < 2) return QLORA_ERR_SHAPE;
  if (!form || !token_tile) return QLORA_ERR_NULL;
  *form = static_cast<int32_t>(product_form(format, backward ? cols : rows, backward ? rows : cols, M, r ? sh.lora_steps : 0,
                                            !backward, num_sms, token_tile));
  return QLORA_OK;
}

qlora_status qlora_mx_moe_workspace_size(int32_t experts, int64_t hidden, int64_t inner, int64_t M, int32_t top_k,
                                         size_t* bytes) {
  MoeLayout l{};
  const qlora_status st = moe_layout(experts, hidden, inner, M, top_k, &l);
  if (st == QLORA_OK && bytes) *bytes = l.total;
  return st;
}

qlora_status qlora_mx_moe_fwd(const qlora_mx_tensor* W13, const qlora_mx_tensor* W2, const uint16_t* router,
                              int32_t experts, const uint16_t* X, int64_t M, int32_t top_k, uint16_t* Y, int32_t* ids,
                              float* probs, void* workspace, size_t workspace_bytes, qlora_stream_t stream) {
  qlora_status st = check_mx(W13);
  if (st == QLORA_OK) st = check_mx(W2);
  if (st != QLORA_OK) return st;
  if (W13->format != QLORA_MXFP4 || W2->format != QLORA_MXFP4) return QLORA_ERR_UNSUPPORTED;
  const int64_t hidden = W13->cols, inner = W2->cols;
  MoeLayout l{};
  if ((st = moe_layout(experts, hidden, inner, M, top_k, &l)) != QLORA_OK) return st;
  if (W13->rows != experts * 2 * inner || W2->rows != experts * hidden) return QLORA_ERR_SHAPE;
  if (!router || !X || !Y || !ids || !probs || !workspace) return QLORA_ERR_NULL;
  if (!aligned16(router) || !aligned16(X) || !aligned16(Y) || !aligned16(ids) || !aligned16(probs) ||
      !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  if (workspace_bytes < l.total) return QLORA_ERR_WORKSPACE;
  DeviceInfo d;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MxMoeArgs a{};
  a.x = X;
  a.router = router;
  a.w13_scales = W13->scales;
  a.w2_scales = W2->scales;
  a.hidden = hidden;
  a.inner = inner;
  a.m = static_cast<int>(M);
  a.experts = experts;
  a.top_k = top_k;
  a.y = Y;
  a.ids = ids;
  a.probs = probs;
  a.x_codes = ws + l.x_codes;
  a.x_scales = ws + l.x_scales;
  a.h_codes = ws + l.h_codes;
  a.h_scales = ws + l.h_scales;
  a.slots = reinterpret_cast<float*>(ws + l.slots);
  a.list = reinterpret_cast<MoeExpert*>(ws + l.list);
  a.n_used = reinterpret_cast<int*>(ws + l.n_used);
  a.counters = reinterpret_cast<uint32_t*>(ws + l.counters);
  a.up_counters = a.counters + hidden / 32;
  a.n_counters = static_cast<int>(l.n_counters);
  a.err = d.err;
  const uint64_t hp = static_cast<uint64_t>(hidden) / 2, ip = static_cast<uint64_t>(inner) / 2;
  CUtensorMap w13, w2, x, h;
  if (!make_map_u8(&w13, W13->codes, hp, static_cast<uint64_t>(W13->rows), hp, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_u8(&w2, W2->codes, ip, static_cast<uint64_t>(W2->rows), ip, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_u8(&x, a.x_codes, hp, static_cast<uint64_t>(M), hp, 128, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_u8(&h, a.h_codes, ip, static_cast<uint64_t>(l.max_used) * 16, ip, 128, 16, CU_TENSOR_MAP_SWIZZLE_128B))
    return QLORA_ERR_CUDA;
  return counted(launch_mx_moe(a, w13, x, w2, h, l.max_used, d.num_sms, reinterpret_cast<cudaStream_t>(stream)), 3) ==
                 cudaSuccess
             ? QLORA_OK
             : QLORA_ERR_CUDA;
}

}  // extern "C"
