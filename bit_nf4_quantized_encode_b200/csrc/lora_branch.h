// lora_branch.h -- the LoRA branch of a linear layer as the host sees it:
// tilings and work-buffer layouts of its rank-r contractions and the launches
// shared by the layers over NF4 (api.cu) and microscaled (mx_api.cu) weights.
// Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"
#include "lora.h"

namespace qlora {

struct LinearShape {
  int64_t rows, cols, m;
  int r, rpad, lora_steps;
  bool decode;      // M <= 16: token tile 16, split-K
};

// The shape of a layer W [rows, cols] with rank r and M token rows, after
// checking r, M, rows and cols; QLORA_ERR_SHAPE otherwise.
qlora_status linear_shape(int64_t rows, int64_t cols, int64_t M, int32_t r, LinearShape* sh);

// One rank-r contraction's tiling: tiles of 128 rows x 64 columns, K splits.
struct RankPlan {
  int m_tiles, n_tiles, ksteps, splits;
  int tiles() const { return m_tiles * n_tiles; }
};
RankPlan rank_tiling(int64_t mdim, int64_t contraction, int lora_steps);
// Slot space of a launch: the most any SM count plans for, so a buffer sized
// without a device lets the launch use its own best split count.
size_t sized_slots(int tiles, int ksteps);

// Work space of X A^T -> bf16(s X A^T) (offsets from `base`): counters (cleared
// by the launch when it splits), partial tiles, the bf16 [M, parts * rpad] result
// (parts: 1 rounded, 2 as RankProblem::out_parts).
struct XaLayout {
  size_t cnt, cnt_end, slots, slot_bytes, sxa, end;
};
XaLayout xa_layout(const LinearShape& s, int parts, size_t base);

// Backward: launch 1 = dY B (and X A^T when it is not supplied), launch 2 =
// dX, launch 3 = dY^T (s X A^T) and X^T (s dY B) (more than 16 tokens; with
// fewer, k_small_grads from the fp32 G and X A^T).  Launch 1's slot space
// covers both of its forms.  parts: how many bf16 parts s G and s X A^T have (1:
// rounded; 2: RankProblem::out_parts).  dx_acc: the fp32 [M, cols] in which the
// decode backward over an NF4 weight adds up dX (split_dx), cleared with the counters.
struct BwdLayout {
  int parts;
  size_t cnt1, cnt2, dx_acc, clear_end, slots1, slots1_bytes, slots2, slots2_bytes, g, xa, sg, sxa, total;
  RankPlan g_plan, xa_plan, db_plan, da_plan;
};
BwdLayout bwd_layout(const LinearShape& s, int parts, bool split_dx);

// Rank-r activations as out_div of RankProblem; out null: none.
struct RankDivide {
  uint16_t* out = nullptr;
  const float* row = nullptr;
  const float* all = nullptr;
};

// XA = X A^T (fp32 to XA_out when asked) and bf16(s XA) [M, rpad], zero-padded
// to a multiple of 64 columns, or (parts = 2) its two parts, or `div` in its place;
// `flush` as RankProblem's; `cleared`: a kernel before has zeroed the counters
// [cnt, cnt_end).
qlora_status run_rank_xa(const LinearShape& sh, const uint16_t* X, const uint16_t* A, float s, float* XA_out, uint8_t* ws,
                         const XaLayout& L, int parts, const RankDivide& div, int flush, bool cleared, const DeviceInfo& d,
                         cudaStream_t cs);
// Launch 1 of the backward, after clearing [0, clear_end) (`cleared`: a kernel before
// has).  dX takes s G from L->sg (sg_for_dx) or divided from `div`; `flush` as
// RankProblem's.
qlora_status run_rank_inputs(const LinearShape& sh, const uint16_t* X, const uint16_t* dY, const uint16_t* A,
                             const uint16_t* B, float s, const float* XA, uint8_t* ws, BwdLayout* L,
                             bool sg_for_dx, const RankDivide& div, int flush, bool cleared, const DeviceInfo& d,
                             cudaStream_t cs);
// Launch 3: dA and dB.
qlora_status run_lora_grads(const LinearShape& sh, const uint16_t* X, const uint16_t* dY, float s, const float* XA,
                            float* dA, float* dB, uint8_t* ws, BwdLayout* L, int flush, const DeviceInfo& d,
                            cudaStream_t cs);

}  // namespace qlora
