// lora_branch.cu -- host side of the LoRA branch (see lora_branch.h).
#include "lora_branch.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gemm.h"
#include "lora.h"

namespace qlora {
namespace {

// The work buffer's split slots are sized independently of the device (for up
// to this many SMs); a launch picks its own split count within that space.
constexpr int kSizingSms = 256;
constexpr int kMaxRankSplits = 32;

// Splits of a launch with `tiles` tiles in all (the problems of one launch
// share them) and `ksteps` k-steps, within `slot_bytes` of slot space.
int launch_splits(int tiles, int ksteps, int num_sms, size_t slot_bytes) {
  // a split count s > 1 needs tiles * s partial tiles of slot space
  const size_t per_split = static_cast<size_t>(tiles) * 64 * 128 * sizeof(float);
  size_t cap = kMaxRankSplits;
  if (per_split > 0 && slot_bytes / per_split < cap) cap = slot_bytes / per_split;
  return rank_splits(tiles, ksteps, num_sms, cap < 2 ? 1 : static_cast<int>(cap));
}
// The plan of a launch must fit its slot region; checked before every launch.
bool slots_fit(int tiles, int splits, size_t slot_bytes) {
  return rank_slot_bytes(tiles, splits) <= slot_bytes;
}
// One rank-r problem of a k_rank launch.
RankProblem rank_problem(const RankPlan& pl, int64_t mdim, int64_t ndim, bool a_mn, bool b_mn, int unit_begin,
                         float* slots, uint32_t* counters) {
  RankProblem p{};
  p.mdim = mdim;
  p.ndim = ndim;
  p.ksteps = pl.ksteps;
  p.m_tiles = pl.m_tiles;
  p.n_tiles = pl.n_tiles;
  p.splits = pl.splits;
  p.unit_begin = unit_begin;
  p.a_mn = a_mn ? 1 : 0;
  p.b_mn = b_mn ? 1 : 0;
  p.slots = slots;
  p.counters = counters;
  return p;
}

}  // namespace

qlora_status linear_shape(int64_t rows, int64_t cols, int64_t M, int32_t r, LinearShape* sh) {
  if (M < 1 || M > kMaxDim) return QLORA_ERR_SHAPE;
  if (rows < 8 || cols < 64 || rows > kMaxDim || cols > kMaxDim || cols % 64 != 0 || rows % 8 != 0)
    return QLORA_ERR_SHAPE;
  if (r < 8 || r > 256 || r % 8 != 0) return QLORA_ERR_SHAPE;
  sh->rows = rows;
  sh->cols = cols;
  sh->m = M;
  sh->r = r;
  sh->lora_steps = (r + 63) / 64;
  sh->rpad = 64 * sh->lora_steps;
  sh->decode = M <= 16;
  return QLORA_OK;
}

RankPlan rank_tiling(int64_t mdim, int64_t contraction, int lora_steps) {
  RankPlan p;
  p.m_tiles = static_cast<int>((mdim + 127) / 128);
  p.n_tiles = lora_steps;
  p.ksteps = static_cast<int>((contraction + 63) / 64);
  p.splits = 1;
  return p;
}
size_t sized_slots(int tiles, int ksteps) {
  static const int kSmCounts[] = {96, 108, 114, 120, 128, 132, 144, 148, 152, 160, 170, 188, 192, 224, kSizingSms};
  size_t most = 0;
  for (int sms : kSmCounts) {
    const size_t b = rank_slot_bytes(tiles, rank_splits(tiles, ksteps, sms, kMaxRankSplits));
    if (b > most) most = b;
  }
  return most;
}

// Work buffer layout, in bytes, each offset 256-aligned; every size is
// independent of the device.
XaLayout xa_layout(const LinearShape& s, int parts, size_t base) {
  XaLayout l{};
  const RankPlan xa = rank_tiling(s.m, s.cols, s.lora_steps);
  size_t o = base;
  l.cnt = o;   o = round_up(o + size_t(xa.tiles()) * 4, 256);
  l.cnt_end = o;
  l.slot_bytes = sized_slots(xa.tiles(), xa.ksteps);
  l.slots = o; o = round_up(o + l.slot_bytes, 256);
  l.sxa = o;   o = round_up(o + size_t(s.m) * s.rpad * 2 * parts, 256);
  l.end = o;
  return l;
}

// The region cleared by one memset first (counters, and dx_acc), then the rest.
BwdLayout bwd_layout(const LinearShape& s, int parts, bool split_dx) {
  BwdLayout l{};
  l.parts = parts;
  l.g_plan = rank_tiling(s.m, s.rows, s.lora_steps);
  l.xa_plan = rank_tiling(s.m, s.cols, s.lora_steps);
  l.db_plan = rank_tiling(s.rows, s.m, s.lora_steps);
  l.da_plan = rank_tiling(s.cols, s.m, s.lora_steps);
  const int k1 = l.g_plan.ksteps > l.xa_plan.ksteps ? l.g_plan.ksteps : l.xa_plan.ksteps;
  const size_t alone = sized_slots(l.g_plan.tiles(), l.g_plan.ksteps);
  const size_t both = sized_slots(l.g_plan.tiles() + l.xa_plan.tiles(), k1);
  l.slots1_bytes = alone > both ? alone : both;
  l.slots2_bytes = s.decode ? 0 : sized_slots(l.db_plan.tiles() + l.da_plan.tiles(), l.db_plan.ksteps);
  size_t o = 0;
  l.cnt1 = o;   o = round_up(o + size_t(l.g_plan.tiles() + l.xa_plan.tiles()) * 4, 256);
  l.cnt2 = o;   o = round_up(o + size_t(l.db_plan.tiles() + l.da_plan.tiles()) * 4, 256);
  l.dx_acc = o; if (split_dx) o = round_up(o + size_t(s.m) * s.cols * 4, 256);
  l.clear_end = o;
  l.slots1 = o; o = round_up(o + l.slots1_bytes, 256);
  l.slots2 = o; o = round_up(o + l.slots2_bytes, 256);
  l.g = o;      if (s.decode) o = round_up(o + size_t(s.m) * s.rpad * 4, 256);
  l.xa = o;     if (s.decode) o = round_up(o + size_t(s.m) * s.rpad * 4, 256);
  l.sg = o;     o = round_up(o + size_t(s.m) * s.rpad * 2 * parts, 256);
  l.sxa = o;    o = round_up(o + size_t(s.m) * s.rpad * 2 * parts, 256);
  l.total = o;
  return l;
}

qlora_status run_rank_xa(const LinearShape& sh, const uint16_t* X, const uint16_t* A, float s, float* XA_out, uint8_t* ws,
                         const XaLayout& L, int parts, const RankDivide& div, int flush, bool cleared, const DeviceInfo& d,
                         cudaStream_t cs) {
  RankPlan xp = rank_tiling(sh.m, sh.cols, sh.lora_steps);
  xp.splits = launch_splits(xp.tiles(), xp.ksteps, d.num_sms, L.slot_bytes);
  if (!slots_fit(xp.tiles(), xp.splits, L.slot_bytes)) return QLORA_ERR_WORKSPACE;
  if (xp.splits > 1 && !cleared && cudaMemsetAsync(ws + L.cnt, 0, L.cnt_end - L.cnt, cs) != cudaSuccess) return QLORA_ERR_CUDA;
  CUtensorMap x_k, a_k;
  if (!make_map(&x_k, X, sh.cols, sh.m, sh.cols * 2, 128) || !make_map(&a_k, A, sh.cols, sh.r, sh.cols * 2, 64))
    return QLORA_ERR_CUDA;
  RankArgs ra{};
  ra.p[0] = rank_problem(xp, sh.m, sh.r, false, false, 0, reinterpret_cast<float*>(ws + L.slots),
                         reinterpret_cast<uint32_t*>(ws + L.cnt));
  ra.p[0].flush = flush;
  ra.p[0].out_f32 = XA_out; ra.p[0].ld_f32 = sh.r;
  ra.p[0].ld_bf16 = sh.rpad; ra.p[0].bf16_cols = sh.rpad; ra.p[0].bf16_scale = s;
  uint16_t* sxa = reinterpret_cast<uint16_t*>(ws + L.sxa);
  ra.p[0].out_div = div.out; ra.p[0].row_div = div.row; ra.p[0].all_div = div.all;
  if (!div.out) (parts == 2 ? ra.p[0].out_parts : ra.p[0].out_bf16) = sxa;
  ra.nprob = 1;
  ra.total_units = xp.tiles() * xp.splits;
  ra.err = d.err;
  return counted(launch_rank(ra, x_k, a_k, x_k, a_k, d.num_sms, cs)) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

qlora_status run_rank_inputs(const LinearShape& sh, const uint16_t* X, const uint16_t* dY, const uint16_t* A,
                             const uint16_t* B, float s, const float* XA, uint8_t* ws, BwdLayout* L,
                             bool sg_for_dx, const RankDivide& div, int flush, bool cleared, const DeviceInfo& d,
                             cudaStream_t cs) {
  float* g32 = sh.decode ? reinterpret_cast<float*>(ws + L->g) : nullptr;     // fp32 G and X A^T: few-token grads
  float* xa32 = sh.decode ? reinterpret_cast<float*>(ws + L->xa) : nullptr;
  uint16_t* sg = reinterpret_cast<uint16_t*>(ws + L->sg);
  uint16_t* sxa = reinterpret_cast<uint16_t*>(ws + L->sxa);
  const bool recompute = XA == nullptr;
  if (!cleared && cudaMemsetAsync(ws, 0, L->clear_end, cs) != cudaSuccess) return QLORA_ERR_CUDA;
  CUtensorMap dy_k, b_mn, x_k, a_k;
  if (!make_map(&dy_k, dY, sh.rows, sh.m, sh.rows * 2, 128) ||
      !make_map(&b_mn, B, sh.r, sh.rows, sh.r * 2, 64) ||
      !make_map(&x_k, X, sh.cols, sh.m, sh.cols * 2, 128) ||
      !make_map(&a_k, A, sh.cols, sh.r, sh.cols * 2, 64))
    return QLORA_ERR_CUDA;
  {
    // splits for this device and this form of launch 1, within the slot space
    if (recompute) {
      const int k1 = L->g_plan.ksteps > L->xa_plan.ksteps ? L->g_plan.ksteps : L->xa_plan.ksteps;
      L->g_plan.splits = L->xa_plan.splits =
          launch_splits(L->g_plan.tiles() + L->xa_plan.tiles(), k1, d.num_sms, L->slots1_bytes);
      // the split count follows the longer contraction: a split of the shorter one
      // without a k-step would hand on an accumulator that nothing has written
      if (L->g_plan.splits > L->g_plan.ksteps) L->g_plan.splits = L->g_plan.ksteps;
      if (L->xa_plan.splits > L->xa_plan.ksteps) L->xa_plan.splits = L->xa_plan.ksteps;
    } else {
      L->g_plan.splits = launch_splits(L->g_plan.tiles(), L->g_plan.ksteps, d.num_sms, L->slots1_bytes);
    }
    if (rank_slot_bytes(L->g_plan.tiles(), L->g_plan.splits) +
            (recompute ? rank_slot_bytes(L->xa_plan.tiles(), L->xa_plan.splits) : 0) > L->slots1_bytes)
      return QLORA_ERR_WORKSPACE;
    RankArgs ra{};
    uint32_t* cnt = reinterpret_cast<uint32_t*>(ws + L->cnt1);
    float* slots = reinterpret_cast<float*>(ws + L->slots1);
    ra.p[0] = rank_problem(L->g_plan, sh.m, sh.r, false, true, 0, slots, cnt);
    ra.p[0].out_f32 = g32; ra.p[0].ld_f32 = sh.rpad;
    const bool two = L->parts == 2;
    ra.p[0].flush = flush;
    // (its parts only where dA or dX takes them)
    if (!two || !sh.decode || sg_for_dx) (two ? ra.p[0].out_parts : ra.p[0].out_bf16) = sg;
    ra.p[0].ld_bf16 = sh.rpad; ra.p[0].bf16_cols = sh.rpad; ra.p[0].bf16_scale = s;
    ra.p[0].out_div = div.out; ra.p[0].row_div = div.row; ra.p[0].all_div = div.all;
    ra.nprob = 1;
    ra.total_units = L->g_plan.tiles() * L->g_plan.splits;
    if (recompute) {
      ra.p[1] = rank_problem(L->xa_plan, sh.m, sh.r, false, false, ra.total_units,
                             slots + rank_slot_bytes(L->g_plan.tiles(), L->g_plan.splits) / 4,
                             cnt + L->g_plan.tiles());
      ra.p[1].flush = flush;
      ra.p[1].out_f32 = xa32; ra.p[1].ld_f32 = sh.rpad;
      if (!sh.decode) (two ? ra.p[1].out_parts : ra.p[1].out_bf16) = sxa;
      ra.p[1].ld_bf16 = sh.rpad; ra.p[1].bf16_cols = sh.rpad; ra.p[1].bf16_scale = s;
      ra.nprob = 2;
      ra.total_units += L->xa_plan.tiles() * L->xa_plan.splits;
    } else if (!sh.decode) {
      ra.cvt_in = XA; ra.cvt_rows = sh.m; ra.cvt_cols = sh.r; ra.cvt_ld_in = sh.r;
      ra.cvt_out = sxa; ra.cvt_ld_out = sh.rpad * L->parts; ra.cvt_cols_out = sh.rpad; ra.cvt_scale = s;
      ra.cvt_parts = two ? 1 : 0;
    }
    ra.err = d.err;
    if (counted(launch_rank(ra, dy_k, b_mn, x_k, a_k, d.num_sms, cs)) != cudaSuccess) return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}

qlora_status run_lora_grads(const LinearShape& sh, const uint16_t* X, const uint16_t* dY, float s, const float* XA,
                            float* dA, float* dB, uint8_t* ws, BwdLayout* L, int flush, const DeviceInfo& d,
                            cudaStream_t cs) {
  const uint16_t* sg = reinterpret_cast<const uint16_t*>(ws + L->sg);
  const uint16_t* sxa = reinterpret_cast<const uint16_t*>(ws + L->sxa);
  // few tokens: fp32 on CUDA cores from the fp32 G and X A^T
  if (sh.decode) {
    const float* g32 = reinterpret_cast<const float*>(ws + L->g);
    const float* xa = XA ? XA : reinterpret_cast<const float*>(ws + L->xa);
    const int64_t ld_xa = XA ? sh.r : sh.rpad;
    if (counted(launch_small_grads(g32, sh.rpad, xa, ld_xa, X, dY, sh.m, sh.rows, sh.cols, sh.r, s,
                                   dA, dB, d.num_sms, cs)) != cudaSuccess)
      return QLORA_ERR_CUDA;
    return QLORA_OK;
  }
  // many tokens, one launch of two contractions over the tokens (bf16 operands, the
  // rank-r ones in as many parts as launch 1 left):
  // dB = dY^T (s X A^T) [rows, r] and dA = (X^T (s G))^T [r, cols], stored transposed.
  CUtensorMap dy_mn, sxa_mn, x_mn, sg_mn;
  if (!make_map(&dy_mn, dY, sh.rows, sh.m, sh.rows * 2, 64) ||
      !make_map(&sxa_mn, sxa, sh.rpad * L->parts, sh.m, sh.rpad * L->parts * 2, 64) ||
      !make_map(&x_mn, X, sh.cols, sh.m, sh.cols * 2, 64) ||
      !make_map(&sg_mn, sg, sh.rpad * L->parts, sh.m, sh.rpad * L->parts * 2, 64))
    return QLORA_ERR_CUDA;
  L->db_plan.splits = L->da_plan.splits =
      launch_splits(L->db_plan.tiles() + L->da_plan.tiles(), L->db_plan.ksteps, d.num_sms, L->slots2_bytes);
  if (!slots_fit(L->db_plan.tiles() + L->da_plan.tiles(), L->db_plan.splits, L->slots2_bytes))
    return QLORA_ERR_WORKSPACE;
  RankArgs rb{};
  uint32_t* cnt2 = reinterpret_cast<uint32_t*>(ws + L->cnt2);
  float* slots2 = reinterpret_cast<float*>(ws + L->slots2);
  rb.p[0] = rank_problem(L->db_plan, sh.rows, sh.r, true, true, 0, slots2, cnt2);
  rb.p[0].out_f32 = dB; rb.p[0].ld_f32 = sh.r;
  const int u0 = L->db_plan.tiles() * L->db_plan.splits;
  rb.p[1] = rank_problem(L->da_plan, sh.cols, sh.r, true, true, u0,
                         slots2 + rank_slot_bytes(L->db_plan.tiles(), L->db_plan.splits) / 4,
                         cnt2 + L->db_plan.tiles());
  rb.p[1].out_f32 = dA; rb.p[1].ld_f32 = sh.cols; rb.p[1].transpose = 1;
  rb.nprob = 2;
  rb.total_units = u0 + L->da_plan.tiles() * L->da_plan.splits;
  rb.p[0].flush = rb.p[1].flush = flush;
  rb.b_parts = L->parts == 2 ? 1 : 0;
  rb.err = d.err;
  if (counted(launch_rank(rb, dy_mn, sxa_mn, x_mn, sg_mn, d.num_sms, cs)) != cudaSuccess) return QLORA_ERR_CUDA;
  return QLORA_OK;
}

}  // namespace qlora
