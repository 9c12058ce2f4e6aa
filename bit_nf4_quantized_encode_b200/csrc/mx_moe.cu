// mx_moe.cu -- a whole mixture-of-experts feed-forward layer for at most 16
// tokens over MXFP4 experts (sm_100a), in three launches:
//
//   k_moe_route  logits = x R^T (fp32); per token the top_k largest (the lowest
//                index first among equal ones) and p = softmax over them; the
//                list of experts in use with their tokens; q(x).
//   k_moe_up     per expert in use: [g; u] = W13 q(x), h = g / (1 + e^-g) * u, q(h).
//   k_moe_down   per expert in use: o = W2 q(h); y[t] = sum_j p[t, j] o_j[t],
//                summed in the order of j by the CTA that completes a row tile.
//
// Both products are those of mx_stream.cu: the weight is the 128-row operand of
// tcgen05's block-scaled kind, the 16 token slots the other one, whichever of
// them an expert serves.  An expert in use has its weight read once, whatever
// the number of its tokens, which is what bounds the layer (17/32 byte per
// weight).  A block of q(h) is 32 rows of the product's tile, the 32 lanes of
// one epilogue warp.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_encode.cuh"
#include "mx_format.cuh"
#include "mx_ptx.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

// ------------------------------------------------------------------ routing
// One cluster of eight CTAs.  The logits are an [experts, 16] product over hidden:
// a CTA takes an eighth of hidden, its warps groups of 16 experts (several warps a
// group where there are few), with m16n8k16 (bf16 in, fp32 sums).  The parts of
// an expert meet in the CTA that owns it (expert mod 8), summed in a fixed order,
// and the logits in the first CTA, which chooses.  Latency is all there is: every
// load of a warp is issued at once.
constexpr int kRouteCtas = 8;
constexpr int kRouteThreads = 512, kRouteWarps = kRouteThreads / 32;

// Order-preserving key of a logit, above 0 (0 marks a taken one); NaN lowest.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));        // -0 is 0
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

// Shared memory: the logits [16][experts] (the first CTA's), the owner's parts
// [8][ceil(experts / 8)][16] and the warps' tiles [16][16][16].
__host__ __device__ constexpr size_t route_smem(int experts) {
  return sizeof(float) * (static_cast<size_t>(16) * experts + static_cast<size_t>(128) * ((experts + 7) / 8) + 16 * 256);
}

__global__ void __launch_bounds__(kRouteThreads) __cluster_dims__(kRouteCtas, 1, 1)
k_moe_route(const MxMoeArgs a) {
  extern __shared__ float smem[];
  __shared__ int s_id[16][16];
  __shared__ uint32_t s_used[kMoeMaxExperts / 32];
  const int per_owner = (a.experts + 7) / 8;
  float* s_logit = smem;
  float* s_in = s_logit + 16 * a.experts;
  float* s_tile = s_in + 128 * per_owner;
  const int warp = warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_rank());
  asm volatile("griddepcontrol.launch_dependents;");

  // q(x): one warp per 1024 elements
  const int segs = static_cast<int>((a.hidden + 1023) / 1024), kt = static_cast<int>(a.hidden / 128);
  for (int u = rank * kRouteWarps + warp; u < a.m * segs; u += kRouteCtas * kRouteWarps) {
    const int tok = u / segs, c = (u - tok * segs) * 1024 + lane * 32;
    const Elems32 e = load32<true>(a.x + static_cast<int64_t>(tok) * a.hidden, c, a.hidden);
    uint32_t sb;
    const uint4 codes = encode32<kMxFp4>(e, 1.0f, sb);
    uint32_t word = sb << (8 * (lane & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    if (c < a.hidden) {                                           // whole tiles of four lanes: hidden % 128 == 0
      *reinterpret_cast<uint4*>(a.x_codes + static_cast<int64_t>(tok) * (a.hidden / 2) + (c >> 1)) = codes;
      if ((lane & 3) == 0) *reinterpret_cast<uint32_t*>(a.x_scales + mx_scale_offset(tok, c / 32, kt)) = word;
    }
  }

  cluster_sync();                          // every CTA runs before the others write to it

  // logits
  const int groups = (a.experts + 15) / 16;
  const int share = groups >= kRouteWarps ? 1 : kRouteWarps / groups;          // warps of a group
  const int steps = static_cast<int>(a.hidden / 64);
  const int s0 = steps * rank / kRouteCtas, s1 = steps * (rank + 1) / kRouteCtas;
  const int64_t row = a.hidden / 8;                                            // of 16-byte pieces
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int round = 0; round * kRouteWarps < groups * share; ++round) {
    const int slot = round * kRouteWarps + warp, grp = slot / share, sub = slot - grp * share;
    if (grp < groups) {
      const int e0 = grp * 16;
      const bool ra = e0 + g < a.experts, rb = e0 + g + 8 < a.experts, ta = g < a.m, tb = g + 8 < a.m;
      const uint4* pa = reinterpret_cast<const uint4*>(a.router) + (e0 + g) * row + t;
      const uint4* xa = reinterpret_cast<const uint4*>(a.x) + g * row + t;
      float d[2][4] = {};
#pragma unroll 2
      for (int s = s0 + sub; s < s1; s += share) {
        uint4 w[2][2], x[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int o = s * 8 + h * 4;
          w[h][0] = ra ? __ldg(pa + o) : zero;
          w[h][1] = rb ? __ldg(pa + 8 * row + o) : zero;
          x[h][0] = ta ? __ldg(xa + o) : zero;
          x[h][1] = tb ? __ldg(xa + 8 * row + o) : zero;
        }
        // a lane's eight columns feed two products of 16, in the same order on both sides
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0[4] = {w[h][0].x, w[h][1].x, w[h][0].y, w[h][1].y};
          const uint32_t a1[4] = {w[h][0].z, w[h][1].z, w[h][0].w, w[h][1].w};
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t b0[2] = {x[h][n].x, x[h][n].y}, b1[2] = {x[h][n].z, x[h][n].w};
            mma_16x8x16(d[n], a0, b0);
            mma_16x8x16(d[n], a1, b1);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_tile[warp * 256 + (g + 8 * (i >> 1)) * 16 + 8 * n + 2 * t + (i & 1)] = d[n][i];
    }
    __syncthreads();
    // this round's experts: the warps of a group in order, to the owner
    const int here = min(groups - round * kRouteWarps / share, kRouteWarps / share);
    for (int i = threadIdx.x; i < here * 256; i += kRouteThreads) {
      const int lg = i >> 8, e = (round * kRouteWarps / share + lg) * 16 + ((i >> 4) & 15), tok = i & 15;
      float v = 0.0f;
      for (int q = 0; q < share; ++q) v += s_tile[(lg * share + q) * 256 + (i & 255)];
      if (e < a.experts)
        st_cluster_f32(cluster_map(smem_u32(s_in + (rank * per_owner + (e >> 3)) * 16 + tok), static_cast<uint32_t>(e & 7)), v);
    }
    __syncthreads();
  }
  cluster_sync();
  for (int i = threadIdx.x; i < per_owner * 16; i += kRouteThreads) {
    const int e = (i >> 4) * 8 + rank, tok = i & 15;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kRouteCtas; ++q) v += s_in[(q * per_owner) * 16 + i];
    if (e < a.experts) st_cluster_f32(cluster_map(smem_u32(s_logit + tok * a.experts + e), 0), v);
  }
  cluster_sync();
  if (rank != 0) return;

  // top-k: one warp per token, top_k rounds of "largest key, lowest index"
  if (warp < a.m) {
    const float* logit = s_logit + warp * a.experts;
    float first = 0.0f, mine = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
      for (int e = lane; e < a.experts; e += 32) {
        bool taken = false;
        for (int i = 0; i < j; ++i) taken |= s_id[warp][i] == e;
        const uint32_t k = taken ? 0u : logit_key(logit[e]);
        if (k > best) { best = k; at = e; }
      }
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      const int id = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
      const float v = logit[id];
      if (j == 0) first = v;
      if (lane == j) mine = expf(v - first);
      if (lane == 0) s_id[warp][j] = id;
      __syncwarp();
    }
    float sum = lane < a.top_k ? mine : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < a.top_k) {
      a.ids[warp * a.top_k + lane] = s_id[warp][lane];
      a.probs[warp * a.top_k + lane] = __fdiv_rn(mine, sum);
    }
  }
  for (int i = threadIdx.x; i < static_cast<int>(a.hidden / 128); i += kRouteThreads) a.counters[i] = 0u;
  for (int i = threadIdx.x; i < kMoeMaxExperts / 32; i += kRouteThreads) s_used[i] = 0u;
  __syncthreads();
  // the experts in use, in ascending order: id, tokens (bits), and per token its j
  for (int i = threadIdx.x; i < a.m * a.top_k; i += kRouteThreads) {
    const int e = s_id[i / a.top_k][i % a.top_k];
    atomicOr(&s_used[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.m * a.top_k; i += kRouteThreads) {
    const int tok = i / a.top_k, e = s_id[tok][i % a.top_k];
    MoeExpert x;
    x.id = e;
    x.tokens = 0;
    x.slots = 0;
    bool lowest = true;                                           // the expert's first token writes its entry
    for (int q = 0; q < a.m; ++q)
      for (int j = 0; j < a.top_k; ++j)
        if (s_id[q][j] == e) {
          lowest &= q >= tok;
          x.tokens |= 1u << q;
          x.slots |= static_cast<uint64_t>(j) << (4 * q);
        }
    if (!lowest) continue;
    int at = __popc(s_used[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < (e >> 5); ++w) at += __popc(s_used[w]);
    a.list[at] = x;
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < (a.experts + 31) / 32; ++w) n += __popc(s_used[w]);
    *a.n_used = n;
  }
}

// ------------------------------------------------------------------ the two products
constexpr int kThreads = 6 * 32;            // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kTile = 128 * 128;            // 128 rows x 256 codes
constexpr int kSlots = 16;                  // token slots: the N operand
constexpr int kAtoms = 2;

// k_moe_up: gate and up tile per stage; k_moe_down: one tile.
__host__ __device__ constexpr int moe_tiles(bool up) { return up ? 2 : 1; }
__host__ __device__ constexpr int moe_stage(bool up) {
  return moe_tiles(up) * (kTile + kAtoms * 512) + kSlots * 128 + kAtoms * 512;
}
__host__ __device__ constexpr int moe_stages(bool up) { return up ? 5 : 10; }
__host__ __device__ constexpr size_t moe_smem(bool up) {
  return 1024 + static_cast<size_t>(moe_stages(up)) * moe_stage(up) + 256;
}
constexpr uint32_t kMoeCols = 128;          // TMEM columns

template <bool kUp>
__global__ void __launch_bounds__(kThreads, 1)
k_moe_product(const MxMoeArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap) {
  constexpr int kStages = moe_stages(kUp);
  constexpr int kStageBytes = moe_stage(kUp);
  constexpr int kW = moe_tiles(kUp);
  constexpr uint32_t kAcc = kW * kSlots;                          // columns of one accumulator set
  constexpr uint32_t kSfw = 2 * kAcc, kSfx = kSfw + kW * 4 * kAtoms;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_gen + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;      // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* epi_bar = acc_empty + 2;         // the 128 epilogue threads meet here (bounded waits)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  uint32_t* last_flag = tmem_slot + 1;

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int splits = kUp ? a.splits : 1;
  const int sp = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t k = kUp ? a.hidden : a.inner;                     // contraction
  const int row_tiles = static_cast<int>((kUp ? a.inner : a.hidden) / 128);
  const int kt = static_cast<int>(k / 128);                       // scale tiles along k
  const int ksteps = static_cast<int>((k + 255) / 256);
  const int kbeg = ksteps * sp / splits, kend = ksteps * (sp + 1) / splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 128);
    }
    mbar_init(epi_bar, 128);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kMoeCols);
    tmem_relinquish();
  }
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (kUp) asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int units = *a.n_used * row_tiles;
  const int first = static_cast<int>(blockIdx.x) / splits, stride = static_cast<int>(gridDim.x) / splits;
  const uint8_t* w_scales = kUp ? a.w13_scales : a.w2_scales;

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    bool alive = true;
    for (int u = first; u < units && alive; u += stride) {
      const int ex = u / row_tiles, rt = u - ex * row_tiles;
      const int id = a.list[ex].id;
      // row tile of the stacked weight, and of the up half
      const int tile0 = (kUp ? id * 2 * row_tiles : id * row_tiles) + rt;
      const uint8_t* xs = kUp ? a.x_scales : a.h_scales + static_cast<int64_t>(ex) * kt * 512;
      for (int ks = kbeg; ks < kend; ++ks) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err)) { alive = false; break; }
        uint8_t* sW = smem_gen + stage * kStageBytes;
        uint8_t* sX = sW + kW * kTile;
        uint8_t* sSw = sX + kSlots * 128;
        const uint32_t sbytes = static_cast<uint32_t>(min(kAtoms, kt - ks * kAtoms) * 512);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], kW * kTile + kSlots * 128 + (kW + 1) * sbytes);
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            tma_load_2d(sW + i * kTile, &wmap, ks * 128, (tile0 + i * row_tiles) * 128, &full[stage]);
            bulk_load(sSw + i * (kAtoms * 512), w_scales + (static_cast<int64_t>(tile0 + i * row_tiles) * kt + ks * kAtoms) * 512,
                      sbytes, &full[stage]);
          }
          tma_load_2d(sX, &xmap, ks * 128, kUp ? 0 : ex * kSlots, &full[stage]);
          bulk_load(sSw + kW * (kAtoms * 512), xs + ks * (kAtoms * 512), sbytes, &full[stage]);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    uint32_t stage = 0, phase = 0, uctr = 0;
    bool alive = true;
    const uint64_t desc0 = smem_desc_sw128(smem0, 16, 1024);         // + (byte offset >> 4)
    const uint64_t sdesc0 = smem_desc_scales(smem0);
    for (int u = first; u < units && alive; u += stride, ++uctr) {
      const uint32_t ab = uctr & 1u;
      if (!mbar_wait_warp(&acc_empty[ab], ((uctr >> 1) & 1u) ^ 1u, a.err)) break;
      for (int ks = kbeg; ks < kend; ++ks) {
        if (!mbar_wait_warp(&full[stage], phase, a.err)) { alive = false; break; }
        tc_fence_after();
        const uint32_t off = stage * (kStageBytes >> 4);
        const uint64_t wd = desc0 + off, xd = wd + (kW * kTile >> 4);
        const uint64_t sw = sdesc0 + off + ((kW * kTile + kSlots * 128) >> 4);
        const int atoms = min(kAtoms, kt - ks * kAtoms);
        const uint32_t d = tmem + ab * kAcc;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < kAtoms; ++t)
            if (t < atoms) {
#pragma unroll
              for (int i = 0; i < kW; ++i)
                tmem_cp_scales(tmem + kSfw + 4 * (i * kAtoms + t), sw + (i * kAtoms + t) * 32);
              tmem_cp_scales(tmem + kSfx + 4 * t, sw + (kW * kAtoms + t) * 32);
            }
#pragma unroll
          for (int q = 0; q < 2 * kAtoms; ++q)
            if (q < 2 * atoms) {
#pragma unroll
              for (int i = 0; i < kW; ++i)
                mma_mxf4_ss(d + i * kSlots, wd + i * (kTile >> 4) + q * 2, xd + q * 2,
                            idesc_mxf4(128, kSlots, true, 2u * (q & 1)), tmem + kSfw + 4 * (i * kAtoms + (q >> 1)),
                            tmem + kSfx + 4 * (q >> 1), ks != kbeg || q != 0 ? 1u : 0u);
            }
          mma_commit(&empty[stage]);
          if (ks == kend - 1) mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  }

  const int quarter = warp & 3, rl = quarter * 32 + lane;
  // h of token t at row rl of the tile -> q(h): a block is the warp's 32 rows
  auto emit_h = [&](int ex, int rt, int t, float g, float up) {
    const float h = __fmul_rn(__fdiv_rn(g, __fadd_rn(1.0f, expf(-g))), up);
    const uint32_t mag = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(h) & 0x7FFFFFFFu);
    const bool bad = mag >= 0x7F800000u;
    const uint32_t sb = bad ? 255u : min(mx_e8m0(mag), 253u);
    float v[8] = {bad ? 0.0f : __fmul_rn(h, mx_e8m0_inverse(bad ? 127u : sb)), 0, 0, 0, 0, 0, 0, 0};
    uint32_t word = (mx_codes8(v) & 15u) << (4 * (lane & 7));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    const int64_t row = static_cast<int64_t>(ex) * kSlots + t;
    if ((lane & 7) == 0)
      *reinterpret_cast<uint32_t*>(a.h_codes + row * (a.inner / 2) + rt * 64 + quarter * 16 + (lane >> 3) * 4) = word;
    if (lane == 0)
      a.h_scales[(static_cast<int64_t>(ex) * row_tiles + rt) * 512 + t * 16 + quarter] = static_cast<uint8_t>(sb);
  };

  if (splits == 1 && warp >= 2) {
    const int et = (warp - 2) * 32 + lane;
    uint32_t uctr = 0, ephase = 0;
    auto epi_sync = [&]() -> bool {
      mbar_arrive(epi_bar);
      const bool ok = mbar_wait(epi_bar, ephase, a.err);
      ephase ^= 1u;
      return ok;
    };
    for (int u = first; u < units; u += stride, ++uctr) {
      const int ex = u / row_tiles, rt = u - ex * row_tiles;
      const MoeExpert info = a.list[ex];
      const uint32_t ab = uctr & 1u;
      if (!mbar_wait(&acc_full[ab], (uctr >> 1) & 1u, a.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ab * kAcc;
      uint32_t v0[16], v1[16];
      tmem_ld16(taddr, v0);
      if (kUp) tmem_ld16(taddr + kSlots, v1);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&acc_empty[ab]);
      if (kUp) {
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          if ((info.tokens >> t) & 1u) emit_h(ex, rt, t, __uint_as_float(v0[t]), __uint_as_float(v1[t]));
      } else {
        const int64_t row = static_cast<int64_t>(rt) * 128 + rl;
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          if ((info.tokens >> t) & 1u) {
            const int j = static_cast<int>((info.slots >> (4 * t)) & 15u);
            a.part[(static_cast<int64_t>(t) * a.top_k + j) * a.hidden + row] = __uint_as_float(v0[t]);
          }
        __threadfence();
        if (!epi_sync()) break;
        if (et == 0) *last_flag = atomicAdd(a.counters + rt, 1u) == static_cast<uint32_t>(units / row_tiles - 1) ? 1u : 0u;
        if (!epi_sync()) break;
        if (*last_flag == 0u) continue;
        __threadfence();
        for (int t = 0; t < a.m; ++t) {
          float y = 0.0f;
          for (int j = 0; j < a.top_k; ++j)
            y = __fmaf_rn(a.probs[t * a.top_k + j], __ldcg(a.part + (static_cast<int64_t>(t) * a.top_k + j) * a.hidden + row), y);
          const __nv_bfloat16 b = __float2bfloat16_rn(y);
          a.y[static_cast<int64_t>(t) * a.hidden + row] = *reinterpret_cast<const uint16_t*>(&b);
        }
      }
    }
  }

  if (kUp && splits > 1) {
    // One tile pair per cluster: CTA q owns tokens q * 16 / splits ...; every CTA
    // sends it that part of its tiles, into the stages, summed in rank order.
    const bool work = first < units;
    if (warp >= 2 && work) {
      mbar_wait(&acc_full[0], 0, a.err);
      tc_fence_after();
    }
    __syncwarp();
    cluster_sync();
    const int own = kSlots / splits;
    if (warp >= 2 && work) {
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      uint32_t v[2][16];
      tmem_ld16(taddr, v[0]);
      tmem_ld16(taddr + kSlots, v[kW - 1]);
      tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < kSlots; ++t)
#pragma unroll
        for (int i = 0; i < kW; ++i)
          st_cluster_f32(cluster_map(smem0 + static_cast<uint32_t>(((sp * own + t % own) * kW + i) * 128 + rl) * 4u,
                                     static_cast<uint32_t>(t / own)),
                         __uint_as_float(v[i][t]));
    }
    cluster_sync();
    if (warp >= 2 && work) {
      const int ex = first / row_tiles, rt = first - ex * row_tiles;
      const MoeExpert info = a.list[ex];
      const float* part = reinterpret_cast<const float*>(smem_gen) + rl;
      for (int c = 0; c < own; ++c) {
        const int t = sp * own + c;
        if (!((info.tokens >> t) & 1u)) continue;
        float g = 0.0f, up = 0.0f;
        for (int q = 0; q < splits; ++q) {
          g += part[((q * own + c) * kW) * 128];
          up += part[((q * own + c) * kW + kW - 1) * 128];
        }
        emit_h(ex, rt, t, g, up);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kMoeCols);
  }
}

template <typename K>
cudaError_t smem_limit(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <bool kUp>
cudaError_t launch_product(const MxMoeArgs& a, const CUtensorMap& w, const CUtensorMap& x, int max_used, int num_sms,
                           cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = smem_limit(k_moe_product<kUp>, moe_smem(kUp), done);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(max_used) * ((kUp ? a.inner : a.hidden) / 128);
  const int splits = kUp ? a.splits : 1;
  int64_t grid = units * splits;
  if (splits == 1 && grid > num_sms) grid = num_sms;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = moe_smem(kUp);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_moe_product<kUp>, a, w, x);
}

}  // namespace

int mx_moe_splits(int64_t units, int ksteps, int num_sms) {
  int s = 1;
  while (s < 4 && units * s * 2 <= num_sms && ksteps >= 4 * s) s *= 2;
  return s;
}

cudaError_t launch_mx_moe(const MxMoeArgs& a, const CUtensorMap& w13, const CUtensorMap& x, const CUtensorMap& w2,
                          const CUtensorMap& h, int max_used, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const size_t smem = route_smem(a.experts);
  cudaError_t e = smem_limit(k_moe_route, route_smem(kMoeMaxExperts), done);
  if (e != cudaSuccess) return e;
  k_moe_route<<<kRouteCtas, kRouteThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_product<true>(a, w13, x, max_used, num_sms, stream)) != cudaSuccess) return e;
  return launch_product<false>(a, w2, h, max_used, num_sms, stream);
}

}  // namespace qlora
