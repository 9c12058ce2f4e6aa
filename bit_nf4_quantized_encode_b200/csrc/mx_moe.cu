// mx_moe.cu -- a whole mixture-of-experts feed-forward layer for at most 16
// tokens over MXFP4 experts (sm_100a), in three launches:
//
//   k_moe_route  logits = x R^T (fp32); per token the top_k largest (the lowest
//                index first among equal ones) and p = softmax over them; the
//                list of experts in use with their tokens; q(x).
//   k_moe_up     per expert in use: [g; u] = W13 q(x), h = g / (1 + e^-g) * u, q(h).
//   k_moe_down   y[t] = sum over its experts, in ascending order, of p W2 q(h).
//
// Both products are those of mx_stream.cu: the weight is the 128-row operand of
// tcgen05's block-scaled kind, the 16 token slots the other one, whichever of
// them an expert serves.  An expert in use has its weight read once, whatever
// the number of its tokens, which is what bounds the layer (17/32 byte per
// weight).  A block of q(h) is 32 rows of the product's tile, the 32 lanes of
// one epilogue warp.  32 experts of 4096 x 1536, 4 of them for each of 16 tokens (27
// in use): routing 7 us, up 33, down 20, 4.1 TB/s in all.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_encode.cuh"
#include "mx_format.cuh"
#include "mx_ptx.cuh"
#include "mx_runs.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

// ------------------------------------------------------------------ routing
// One cluster of eight CTAs.  The logits are an [experts, 16] product over hidden:
// a CTA takes an eighth of hidden, its warps groups of 16 experts (several warps a
// group where there are few), with m16n8k16 (bf16 in, fp32 sums).  The parts meet
// in the first CTA, which sums them in a fixed order and chooses: a warp per token
// keeps the token's logits in registers.  Latency is all there is.
constexpr int kRouteCtas = 8;
constexpr int kRouteThreads = 512, kRouteWarps = kRouteThreads / 32;

// Order-preserving key of a logit, above 0 (0 marks a taken one); NaN highest, so that
// it shows in the token's probabilities and y instead of dropping an expert unseen.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));        // -0 is 0
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

// Shared memory: the CTAs' parts of the logits [8][16][experts] (the first CTA's),
// the warps' tiles [16][16][16].
__host__ __device__ constexpr size_t route_smem(int experts) {
  return sizeof(float) * (static_cast<size_t>(kRouteCtas) * 16 * experts + kRouteWarps * 256);
}
constexpr int kKeys = kMoeMaxExperts / 32;          // logits of a lane

__global__ void __launch_bounds__(kRouteThreads) __cluster_dims__(kRouteCtas, 1, 1)
k_moe_route(const MxMoeArgs a) {
  extern __shared__ float smem[];
  __shared__ uint32_t s_mask[kMoeMaxExperts];        // an expert's tokens
  __shared__ unsigned long long s_slot[kMoeMaxExperts];
  __shared__ int s_count[kMoeMaxExperts / 32];
  float* s_in = smem;
  float* s_tile = s_in + kRouteCtas * 16 * a.experts;
  const int warp = warp_index(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_rank());
  asm volatile("griddepcontrol.launch_dependents;");
  for (int i = rank * kRouteThreads + threadIdx.x; i < a.n_counters; i += kRouteCtas * kRouteThreads) a.counters[i] = 0u;
  cluster_arrive();                        // every CTA runs before the others write to it: waited for below

  // q(x): one warp per 1024 elements
  const int segs = static_cast<int>((a.hidden + 1023) / 1024), kt = static_cast<int>(a.hidden / 128);
  for (int u = rank * kRouteWarps + warp; u < a.m * segs; u += kRouteCtas * kRouteWarps) {
    const int tok = u / segs, c = (u - tok * segs) * 1024 + lane * 32;
    const Elems32 e = load32<true>(a.x + static_cast<int64_t>(tok) * a.hidden, c, a.hidden, a.hidden);
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
    if (round == 0) cluster_wait();
    // the experts of these tiles: the warps of a group in order
    const int e0 = round * kRouteWarps / share * 16, here = min(a.experts - e0, kRouteWarps / share * 16);
    for (int i = threadIdx.x; i < here * 16; i += kRouteThreads) {
      const int e = i >> 4, tok = i & 15;
      float v = 0.0f;
      for (int q = 0; q < share; ++q) v += s_tile[((e >> 4) * share + q) * 256 + (i & 255)];
      st_cluster_f32(cluster_map(smem_u32(s_in + (rank * 16 + tok) * a.experts + e0 + e), 0), v);
    }
    __syncthreads();
  }
  cluster_sync();
  if (rank != 0) return;
  for (int e = threadIdx.x; e < kMoeMaxExperts; e += kRouteThreads) {
    s_mask[e] = 0u;
    s_slot[e] = 0ull;
  }
  __syncthreads();

  // top-k: one warp per token, top_k rounds of "largest key, lowest index"
  if (warp < a.m) {
    uint32_t key[kKeys];
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int e = i * 32 + lane;
      key[i] = 0u;
      if (e < a.experts) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kRouteCtas; ++q) v += s_in[(q * 16 + warp) * a.experts + e];
        key[i] = logit_key(v);
      }
    }
    float first = 0.0f, mine = 0.0f;
    int my_id = 0;
    for (int j = 0; j < a.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (key[i] > best) { best = key[i]; at = i; }
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      const uint32_t id = __reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu);
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (static_cast<uint32_t>(i * 32 + lane) == id) key[i] = 0u;
      if (j == 0) first = key_logit(top);
      if (lane == j) {
        mine = expf(key_logit(top) - first);
        my_id = static_cast<int>(id);
      }
    }
    float sum = lane < a.top_k ? mine : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < a.top_k) {
      a.ids[warp * a.top_k + lane] = my_id;
      a.probs[warp * a.top_k + lane] = __fdiv_rn(mine, sum);
      atomicOr(&s_mask[my_id], 1u << warp);
      atomicOr(&s_slot[my_id], static_cast<unsigned long long>(lane) << (4 * warp));
    }
  }
  __syncthreads();
  // the experts in use, in ascending order: id, tokens (bits), and per token its j
  static_assert(kMoeMaxExperts <= kRouteThreads);
  const int e = threadIdx.x;
  const uint32_t mask = e < kMoeMaxExperts ? s_mask[e] : 0u;
  const uint32_t used = __ballot_sync(0xFFFFFFFFu, mask != 0u);
  if (e < kMoeMaxExperts && lane == 0) s_count[warp] = __popc(used);
  __syncthreads();
  if (mask != 0u) {
    int at = __popc(used & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) at += s_count[w];
    MoeExpert x;
    x.id = e;
    x.tokens = mask;
    x.slots = s_slot[e];
    a.list[at] = x;
  }
  if (threadIdx.x == 0) {
    int n = 0;
    for (int w = 0; w < kMoeMaxExperts / 32; ++w) n += s_count[w];
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
__host__ __device__ constexpr int moe_stages(bool up) { return up ? 6 : 10; }
__host__ __device__ constexpr size_t moe_smem(bool up) {
  return 1024 + static_cast<size_t>(moe_stages(up)) * moe_stage(up) + 256;
}
constexpr uint32_t kMoeCols = 128;          // TMEM columns

// h of token t at a lane's row -> q(h): a block is the warp's 32 rows.
__device__ __forceinline__ void emit_h(const MxMoeArgs& a, int ex, int rt, int row_tiles, int t, int quarter, int lane,
                                       float g, float up) {
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
}

// The steps (256 of the contraction) are dealt in equal runs (mx_runs.cuh).
// k_moe_up: a tile is 128 gate rows and the 128 up rows beside them of an expert
// in use.  k_moe_down: a tile is 128 rows of y, its steps run over all experts in
// use; an expert's product leaves the accumulator at its last step (or the run's)
// and is added to the rows' y in registers, times its tokens' p.
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int k = static_cast<int>(kUp ? a.hidden : a.inner);       // contraction
  const int row_tiles = static_cast<int>((kUp ? a.inner : a.hidden) / 128);
  const int kt = k / 128;                                         // scale tiles along k
  const int ksteps = (k + 255) / 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 128);
    }
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
  const int n_used = *a.n_used;
  const int per_tile = kUp ? ksteps : ksteps * n_used;
  const int tiles = kUp ? n_used * row_tiles : row_tiles;
  const int64_t total = static_cast<int64_t>(tiles) * per_tile;
  // The grid is for the most experts that can be in use; no run is empty.  With
  // fewer tiles than CTAs every tile has the same number of runs to itself.
  const int runs = tiles <= static_cast<int>(gridDim.x) ? tiles * max(1, min(static_cast<int>(gridDim.x) / tiles, per_tile / 2))
                                                        : static_cast<int>(gridDim.x);
  const int run = static_cast<int>(blockIdx.x);
  const int64_t begin = run_begin(total, min(run, runs), runs);
  const int nsteps = run < runs ? static_cast<int>(run_begin(total, run + 1, runs) - begin) : 0;
  const int tile0 = static_cast<int>(begin / per_tile), step0 = static_cast<int>(begin - static_cast<int64_t>(tile0) * per_tile);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const uint8_t* w_scales = kUp ? a.w13_scales : a.w2_scales;
    uint32_t stage = 0, phase = 0;
    int ex = kUp ? tile0 / row_tiles : step0 / ksteps;            // place in the list of experts in use
    int rt = kUp ? tile0 - ex * row_tiles : tile0, ks = kUp ? step0 : step0 - ex * ksteps;
    bool fresh = true;
    int wt = 0;                                                   // row tile of the stacked weight
    for (int i = 0; i < nsteps; ++i) {
      if (fresh) wt = a.list[ex].id * (kUp ? 2 * row_tiles : row_tiles) + rt;
      if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err)) break;
      uint8_t* sW = smem_gen + stage * kStageBytes;
      uint8_t* sX = sW + kW * kTile;
      uint8_t* sSw = sX + kSlots * 128;
      const uint32_t sbytes = static_cast<uint32_t>(min(kAtoms, kt - ks * kAtoms) * 512);
      const uint8_t* xs = (kUp ? a.x_scales : a.h_scales + static_cast<int64_t>(ex) * kt * 512) + ks * (kAtoms * 512);
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[stage], kW * kTile + kSlots * 128 + (kW + 1) * sbytes);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          tma_load_2d(sW + w * kTile, &wmap, ks * 128, (wt + w * row_tiles) * 128, &full[stage]);
          bulk_load(sSw + w * (kAtoms * 512), w_scales + (static_cast<int64_t>(wt + w * row_tiles) * kt + ks * kAtoms) * 512,
                    sbytes, &full[stage]);
        }
        tma_load_2d(sX, &xmap, ks * 128, kUp ? 0 : ex * kSlots, &full[stage]);
        bulk_load(sSw + kW * (kAtoms * 512), xs, sbytes, &full[stage]);
      }
      __syncwarp();
      fresh = ++ks == ksteps;
      if (fresh) {                                                // the next expert's rows (down) or row tile (up)
        ks = 0;
        if (kUp) {
          if (++rt == row_tiles) { rt = 0; ++ex; }
        } else if (++ex == n_used) {
          ex = 0;
          ++rt;
        }
      }
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0, seg = 0;
    const uint64_t desc0 = smem_desc_sw128(smem0, 16, 1024);         // + (byte offset >> 4)
    const uint64_t sdesc0 = smem_desc_scales(smem0);
    int ks = kUp ? step0 : step0 % ksteps;
    bool fresh = true;
    for (int i = 0; i < nsteps; ++i) {
      const uint32_t ab = seg & 1u;
      if (fresh && !mbar_wait_warp(&acc_empty[ab], ((seg >> 1) & 1u) ^ 1u, a.err)) break;
      if (!mbar_wait_warp(&full[stage], phase, a.err)) break;
      tc_fence_after();
      const uint32_t off = stage * (kStageBytes >> 4);
      const uint64_t wd = desc0 + off, xd = wd + (kW * kTile >> 4);
      const uint64_t sw = sdesc0 + off + ((kW * kTile + kSlots * 128) >> 4);
      const int atoms = min(kAtoms, kt - ks * kAtoms);
      const uint32_t d = tmem + ab * kAcc;
      const bool last = ks == ksteps - 1 || i == nsteps - 1;
      if (elect_one()) {
#pragma unroll
        for (int t = 0; t < kAtoms; ++t)
          if (t < atoms) {
#pragma unroll
            for (int w = 0; w < kW; ++w)
              tmem_cp_scales(tmem + kSfw + 4 * (w * kAtoms + t), sw + (w * kAtoms + t) * 32);
            tmem_cp_scales(tmem + kSfx + 4 * t, sw + (kW * kAtoms + t) * 32);
          }
#pragma unroll
        for (int q = 0; q < 2 * kAtoms; ++q)
          if (q < 2 * atoms) {
#pragma unroll
            for (int w = 0; w < kW; ++w)
              mma_mxf4_ss(d + w * kSlots, wd + w * (kTile >> 4) + q * 2, xd + q * 2,
                          idesc_mxf4(128, kSlots, true, 2u * (q & 1)), tmem + kSfw + 4 * (w * kAtoms + (q >> 1)),
                          tmem + kSfx + 4 * (q >> 1), !fresh || q != 0 ? 1u : 0u);
          }
        mma_commit(&empty[stage]);
        if (last) mma_commit(&acc_full[ab]);
      }
      __syncwarp();
      fresh = last;
      if (last) ++seg;
      if (++ks == ksteps) ks = 0;
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
  } else {
    // ------------------------------------------------ epilogue
    const int quarter = warp & 3, rl = quarter * 32 + lane;
    const int64_t slot_floats = static_cast<int64_t>(kW) * a.m * 128;
    int tile = tile0, s = step0, left = nsteps;
    float y[kSlots];
#pragma unroll
    for (int t = 0; t < kSlots; ++t) y[t] = 0.0f;
    int from = step0;                                             // first step of this run's part of the tile
    for (uint32_t seg = 0; left > 0; ++seg) {
      const int ex = kUp ? tile / row_tiles : s / ksteps;
      const int ks = kUp ? s : s - ex * ksteps;
      const int steps = min(ksteps - ks, left);
      left -= steps;
      s += steps;
      const MoeExpert info = a.list[ex];
      const uint32_t ab = seg & 1u;
      const bool whole = from == 0 && s == per_tile, ends = kUp || s == per_tile || left == 0;
      // all that does not need the products, before waiting for them
      Parts p{};
      uint32_t* counter = (kUp ? a.up_counters : a.counters) + tile * 4 + quarter;
      bool alone = false;                                         // the other runs' parts are there
      if (ends && !whole) {
        p = parts_of(a.slots + rl, slot_floats, total, static_cast<int64_t>(tile) * per_tile, per_tile, runs);
        alone = others_counted(counter, p.n);
      }
      float pr[kSlots];
      if (!kUp) {
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          pr[t] = (info.tokens >> t) & 1u ? __ldcg(a.probs + t * a.top_k + static_cast<int>((info.slots >> (4 * t)) & 15u)) : 0.0f;
      }
      if (!mbar_wait_warp(&acc_full[ab], (seg >> 1) & 1u, a.err)) break;
      tc_fence_after();
      if (ends && !whole && !alone && left == 0) alone = others_counted(counter, p.n);
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ab * kAcc;
      uint32_t v0[16], v1[16];
      tmem_ld16(taddr, v0);
      if (kUp) tmem_ld16(taddr + kSlots, v1);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(&acc_empty[ab]);
      float* mine = my_slot(a.slots, slot_floats, tile == tile0) + rl;
      const int me = run - p.c0;
      if constexpr (kUp) {
        const int rt = tile - ex * row_tiles;
        auto emit = [&](int t, float g, float up) { emit_h(a, ex, rt, row_tiles, t, quarter, lane, g, up); };
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          if ((info.tokens >> t) & 1u) {
            float gu[2] = {__uint_as_float(v0[t]), __uint_as_float(v1[t])};
            if (alone) add_parts<2>(p, me, 2 * t, 2 * kSlots, gu);
            if (whole || alone) {
              emit(t, gu[0], gu[1]);
            } else {
              mine[(2 * t) * 128] = gu[0];
              mine[(2 * t + 1) * 128] = gu[1];
            }
          }
        if (!whole && !alone && count_part(counter, p.n))
          for (uint32_t left_t = info.tokens; left_t != 0u; left_t &= left_t - 1u) {
            const int t = __ffs(static_cast<int>(left_t)) - 1;
            Parts pt = p;
            pt.first += (2 * t) * 128;
            float gu[2];
            join_parts<2, 8>(pt, 2, [&](int i, float v) { gu[i] = v; });
            emit(t, gu[0], gu[1]);
          }
      } else {
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
          if ((info.tokens >> t) & 1u) y[t] = __fmaf_rn(pr[t], __uint_as_float(v0[t]), y[t]);
        if (!ends) continue;                                      // more experts of this tile
        const int64_t row = static_cast<int64_t>(tile) * 128 + rl;
        auto store = [&](int t, float v) {
          const __nv_bfloat16 b = __float2bfloat16_rn(v);
          a.y[static_cast<int64_t>(t) * a.hidden + row] = *reinterpret_cast<const uint16_t*>(&b);
        };
        if (alone) add_parts<kSlots>(p, me, 0, a.m, y);
#pragma unroll
        for (int t = 0; t < kSlots; ++t) {
          if (t < a.m) {
            if (whole || alone) store(t, y[t]);
            else mine[t * 128] = y[t];
          }
          y[t] = 0.0f;
        }
        if (!whole && !alone && count_part(counter, p.n)) join_columns(p, a.m, store);
      }
      ++tile;
      s = from = 0;
    }
  }

  tc_fence_before();
  __syncwarp();
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
  // runs of two steps at least where every expert that can be in use is
  const int64_t k = kUp ? a.hidden : a.inner, rows = kUp ? a.inner : a.hidden;
  const int64_t steps = static_cast<int64_t>(max_used) * (rows / 128) * ((k + 255) / 256);
  int64_t grid = (steps + 1) / 2;
  if (grid > num_sms) grid = num_sms;
  if (grid > kMxMaxRuns) grid = kMxMaxRuns;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = moe_smem(kUp);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_moe_product<kUp>, a, w, x);
}

}  // namespace

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
