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
#include "mx_format.cuh"
#include "mx_ptx.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

// ------------------------------------------------------------------ routing
// One cluster of CTAs: each takes a part of the experts' logits and of the
// tokens' quantisation; the logits meet in the first CTA's shared memory.
constexpr int kRouteCtas = 8;
constexpr int kRouteThreads = 512;

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = __fmaf_rn(bf16_lo(x[i]), bf16_lo(y[i]), acc);
    acc = __fmaf_rn(bf16_hi(x[i]), bf16_hi(y[i]), acc);
  }
  return acc;
}

// Order-preserving key of a logit, above 0 (0 marks a taken one); NaN lowest.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));        // -0 is 0
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kRouteThreads) __cluster_dims__(kRouteCtas, 1, 1)
k_moe_route(const MxMoeArgs a) {
  extern __shared__ float s_logit[];                             // [m][experts], the first CTA's is used
  __shared__ int s_id[16][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  asm volatile("griddepcontrol.launch_dependents;");
  cluster_sync();                          // the first CTA runs before the others write to it

  // logits: one warp per expert, the router's row once for all tokens
  const int nvec = static_cast<int>(a.hidden / 8);
  for (int e = static_cast<int>(rank) * (kRouteThreads / 32) + warp; e < a.experts; e += kRouteCtas * (kRouteThreads / 32)) {
    const uint4* rr = reinterpret_cast<const uint4*>(a.router + static_cast<int64_t>(e) * a.hidden);
    float acc[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) acc[t] = 0.0f;
    for (int i = lane; i < nvec; i += 32) {
      const uint4 w = __ldg(rr + i);
#pragma unroll
      for (int t = 0; t < 16; ++t)
        if (t < a.m) acc[t] = dot8(w, __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.hidden) + i), acc[t]);
    }
#pragma unroll
    for (int t = 0; t < 16; ++t)
      if (t < a.m) {
        float v = acc[t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (lane == 0) st_cluster_f32(cluster_map(smem_u32(s_logit + t * a.experts + e), 0), v);
      }
  }
  // q(x): one warp per 256 elements
  const int chunks = static_cast<int>((a.hidden + 255) / 256);
  for (int u = static_cast<int>(rank) * (kRouteThreads / 32) + warp; u < a.m * chunks; u += kRouteCtas * (kRouteThreads / 32)) {
    const int t = u / chunks;
    const int64_t c = static_cast<int64_t>(u - t * chunks) * 256 + lane * 8;
    const bool in = c < a.hidden;
    uint4 q = make_uint4(0, 0, 0, 0);
    if (in) q = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * a.hidden + c));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t mag = 0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mag = max(mag, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
    const bool bad = mag >= 0x7F80u;
    const uint32_t sb = bad ? 255u : mx_e8m0(mag << 16);
    const float inv = bad ? 0.0f : mx_e8m0_inverse(sb);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], inv);
    const uint32_t codes = bad ? 0u : mx_codes8(v);
    uint32_t word = sb << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
    if (in) {
      *reinterpret_cast<uint32_t*>(a.x_codes + static_cast<int64_t>(t) * (a.hidden / 2) + (c >> 1)) = codes;
      if ((lane & 15) == 0)
        *reinterpret_cast<uint32_t*>(a.x_scales + mx_scale_offset(t, c / 32, a.hidden / 128)) = word;
    }
  }
  cluster_sync();
  if (rank != 0) return;

  // top-k: one warp per token, top_k rounds of "largest key, lowest index"
  if (warp < a.m) {
    uint32_t* key = reinterpret_cast<uint32_t*>(s_logit + warp * a.experts);
    float first = 0.0f, mine = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      uint32_t best = 0;
      int at = 0;
      for (int e = lane; e < a.experts; e += 32) {
        // a taken logit is remembered by its index, the logits stay as they are
        bool taken = false;
        for (int i = 0; i < j; ++i) taken |= s_id[warp][i] == e;
        const uint32_t k = taken ? 0u : logit_key(__uint_as_float(key[e]));
        if (k > best) { best = k; at = e; }
      }
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
      const int id = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
      const float v = __uint_as_float(key[id]);
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
  __syncthreads();
  // the experts in use, in ascending order: id, tokens (bits), and per token its j
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      uint32_t mask = 0;
      uint64_t slot = 0;                                         // four bits per token
      if (e < a.experts)
        for (int t = 0; t < a.m; ++t)
          for (int j = 0; j < a.top_k; ++j)
            if (s_id[t][j] == e) {
              mask |= 1u << t;
              slot |= static_cast<uint64_t>(j) << (4 * t);
            }
      const uint32_t used = __ballot_sync(0xFFFFFFFFu, mask != 0);
      if (mask != 0) {
        MoeExpert x;
        x.id = e;
        x.tokens = mask;
        x.slots = slot;
        a.list[n + __popc(used & ((1u << lane) - 1u))] = x;
      }
      n += __popc(used);
    }
    if (lane == 0) *a.n_used = n;
  }
  for (int i = threadIdx.x; i < static_cast<int>(a.hidden / 128); i += kRouteThreads) a.counters[i] = 0u;
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
__host__ __device__ constexpr int moe_stages(bool up) { return up ? 5 : 5; }
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
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
    if (lane == 0) {
      uint32_t it = 0;
      bool alive = true;
      for (int u = first; u < units && alive; u += stride) {
        const int ex = u / row_tiles, rt = u - ex * row_tiles;
        const int64_t id = a.list[ex].id;
        // first row of the tile in the stacked weight, and of the up half
        const int64_t row0 = (kUp ? id * 2 * a.inner : id * a.hidden) + static_cast<int64_t>(rt) * 128;
        const uint8_t* xs = kUp ? a.x_scales : a.h_scales + static_cast<int64_t>(ex) * kt * 512;
        for (int ks = kbeg; ks < kend; ++ks, ++it) {
          const uint32_t stage = it % kStages, phase = (it / kStages) & 1u;
          if (!mbar_wait(&empty[stage], phase ^ 1u, a.err)) { alive = false; break; }
          uint8_t* sW = smem_gen + stage * kStageBytes;
          uint8_t* sX = sW + kW * kTile;
          uint8_t* sSw = sX + kSlots * 128;
          const int atoms = min(kAtoms, kt - ks * kAtoms);
          const uint32_t sbytes = static_cast<uint32_t>(atoms * 512);
          mbar_arrive_expect_tx(&full[stage], kW * kTile + kSlots * 128 + (kW + 1) * sbytes);
#pragma unroll
          for (int i = 0; i < kW; ++i) {
            const int64_t r = row0 + i * a.inner;
            tma_load_2d(sW + i * kTile, &wmap, ks * 128, static_cast<int32_t>(r), &full[stage]);
            bulk_load(sSw + i * (kAtoms * 512), w_scales + (r / 128 * kt + ks * kAtoms) * 512, sbytes, &full[stage]);
          }
          tma_load_2d(sX, &xmap, ks * 128, kUp ? 0 : ex * kSlots, &full[stage]);
          bulk_load(sSw + kW * (kAtoms * 512), xs + ks * (kAtoms * 512), sbytes, &full[stage]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, uctr = 0;
      bool alive = true;
      for (int u = first; u < units && alive; u += stride, ++uctr) {
        const uint32_t ab = uctr & 1u;
        if (!mbar_wait(&acc_empty[ab], ((uctr >> 1) & 1u) ^ 1u, a.err)) break;
        tc_fence_after();
        for (int ks = kbeg; ks < kend; ++ks, ++it) {
          const uint32_t stage = it % kStages, phase = (it / kStages) & 1u;
          if (!mbar_wait(&full[stage], phase, a.err)) { alive = false; break; }
          tc_fence_after();
          const uint32_t sW = smem0 + stage * kStageBytes, sX = sW + kW * kTile, sSw = sX + kSlots * 128;
          const int atoms = min(kAtoms, kt - ks * kAtoms);
          for (int t = 0; t < atoms; ++t) {
#pragma unroll
            for (int i = 0; i < kW; ++i)
              tmem_cp_scales(tmem + kSfw + 4 * (i * kAtoms + t), smem_desc_scales(sSw + (i * kAtoms + t) * 512));
            tmem_cp_scales(tmem + kSfx + 4 * t, smem_desc_scales(sSw + (kW * kAtoms + t) * 512));
          }
          for (int q = 0; q < 2 * atoms; ++q) {
            const uint64_t xd = smem_desc_sw128(sX + q * 32, 16, 1024);
#pragma unroll
            for (int i = 0; i < kW; ++i)
              mma_mxf4_ss(tmem + ab * kAcc + i * kSlots, smem_desc_sw128(sW + i * kTile + q * 32, 16, 1024), xd,
                          idesc_mxf4(128, kSlots, true, 2u * (q & 1)), tmem + kSfw + 4 * (i * kAtoms + (q >> 1)),
                          tmem + kSfx + 4 * (q >> 1), ks != kbeg || q != 0 ? 1u : 0u);
          }
          mma_commit(&empty[stage]);
        }
        if (alive) mma_commit(&acc_full[ab]);
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
  const size_t smem = static_cast<size_t>(a.m) * a.experts * sizeof(float);
  cudaError_t e = smem_limit(k_moe_route, 16 * kMoeMaxExperts * sizeof(float), done);
  if (e != cudaSuccess) return e;
  k_moe_route<<<kRouteCtas, kRouteThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_product<true>(a, w13, x, max_used, num_sms, stream)) != cudaSuccess) return e;
  return launch_product<false>(a, w2, h, max_used, num_sms, stream);
}

}  // namespace qlora
