// lora.cu -- the rank-r contractions of the LoRA branch on tcgen05 / TMEM / TMA.
//
// What is computed (QLoRA, arXiv:2305.14314; automatone "QLoRA paper
// explained", section "How it works": the 16-bit LoRA adapters sit beside the
// frozen 4-bit weight, and the gradients land only on them):
//   forward   XA = X A^T                          [M, r]  (contraction over K)
//   backward  G  = dY B                           [M, r]  (contraction over N)
//             dB = dY^T (s XA)                    [N, r]  (contraction over the tokens)
//             dA = ((s G)^T X) = (X^T (s G))^T    [r, K]  (contraction over the tokens)
// Each is D[mdim, ndim] = P Q^T with the long operand P streamed once by TMA
// and the rank-r operand Q (small, L2-resident) beside it; ndim = r <= 256.
//
// One launch runs up to two such problems (XA with G; dB with dA), each cut
// into (128-row tile, 64-column tile, K split) units spread over a persistent
// grid.  A problem whose tiles alone would not fill the GPU splits its
// contraction; the partial tiles then go to slots in global memory and the
// unit that completes a tile's count (an atomic counter) sums the slots in
// split order, so every result is bit-reproducible from run to run -- no fp32
// atomics anywhere.  The epilogue writes any of: the fp32 result (optionally
// transposed, for dA), and bf16(scale * result) zero-padded to a multiple of
// 64 columns (the rank-r operand of the fused dequant-GEMM and of the next
// contraction), or that value as two bf16 parts, so no separate convert kernel
// runs.  A side job converts a caller-supplied fp32 X A^T the same way.  A rank-r
// operand in two parts (the layer over a microscaled weight) has both beside the
// one tile of the long operand: G, dA and dB of 8192 tokens, 8192 x 8192, rank 64, in
// 98 us; from rounded operands, which put the gradients 1e-3 off, in 87.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "bf16_parts.cuh"
#include "lora.h"
#include "mx_ptx.cuh"
#include "nf4_device.cuh"

namespace qlora {
namespace {

constexpr int kStages = 6;
constexpr int kABytes = 128 * 128;     // 128 x 64 bf16
constexpr int kBBytes = 64 * 128;      // 64 x 64 bf16
// Q in two parts: both tiles beside the one of P, multiplied one after the other,
// so the long operand is still read once.
__host__ __device__ constexpr int stage_bytes(bool parts) { return kABytes + (parts ? 2 : 1) * kBBytes; }
constexpr int kThreads = 6 * 32;       // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr uint32_t kTmemCols = 128;    // two 64-column accumulators
constexpr size_t rank_smem(bool parts) { return 1024 + kStages * stage_bytes(parts) + 256; }

struct UnitPos {
  int prob, mt, nt, sp, kbeg, nk;
};

__device__ __forceinline__ UnitPos unit_pos(const RankArgs& a, int u) {
  UnitPos w;
  w.prob = (a.nprob > 1 && u >= a.p[1].unit_begin) ? 1 : 0;
  const RankProblem& p = a.p[w.prob];
  const int local = u - p.unit_begin;
  w.sp = local % p.splits;
  const int rest = local / p.splits;
  w.nt = rest % p.n_tiles;
  w.mt = rest / p.n_tiles;
  w.kbeg = static_cast<int>((static_cast<int64_t>(p.ksteps) * w.sp) / p.splits);
  w.nk = static_cast<int>((static_cast<int64_t>(p.ksteps) * (w.sp + 1)) / p.splits) - w.kbeg;
  return w;
}


__device__ __forceinline__ float4 ld_cg4(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// First and second parts of two values, packed.
__device__ __forceinline__ void bf16_parts2(float a, float b, uint32_t& first, uint32_t& second) {
  const BfParts x = bf16_parts(a), y = bf16_parts(b);
  first = pack_bf16x2(x.first, y.first);
  second = pack_bf16x2(x.second, y.second);
}

// bf16(s * v) of row `row`, columns c0 .. c0 + 63 below bf16_cols; columns past
// ndim hold zeros (zero-filled operand).
__device__ __forceinline__ void store_bf16_row(const RankProblem& p, int64_t row, int64_t c0, const float (&v)[64]) {
  uint16_t* dst = p.out_bf16 + row * p.ld_bf16 + c0;
  const float s = p.bf16_scale;
#pragma unroll
  for (int c = 0; c < 64; c += 8)
    if (c0 + c < p.bf16_cols) {
      uint4 q;
      q.x = pack_bf16x2(__fmul_rn(s, v[c]), __fmul_rn(s, v[c + 1]));
      q.y = pack_bf16x2(__fmul_rn(s, v[c + 2]), __fmul_rn(s, v[c + 3]));
      q.z = pack_bf16x2(__fmul_rn(s, v[c + 4]), __fmul_rn(s, v[c + 5]));
      q.w = pack_bf16x2(__fmul_rn(s, v[c + 6]), __fmul_rn(s, v[c + 7]));
      *reinterpret_cast<uint4*>(dst + c) = q;
    }
}

// v as two bf16 parts (lora.h), 64 columns.  The end of a kernel of a few
// microseconds runs this code once, and fetching it takes longer than running it, so
// it works on pairs and has no other path for what is not finite: there the second
// part (inf - inf or finite - inf) is bounded by 2^120, which no other reaches (2^119)
// and which leaves the first one's Inf or NaN as it is.
__device__ __forceinline__ void store_parts_row(uint16_t* dst, const float (&v)[64]) {
#pragma unroll
  for (int c = 0; c < 64; c += 8) {
    uint32_t first[4], second[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v[c + 2 * i], b = v[c + 2 * i + 1];
      first[i] = pack_bf16x2(a, b);
      second[i] = pack_bf16x2(__fsub_rn(a, bf16_lo(first[i])), __fsub_rn(b, bf16_hi(first[i])));
      asm("min.bf16x2 %0, %0, %1;" : "+r"(second[i]) : "r"(0x7B807B80u));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(second[i]) : "r"(0xFB80FB80u));
    }
    *reinterpret_cast<uint4*>(dst + c) = make_uint4(first[0], first[1], first[2], first[3]);
    *reinterpret_cast<uint4*>(dst + 64 + c) = make_uint4(second[0], second[1], second[2], second[3]);
  }
}

// The final values of row `row`, columns c0 .. c0 + 63 of problem p's D.
__device__ __forceinline__ void store_final(const RankProblem& p, int64_t row, int64_t c0, const float (&v)[64]) {
  if (row >= p.mdim) return;
  if (p.out_f32) {
    if (p.transpose) {                      // out[j * ld + row]: lanes walk rows, coalesced per column
#pragma unroll
      for (int c = 0; c < 64; ++c)
        if (c0 + c < p.ndim) p.out_f32[(c0 + c) * p.ld_f32 + row] = v[c];
    } else {
      float* dst = p.out_f32 + row * p.ld_f32 + c0;
#pragma unroll
      for (int c = 0; c < 64; c += 4)       // ndim and ld are multiples of 8: whole 16-byte pieces
        if (c0 + c < p.ndim) *reinterpret_cast<float4*>(dst + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
    }
  }
  if (p.out_bf16) store_bf16_row(p, row, c0, v);
  if ((p.out_parts || p.out_div) && c0 < p.bf16_cols) {
    float d[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) d[c] = __fmul_rn(p.bf16_scale, v[c]);
    const int64_t at = row * (2 * p.bf16_cols) + 2 * c0;
    if (p.out_parts) store_parts_row(p.out_parts + at, d);
    if (p.out_div) {
      // one divisor after the other: their product may be below what a float holds
      // (row_div: powers of two), and all_div's reciprocal taken where it is a normal
      // float: 64 divisions of a thread took longer than the contraction of few tokens
      const float by_row = 1.0f / p.row_div[row], all = p.all_div[0];
      const float shift = all < 0x1p-126f ? 0x1p64f : all > 0x1p126f ? 0x1p-64f : 1.0f;
      const float by_all = 1.0f / __fmul_rn(all, shift);
#pragma unroll
      for (int c = 0; c < 64; ++c) d[c] = __fmul_rn(__fmul_rn(__fmul_rn(d[c], by_row), by_all), shift);
      store_parts_row(p.out_div + at, d);
    }
  }
}

template <bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
k_rank(const RankArgs a, const __grid_constant__ CUtensorMap am0, const __grid_constant__ CUtensorMap bm0,
       const __grid_constant__ CUtensorMap am1, const __grid_constant__ CUtensorMap bm1) {
  constexpr int kStageBytes = stage_bytes(kParts);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_gen + kStages * kStageBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* acc_full = bars + 2 * kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* epi_bar = acc_empty + 2;         // the 128 epilogue threads meet here (bounded waits)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
  uint32_t* last_flag = tmem_slot + 1;

  const int warp = warp_index();             // TMA and MMA are issued by an elected lane of a uniform warp
  const int lane = threadIdx.x & 31;
  const int nunits = a.total_units;

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
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&am0);
    tma_prefetch_desc(&bm0);
    if (a.nprob > 1) {
      tma_prefetch_desc(&am1);
      tma_prefetch_desc(&bm1);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    uint32_t stage = 0, phase = 0;
    bool alive = true;
    for (int u = blockIdx.x; u < nunits && alive; u += gridDim.x) {
      const UnitPos w = unit_pos(a, u);
      const RankProblem& p = a.p[w.prob];
      const CUtensorMap* am = w.prob ? &am1 : &am0;
      const CUtensorMap* bm = w.prob ? &bm1 : &bm0;
      const bool a_mn = p.a_mn != 0, b_mn = kParts || p.b_mn != 0;
      auto load = [&](uint32_t st, int k0) {
        uint8_t* sA = smem_gen + st * kStageBytes;
        uint8_t* sB = sA + kABytes;
        mbar_arrive_expect_tx(&full[st], kStageBytes);
        if (a_mn) {   // A^T stored [k][m]: two 64-wide MN boxes
          tma_load_2d(sA, am, w.mt * 128, k0, &full[st]);
          tma_load_2d(sA + 8192, am, w.mt * 128 + 64, k0, &full[st]);
        } else {
          tma_load_2d(sA, am, k0, w.mt * 128, &full[st]);
        }
        if constexpr (kParts) {
          tma_load_2d(sB, bm, w.nt * 128, k0, &full[st]);
          tma_load_2d(sB + kBBytes, bm, w.nt * 128 + 64, k0, &full[st]);
        } else if (b_mn) {
          tma_load_2d(sB, bm, w.nt * 64, k0, &full[st]);
        } else {
          tma_load_2d(sB, bm, k0, w.nt * 64, &full[st]);
        }
      };
      // two consecutive k-steps at a time: both stages are claimed first and
      // their loads issued back to back, so every row of the long operand is
      // requested in 256-byte runs rather than 128-byte ones
      for (int j = 0; j < w.nk; j += 2) {
        const bool two = j + 1 < w.nk;
        const uint32_t stage2 = stage + 1 == kStages ? 0 : stage + 1, phase2 = stage2 == 0 ? phase ^ 1u : phase;
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err) ||
            (two && !mbar_wait_warp(&empty[stage2], phase2 ^ 1u, a.err))) {
          alive = false;
          break;
        }
        if (elect_one()) {
          load(stage, (w.kbeg + j) * 64);
          if (two) load(stage2, (w.kbeg + j + 1) * 64);
        }
        __syncwarp();
        stage = two ? stage2 : stage;
        phase = two ? phase2 : phase;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0, uctr = 0;
    bool alive = true;
    // uctr counts accumulator fillings: one per unit, or one per `flush` k-steps
    for (int u = blockIdx.x; u < nunits && alive; u += gridDim.x) {
      const UnitPos w = unit_pos(a, u);
      const RankProblem& p = a.p[w.prob];
      const bool a_mn = p.a_mn != 0, b_mn = kParts || p.b_mn != 0;
      const uint32_t idesc = idesc_bf16(128, 64, a_mn, b_mn);
      const int piece = p.flush > 0 ? p.flush : w.nk;
      // a K = 16 slice: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
      const uint64_t a0 = a_mn ? smem_desc_sw128(smem0, 8192, 1024) : smem_desc_sw128(smem0, 16, 1024);
      const uint64_t b0 = (b_mn ? smem_desc_sw128(smem0, 8192, 1024) : smem_desc_sw128(smem0, 16, 1024)) + (kABytes >> 4);
      const uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
      int left = 0;                            // k-steps to go of this filling
      for (int j = 0; j < w.nk; ++j) {
        const uint32_t ab = uctr & 1u, aphase = (uctr >> 1) & 1u;
        const bool fresh = left == 0;
        if (fresh) {
          left = w.nk - j < piece ? w.nk - j : piece;
          if (!mbar_wait_warp(&acc_empty[ab], aphase ^ 1u, a.err)) { alive = false; break; }
        }
        if (!mbar_wait_warp(&full[stage], phase, a.err)) { alive = false; break; }
        tc_fence_after();
        const uint32_t off = stage * (kStageBytes >> 4);
        const bool last = --left == 0;
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < (kParts ? 2 : 1); ++q)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ss(tmem_base + ab * 64, a0 + off + kk * a_step, b0 + off + q * (kBBytes >> 4) + kk * b_step, idesc,
                          !fresh || q + kk != 0 ? 1u : 0u);
          mma_commit(&empty[stage]);
          if (last) mma_commit(&acc_full[ab]);
        }
        __syncwarp();
        if (last) ++uctr;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------ epilogue (warps 2..5)
    const int quarter = warp & 3;            // warps 2,3,4,5 -> TMEM lane quarters 2,3,0,1
    const int et = (warp - 2) * 32 + lane;   // 0 .. 127
    uint32_t uctr = 0, ephase = 0;
    // all 128 epilogue threads arrive, then wait for the phase (bounded)
    auto epi_sync = [&]() -> bool {
      mbar_arrive(epi_bar);
      const bool ok = mbar_wait(epi_bar, ephase, a.err);
      ephase ^= 1u;
      return ok;
    };
    bool alive = true;
    for (int u = blockIdx.x; u < nunits; u += gridDim.x) {
      const UnitPos w = unit_pos(a, u);
      const RankProblem& p = a.p[w.prob];
      const int rl = quarter * 32 + lane;                   // row inside the tile
      const int64_t row = static_cast<int64_t>(w.mt) * 128 + rl;
      const int fills = p.flush > 0 ? (w.nk + p.flush - 1) / p.flush : 1;
      float v[64];
      for (int f = 0; f < fills; ++f, ++uctr) {
        const uint32_t ab = uctr & 1u, aphase = (uctr >> 1) & 1u;
        if (!mbar_wait(&acc_full[ab], aphase, a.err)) { alive = false; break; }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + ab * 64;
        uint32_t r0[32], r1[32];
        tmem_ld32(taddr, r0);
        tmem_ld32(taddr + 32, r1);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&acc_empty[ab]);                         // TMEM free for the next filling
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          v[c] = f == 0 ? __uint_as_float(r0[c]) : v[c] + __uint_as_float(r0[c]);
          v[32 + c] = f == 0 ? __uint_as_float(r1[c]) : v[32 + c] + __uint_as_float(r1[c]);
        }
      }
      if (!alive) break;
      const int64_t c0 = static_cast<int64_t>(w.nt) * 64;
      if (p.splits == 1) {
        store_final(p, row, c0, v);
        continue;
      }
      // split contraction: partial to this split's slot ([64 cols][128 rows],
      // coalesced per column), then count; the unit completing the count sums
      // all slots of the tile in split order
      const int tile = w.mt * p.n_tiles + w.nt;
      float* slot_tile = p.slots + static_cast<int64_t>(tile) * p.splits * (64 * 128);
      float* mine = slot_tile + static_cast<int64_t>(w.sp) * (64 * 128);
#pragma unroll
      for (int c = 0; c < 64; ++c) mine[c * 128 + rl] = v[c];
      __threadfence();
      if (!epi_sync()) break;
      if (et == 0) *last_flag = (atomicAdd(p.counters + tile, 1u) == static_cast<uint32_t>(p.splits - 1)) ? 1u : 0u;
      if (!epi_sync()) break;
      const bool last = *last_flag != 0u;
      if (!last) continue;
      __threadfence();
      float sum[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) sum[c] = 0.0f;
      for (int s = 0; s < p.splits; ++s) {
        if (s == w.sp) {
#pragma unroll
          for (int c = 0; c < 64; ++c) sum[c] += v[c];
        } else {
          const float* src = slot_tile + static_cast<int64_t>(s) * (64 * 128) + rl;
#pragma unroll
          for (int c = 0; c < 64; ++c) sum[c] += __ldcg(src + c * 128);
        }
      }
      store_final(p, row, c0, sum);
    }
    // side job: bf16(scale * in) of a caller's fp32 matrix, zero-padded (or its
    // two parts), one row per epilogue thread over the whole grid
    if (a.cvt_in) {
      const int64_t gt = static_cast<int64_t>(blockIdx.x) * 128 + et;
      for (int64_t i = gt; i < a.cvt_rows; i += static_cast<int64_t>(gridDim.x) * 128) {
        const float* src = a.cvt_in + i * a.cvt_ld_in;
        uint16_t* dst = a.cvt_out + i * a.cvt_ld_out;
        for (int64_t c = 0; c < a.cvt_cols_out; c += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = (c + e < a.cvt_cols) ? __fmul_rn(a.cvt_scale, src[c + e]) : 0.0f;
          uint32_t first[4], second[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) bf16_parts2(f[2 * e], f[2 * e + 1], first[e], second[e]);
          uint16_t* at = dst + (a.cvt_parts ? (c & ~int64_t{63}) * 2 + (c & 63) : c);
          *reinterpret_cast<uint4*>(at) = make_uint4(first[0], first[1], first[2], first[3]);
          if (a.cvt_parts) *reinterpret_cast<uint4*>(at + 64) = make_uint4(second[0], second[1], second[2], second[3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool kParts>
cudaError_t launch_t(const RankArgs& args, const CUtensorMap& am0, const CUtensorMap& bm0, const CUtensorMap& am1,
                     const CUtensorMap& bm1, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_rank<kParts>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(rank_smem(kParts)));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int grid = args.total_units < num_sms ? args.total_units : num_sms;
  k_rank<kParts><<<grid, kThreads, rank_smem(kParts), stream>>>(args, am0, bm0, am1, bm1);
  return cudaGetLastError();
}

}  // namespace

int rank_splits(int tiles, int ksteps, int num_sms, int max_splits) {
  // makespan model: waves of units over the SMs times the k-steps of a unit
  // plus two k-steps of fixed cost (epilogue, split fix-up)
  // each split adds a 32 KB partial tile written and read back: beyond the
  // splits a tile needs to spread over the SMs (about two units per SM), at
  // most 4
  int spread = tiles > 0 ? (2 * num_sms + tiles - 1) / tiles : 1;
  if (spread < 4) spread = 4;
  if (max_splits > spread) max_splits = spread;
  int best = 1;
  int64_t best_cost = -1;
  const int cap = ksteps / 4 > 1 ? ksteps / 4 : 1;          // at least 4 k-steps per split
  for (int s = 1; s <= max_splits && s <= cap; ++s) {
    const int64_t waves = (static_cast<int64_t>(tiles) * s + num_sms - 1) / num_sms;
    const int64_t cost = waves * ((ksteps + s - 1) / s + 2);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

size_t rank_slot_bytes(int tiles, int splits) {
  return splits > 1 ? static_cast<size_t>(tiles) * splits * 64 * 128 * sizeof(float) : 0;
}

cudaError_t launch_rank(const RankArgs& args, const CUtensorMap& am0, const CUtensorMap& bm0,
                        const CUtensorMap& am1, const CUtensorMap& bm1, int num_sms, cudaStream_t stream) {
  return args.b_parts ? launch_t<true>(args, am0, bm0, am1, bm1, num_sms, stream)
                      : launch_t<false>(args, am0, bm0, am1, bm1, num_sms, stream);
}

}  // namespace qlora
