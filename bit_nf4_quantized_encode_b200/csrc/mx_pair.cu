// mx_pair.cu -- the product of two microscaled 4-bit operands for many tokens:
// pairs of CTAs (cta_group::2) on one tile of 256 weight rows x 256 (or 128)
// tokens (sm_100a).  The formula and the operands are those of mx_stream.cu.
//
// Why pairs: one CTA's 128 x 256 tile reads 12 KB of shared memory per 64 of the
// contraction and TMA writes as much, which is what bounds it; a pair holds each
// half of the tokens once, 8 KB a CTA for twice the tile.
//
// 8192 x 8192 by 8192 tokens, MXFP4: 192 us, 5.7 PFLOP/s, with the SM clock at 1.6
// GHz under the power limit (the tensor pipe active 66% of the time; loads alone
// 155 us).  One CTA with tiles of 128 x 128 took 548 us.  NVFP4's epilogue has its
// token scales in shared memory, fetched while the products run: 243 us with the
// quantiser, 256 with a read-only load of them per element.
//
// TMEM (512 columns): two accumulators of 256 columns that share 48 columns,
// and the scales of one stage.  The epilogue drains the shared columns first;
// the next tile's products start then, while the other 208 drain.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_format.cuh"
#include "mx_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 6 * 32;            // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kABytes = 128 * 128;          // a CTA's 128 rows x 256 codes
constexpr uint32_t kAcc1 = 208;             // first column of the second accumulator (256 columns)
constexpr uint32_t kSfCols = 464;           // first column of the scales (48 columns)

__host__ __device__ constexpr int atoms_of(int fmt) { return fmt == kMxFp4 ? 2 : 4; }
__host__ __device__ constexpr int pair_stage(int fmt, int bn) {
  return kABytes + bn / 2 * 128 + atoms_of(fmt) * 512 * (1 + bn / 128);
}
__host__ __device__ constexpr int pair_stages(int fmt, int bn) {
  return bn == 256 ? (fmt == kMxFp4 ? 6 : 5) : (fmt == kMxFp4 ? 8 : 7);
}
__host__ __device__ constexpr size_t pair_smem(int fmt, int bn) {
  return 1024 + static_cast<size_t>(pair_stages(fmt, bn)) * pair_stage(fmt, bn) + 256;
}

struct Tile {
  int mt, tt;
};
__device__ __forceinline__ Tile tile_of(int u, const MxGemmArgs& a) {
  const int per_group = a.m_group * a.t_tiles;
  const int gi = u / per_group;
  const int r = u - gi * per_group;
  const int gsz = min(a.m_group, a.m_tiles - gi * a.m_group);
  return {gi * a.m_group + r % gsz, r / gsz};
}

template <int kFmt, int kBN>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
k_mx_pair(const MxGemmArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
          const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap,
          const __grid_constant__ CUtensorMap lwmap, const __grid_constant__ CUtensorMap lxmap) {
  constexpr int kStages = pair_stages(kFmt, kBN);
  constexpr int kStageBytes = pair_stage(kFmt, kBN);
  constexpr int kAtoms = atoms_of(kFmt);
  constexpr int kRB = kBN / 128;             // row tiles of the tokens' scales
  constexpr int kBBytes = kBN / 2 * 128;     // a CTA's half of the tokens
  constexpr uint32_t kSfa = kSfCols, kSfb = kSfCols + 4 * kAtoms;
  constexpr int kChunks = kBN / 16, kShared = 3;      // 16-column pieces of an accumulator, of them shared (kBN = 256)

  extern __shared__ uint8_t smem_raw[];
  __shared__ float4 s_gx[4][kFmt == kNvFp4 ? kBN / 4 : 1];     // an epilogue warp's token scales
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_gen + kStages * kStageBytes);   // the leader's count both CTAs' bytes
  uint64_t* empty = full + kStages;          // commit, in both CTAs
  uint64_t* acc_full = empty + kStages;      // commit, in both CTAs
  uint64_t* acc_free = acc_full + 1;         // the leader's: one arrival per epilogue warp of the pair
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_free + 1);

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int ntiles = a.m_tiles * a.t_tiles;
  const int first = static_cast<int>(blockIdx.x) >> 1, stride = static_cast<int>(gridDim.x) >> 1;
  const int nk = a.ksteps + 2 * a.lora_steps;      // each 64 ranks twice: the activations' two bf16 parts

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 8);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&wsmap);
    tma_prefetch_desc(&xsmap);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                            // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer, one per CTA
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t full0 = cluster_map(smem_u32(full), 0);
    uint32_t stage = 0, phase = 0;
    bool alive = true;
    for (int u = first; u < ntiles && alive; u += stride) {
      const Tile w = tile_of(u, a);
      const int row0 = w.mt * 256 + static_cast<int>(rank) * 128;
      const int tok0 = w.tt * kBN + static_cast<int>(rank) * (kBN / 2);
      const int ws0 = static_cast<int>(row0 / 128 * a.kt), xs0 = static_cast<int>(w.tt * kRB * a.kt);
      for (int j = 0; j < nk; ++j) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err)) { alive = false; break; }
        const uint32_t bar = full0 + stage * 8u;
        uint8_t* sA = smem_gen + stage * kStageBytes;
        uint8_t* sB = sA + kABytes;
        if (elect_one()) {
          if (j < a.ksteps) {
            uint8_t* sSa = sB + kBBytes;
            uint8_t* sSb = sSa + kAtoms * 512;
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
            tma_load_2d_pair(sA, &wmap, j * 128, row0, bar);
            tma_load_2d_pair(sB, &xmap, j * 128, tok0, bar);
            // a row tile's scales past its last one are the next row tile's: loaded, not used
            tma_load_2d_pair(sSa, &wsmap, 0, ws0 + j * kAtoms, bar);
#pragma unroll
            for (int b = 0; b < kRB; ++b)
              tma_load_2d_pair(sSb + b * (kAtoms * 512), &xsmap, 0, xs0 + b * static_cast<int>(a.kt) + j * kAtoms, bar);
          } else {
            const int part = j - a.ksteps, r0 = (part >> 1) * 64;
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (kABytes + kBBytes));
            if (a.lora_mn) {
              tma_load_2d_pair(sA, &lwmap, row0, r0, bar);
              tma_load_2d_pair(sA + 8192, &lwmap, row0 + 64, r0, bar);
            } else {
              tma_load_2d_pair(sA, &lwmap, r0, row0, bar);
            }
            tma_load_2d_pair(sB, &lxmap, part * 64, tok0, bar);
          }
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer, the leader's
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, n = 0;
      bool alive = true;
      const uint32_t lora_idesc = idesc_bf16(256, kBN, a.lora_mn != 0, false);
      const uint64_t desc0 = smem_desc_sw128(smem0, 16, 1024);       // + (byte offset >> 4)
      const uint64_t sdesc0 = smem_desc_scales(smem0);
      for (int u = first; u < ntiles && alive; u += stride, ++n) {
        if (n > 0 && !mbar_wait_warp(acc_free, (n - 1) & 1u, a.err)) break;
        tc_fence_after();
        const uint32_t d = tmem + (n & 1u) * kAcc1;
        for (int j = 0; j < nk; ++j) {
          if (!mbar_wait_warp(&full[stage], phase, a.err)) { alive = false; break; }
          tc_fence_after();
          const uint32_t off = stage * (kStageBytes >> 4);
          const uint64_t ad = desc0 + off, bd = ad + (kABytes >> 4);
          if (elect_one()) {
            if (j < a.ksteps) {
              const uint64_t sa = sdesc0 + off + ((kABytes + kBBytes) >> 4), sb = sa + (kAtoms * 512 >> 4);
#pragma unroll
              for (int t = 0; t < kAtoms; ++t) {
                tmem_cp_scales_pair(tmem + kSfa + 4 * t, sa + t * 32);
#pragma unroll
                for (int b = 0; b < kRB; ++b)
                  tmem_cp_scales_pair(tmem + kSfb + 4 * (t * kRB + b), sb + (b * kAtoms + t) * 32);
              }
              const int slices = static_cast<int>(min(static_cast<int64_t>(4), (a.k - static_cast<int64_t>(j) * 256 + 63) / 64));
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (q < slices) {
                  const uint32_t acc = (j | q) != 0 ? 1u : 0u;
                  if (kFmt == kMxFp4)
                    mma_fp4_pair<true>(d, ad + q * 2, bd + q * 2, idesc_mxf4(256, kBN, true, 2u * (q & 1)),
                                       tmem + kSfa + 4 * (q >> 1), tmem + kSfb + 4 * kRB * (q >> 1), acc);
                  else
                    mma_fp4_pair<false>(d, ad + q * 2, bd + q * 2, idesc_mxf4(256, kBN, false, 0), tmem + kSfa + 4 * q,
                                        tmem + kSfb + 4 * kRB * q, acc);
                }
              }
            } else {
              // A K = 16 slice: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
              const uint64_t la = a.lora_mn ? smem_desc_sw128(smem0, 8192, 1024) + off : ad;
              const uint32_t step = a.lora_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
              for (int q = 0; q < 4; ++q) mma_bf16_pair(d, la + q * step, bd + q * 2, lora_idesc, 1u);
            }
            mma_commit_pair(&empty[stage]);
            if (j == nk - 1) mma_commit_pair(acc_full);
          }
          __syncwarp();
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else {
    // ------------------------------------------------ epilogue: this CTA's 128 rows x kBN tokens
    asm volatile("griddepcontrol.wait;" ::: "memory");      // x_global
    const int quarter = warp & 3;
    const uint32_t free_bar = cluster_map(smem_u32(acc_free), 0);
    uint32_t n = 0;
    for (int u = first; u < ntiles; u += stride, ++n) {
      const Tile w = tile_of(u, a);
      const int64_t row = static_cast<int64_t>(w.mt) * 256 + rank * 128 + quarter * 32 + lane;
      const bool row_ok = row < a.rows;
      MxRowScale gw = {1.0f, 1.0f};
      if (kFmt == kNvFp4 && row_ok) gw = mx_row_scale(__ldg(a.w_global + (a.w_per_row ? row : 0)));
      if (kFmt == kNvFp4) {
        // the scales are written by the kernel before, which this one's start overlaps:
        // no read-only loads
        __syncwarp();                        // all lanes are done with the tile before
#pragma unroll
        for (int i = 0; i < kBN / 32; ++i) {
          const int64_t t = static_cast<int64_t>(w.tt) * kBN + i * 32 + lane;
          reinterpret_cast<float*>(s_gx[quarter])[i * 32 + lane] = t < a.m ? __ldcg(a.x_global + t) : 1.0f;
        }
        __syncwarp();
      }
      if (!mbar_wait(acc_full, n & 1u, a.err)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (n & 1u) * kAcc1;
      // the columns that the two accumulators share come first
      const int c0 = (n & 1u) ? 0 : (kBN == 256 ? kChunks - kShared : 0);
#pragma unroll 1
      for (int i = 0; i < kChunks; ++i) {
        const int cc = c0 + i < kChunks ? c0 + i : c0 + i - kChunks;
        uint32_t v[16];
        tmem_ld16(taddr + cc * 16, v);
        tmem_wait_ld();
        if (i == kShared - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(free_bar);
        }
        const int64_t t0 = static_cast<int64_t>(w.tt) * kBN + cc * 16;
        uint16_t* dst = a.out + t0 * a.rows + row;
        auto store = [&](auto scaled) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const __nv_bfloat16 b = __float2bfloat16_rn(scaled(__uint_as_float(v[c]), c));
            if (row_ok && t0 + c < a.m) __stcs(dst + c * a.rows, *reinterpret_cast<const unsigned short*>(&b));
          }
        };
        if constexpr (kFmt == kMxFp4) {
          store([](float y, int) { return y; });
        } else {
          float4 gx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) gx[c] = s_gx[quarter][cc * 4 + c];
          store([&](float y, int c) { return mx_scaled(y, (&gx[c >> 2].x)[c & 3], gw); });
        }
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  cluster_sync();                            // no CTA leaves while its pair still reads or signals it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int kFmt, int kBN>
cudaError_t launch_t(const MxGemmArgs& a, const MxMaps& m, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr size_t smem = pair_smem(kFmt, kBN);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_mx_pair<kFmt, kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.t_tiles;
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_mx_pair<kFmt, kBN>, a, m.w, m.x, m.w_scales, m.x_scales, m.lora_w, m.lora_x);
}

}  // namespace

cudaError_t launch_mx_pair(int fmt, int token_tile, const MxGemmArgs& a, const MxMaps& m, int num_sms,
                           cudaStream_t stream) {
  if (fmt == kMxFp4)
    return token_tile == 256 ? launch_t<kMxFp4, 256>(a, m, num_sms, stream) : launch_t<kMxFp4, 128>(a, m, num_sms, stream);
  return token_tile == 256 ? launch_t<kNvFp4, 256>(a, m, num_sms, stream) : launch_t<kNvFp4, 128>(a, m, num_sms, stream);
}

}  // namespace qlora
