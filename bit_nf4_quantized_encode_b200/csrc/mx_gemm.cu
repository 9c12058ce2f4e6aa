// mx_gemm.cu -- the product of two microscaled 4-bit operands on tcgen05's
// block-scaled instructions (sm_100a).
//
//   out[t, n] = bf16( gx[t] gw[n] sum_k x[t, k] w[n, k]  +  lora_x[t] . lora_w[n] )
//
// x and w are e2m1 codes times block scales (E8M0 per 32 or E4M3 per 16), gx
// and gw the global scales of NVFP4.  The tensor core multiplies by the block
// scales itself and sums in fp32, so nothing is expanded: per 256 elements of
// the contraction a stage holds 128 bytes of codes per row and the scale tiles,
// which tcgen05.cp moves to TMEM.  The weight is the M operand (128 rows), the
// tokens the N operand, for few tokens as for many.  The rank-r term is a
// bf16 x bf16 product accumulated into the same TMEM tile (64 ranks a stage);
// with global scales its activation side arrives divided by gx gw.
//
// Few tokens: a tile's contraction is shared by the CTAs of a cluster, whose
// partial tiles meet in distributed shared memory and are summed in rank order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 6 * 32;            // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kABytes = 128 * 128;          // 128 rows x 256 codes

__host__ __device__ constexpr int atoms_per_stage(int fmt) { return fmt == kMxFp4 ? 2 : 4; }
__host__ __device__ constexpr int row_atoms(int bn) { return bn > 128 ? 2 : 1; }
__host__ __device__ constexpr int stage_bytes(int fmt, int bn) {
  return kABytes + bn * 128 + atoms_per_stage(fmt) * 512 * (1 + row_atoms(bn));
}
__host__ __device__ constexpr int num_stages(int bn) { return bn >= 128 ? 5 : (bn >= 64 ? 4 : 5); }
__host__ __device__ constexpr size_t smem_bytes(int fmt, int bn) {
  return 1024 + static_cast<size_t>(num_stages(bn)) * stage_bytes(fmt, bn) + 256;
}
__host__ __device__ constexpr int scale_cols(int fmt, int bn) { return atoms_per_stage(fmt) * 4 * (1 + row_atoms(bn)); }
__host__ __device__ constexpr uint32_t tmem_cols(int fmt, int bn) {
  const int need = 2 * bn + scale_cols(fmt, bn);
  uint32_t c = 32;
  while (static_cast<int>(c) < need) c *= 2;
  return c;
}

struct Tile {
  int mt, tt;
};
// Row tiles run fastest inside a group of m_group, which sweeps all token tiles.
__device__ __forceinline__ Tile tile_of(int u, const MxGemmArgs& a) {
  const int per_group = a.m_group * a.t_tiles;
  const int gi = u / per_group;
  const int r = u - gi * per_group;
  const int gsz = min(a.m_group, a.m_tiles - gi * a.m_group);
  return {gi * a.m_group + r % gsz, r / gsz};
}

template <int kFmt, int kBN>
__global__ void __launch_bounds__(kThreads)
k_mx_gemm(const MxGemmArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
          const __grid_constant__ CUtensorMap lwmap, const __grid_constant__ CUtensorMap lxmap) {
  constexpr int kStages = num_stages(kBN);
  constexpr int kStageBytes = stage_bytes(kFmt, kBN);
  constexpr int kAtoms = atoms_per_stage(kFmt);
  constexpr int kRB = row_atoms(kBN);
  constexpr uint32_t kCols = tmem_cols(kFmt, kBN);
  constexpr uint32_t kSfa = 2 * kBN, kSfb = kSfa + 4 * kAtoms;      // TMEM columns of the scales

  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_gen + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;      // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = a.splits;
  const int sp = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int ntiles = a.m_tiles * a.t_tiles;
  const int first = static_cast<int>(blockIdx.x) / splits, stride = static_cast<int>(gridDim.x) / splits;
  const int kbeg = static_cast<int>(static_cast<int64_t>(a.ksteps) * sp / splits);
  const int kend = static_cast<int>(static_cast<int64_t>(a.ksteps) * (sp + 1) / splits);
  const int lsteps = sp == splits - 1 ? a.lora_steps : 0;           // the rank-r steps follow the last split
  const int nk = kend - kbeg + lsteps;

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
    tmem_alloc(tmem_slot, kCols);
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

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      // The activations come from the kernel before this one, the weight does not.
      asm volatile("griddepcontrol.wait;" ::: "memory");
      uint32_t it = 0;
      bool alive = true;
      const int64_t x_row_tiles = (a.m + 127) / 128;
      for (int u = first; u < ntiles && alive; u += stride) {
        const Tile w = tile_of(u, a);
        for (int j = 0; j < nk; ++j, ++it) {
          const uint32_t stage = it % kStages, phase = (it / kStages) & 1u;
          if (!mbar_wait(&empty[stage], phase ^ 1u, a.err)) { alive = false; break; }
          uint8_t* sA = smem_gen + stage * kStageBytes;
          uint8_t* sB = sA + kABytes;
          const int ks = kbeg + j;
          if (ks < kend) {
            uint8_t* sSa = sB + kBN * 128;
            uint8_t* sSb = sSa + kAtoms * 512;
            const int atoms = min(kAtoms, static_cast<int>(a.kt) - ks * kAtoms);
            const int64_t rt = static_cast<int64_t>(w.tt) * kBN / 128;
            const int nrb = kRB == 1 || rt + 1 >= x_row_tiles ? 1 : 2;
            mbar_arrive_expect_tx(&full[stage], kABytes + kBN * 128 + static_cast<uint32_t>(atoms * 512 * (1 + nrb)));
            tma_load_2d(sA, &wmap, ks * 128, w.mt * 128, &full[stage]);
            bulk_load(sSa, a.w_scales + (static_cast<int64_t>(w.mt) * a.kt + ks * kAtoms) * 512,
                      static_cast<uint32_t>(atoms * 512), &full[stage]);
            tma_load_2d(sB, &xmap, ks * 128, w.tt * kBN, &full[stage]);
            for (int b = 0; b < nrb; ++b)
              bulk_load(sSb + b * (kAtoms * 512), a.x_scales + ((rt + b) * a.kt + ks * kAtoms) * 512,
                        static_cast<uint32_t>(atoms * 512), &full[stage]);
          } else {
            const int r0 = (ks - kend) * 64;
            mbar_arrive_expect_tx(&full[stage], kABytes + kBN * 128);
            if (a.lora_mn) {
              tma_load_2d(sA, &lwmap, w.mt * 128, r0, &full[stage]);
              tma_load_2d(sA + 8192, &lwmap, w.mt * 128 + 64, r0, &full[stage]);
            } else {
              tma_load_2d(sA, &lwmap, r0, w.mt * 128, &full[stage]);
            }
            tma_load_2d(sB, &lxmap, r0, w.tt * kBN, &full[stage]);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, uctr = 0;
      bool alive = true;
      const uint32_t lora_idesc = idesc_bf16(128, kBN, a.lora_mn != 0, false);
      for (int u = first; u < ntiles && alive; u += stride, ++uctr) {
        const uint32_t ab = uctr & 1u;
        if (!mbar_wait(&acc_empty[ab], ((uctr >> 1) & 1u) ^ 1u, a.err)) break;
        tc_fence_after();
        const uint32_t d = tmem + ab * kBN;
        for (int j = 0; j < nk; ++j, ++it) {
          const uint32_t stage = it % kStages, phase = (it / kStages) & 1u;
          if (!mbar_wait(&full[stage], phase, a.err)) { alive = false; break; }
          tc_fence_after();
          const uint32_t sA = smem0 + stage * kStageBytes;
          const uint32_t sB = sA + kABytes;
          const int ks = kbeg + j;
          if (ks < kend) {
            const uint32_t sSa = sB + kBN * 128, sSb = sSa + kAtoms * 512;
            const int atoms = min(kAtoms, static_cast<int>(a.kt) - ks * kAtoms);
            for (int t = 0; t < atoms; ++t) {
              tmem_cp_scales(tmem + kSfa + 4 * t, smem_desc_scales(sSa + t * 512));
#pragma unroll
              for (int b = 0; b < kRB; ++b)
                tmem_cp_scales(tmem + kSfb + 4 * (t * kRB + b), smem_desc_scales(sSb + (b * kAtoms + t) * 512));
            }
            const int slices = static_cast<int>(min(static_cast<int64_t>(4), (a.k - static_cast<int64_t>(ks) * 256 + 63) / 64));
            for (int q = 0; q < slices; ++q) {
              const uint64_t ad = smem_desc_sw128(sA + q * 32, 16, 1024);
              const uint64_t bd = smem_desc_sw128(sB + q * 32, 16, 1024);
              const uint32_t acc = (j | q) != 0 ? 1u : 0u;
              if (kFmt == kMxFp4)
                mma_mxf4_ss(d, ad, bd, idesc_mxf4(128, kBN, true, 2u * (q & 1)), tmem + kSfa + 4 * (q >> 1),
                            tmem + kSfb + 4 * kRB * (q >> 1), acc);
              else
                mma_nvf4_ss(d, ad, bd, idesc_mxf4(128, kBN, false, 0), tmem + kSfa + 4 * q, tmem + kSfb + 4 * kRB * q, acc);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t ad = a.lora_mn ? smem_desc_sw128(sA + q * 2048, 8192, 1024)
                                            : smem_desc_sw128(sA + q * 32, 16, 1024);
              mma_bf16_ss(d, ad, smem_desc_sw128(sB + q * 32, 16, 1024), lora_idesc, (j | q) != 0 ? 1u : 0u);
            }
          }
          mma_commit(&empty[stage]);
        }
        if (alive) mma_commit(&acc_full[ab]);
      }
    }
  } else if (splits == 1) {
    // ------------------------------------------------ epilogue: TMEM -> global
    asm volatile("griddepcontrol.wait;" ::: "memory");      // x_global
    const int quarter = warp & 3;
    uint32_t uctr = 0;
    for (int u = first; u < ntiles; u += stride, ++uctr) {
      const Tile w = tile_of(u, a);
      const uint32_t ab = uctr & 1u;
      if (!mbar_wait(&acc_full[ab], (uctr >> 1) & 1u, a.err)) break;
      tc_fence_after();
      const int64_t row = static_cast<int64_t>(w.mt) * 128 + quarter * 32 + lane;
      const bool row_ok = row < a.rows;
      float gw = 1.0f;
      if (a.w_global && row_ok) gw = __ldg(a.w_global + (a.w_per_row ? row : 0));
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ab * kBN;
      constexpr int kChunk = kBN < 32 ? kBN : 32;
#pragma unroll 1
      for (int cc = 0; cc < kBN / kChunk; ++cc) {
        uint32_t v[kChunk];
        if constexpr (kChunk == 32) tmem_ld32(taddr + cc * 32, v);
        else tmem_ld16(taddr, v);
        tmem_wait_ld();
        const int64_t t0 = static_cast<int64_t>(w.tt) * kBN + cc * kChunk;
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          if (row_ok && t0 + c < a.m) {
            float val = __uint_as_float(v[c]);
            if (a.x_global) val = __fmul_rn(val, __fmul_rn(__ldg(a.x_global + t0 + c), gw));
            const __nv_bfloat16 b = __float2bfloat16_rn(val);
            __stcs(a.out + (t0 + c) * a.rows + row, *reinterpret_cast<const unsigned short*>(&b));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[ab]);
    }
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    mbar_wait(&acc_full[0], 0, a.err);
    tc_fence_after();
  }

  if (splits > 1) {
    // ------------------------------------------------ one tile per cluster: join the partial tiles.
    // CTA q owns columns q * kBN / splits ...; every CTA sends it that part of
    // its own tile, into the stages (all MMAs of the cluster are done), and the
    // owner sums the parts in rank order.
    __syncwarp();
    cluster_sync();
    const int quarter = warp & 3;
    const int rl = quarter * 32 + lane;
    const int own = kBN / splits;
    if (warp >= 2) {
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
      constexpr int kChunk = kBN < 32 ? kBN : 32;
#pragma unroll 1
      for (int cc = 0; cc < kBN / kChunk; ++cc) {
        uint32_t v[kChunk];
        if constexpr (kChunk == 32) tmem_ld32(taddr + cc * 32, v);
        else tmem_ld16(taddr, v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          const int col = cc * kChunk + c;
          const uint32_t dst = smem0 + static_cast<uint32_t>((sp * own + col % own) * 128 + rl) * 4u;
          st_cluster_f32(cluster_map(dst, static_cast<uint32_t>(col / own)), __uint_as_float(v[c]));
        }
      }
    }
    cluster_sync();
    if (warp >= 2 && first < ntiles) {
      const Tile w = tile_of(first, a);
      const int64_t row = static_cast<int64_t>(w.mt) * 128 + rl;
      const float* part = reinterpret_cast<const float*>(smem_gen) + rl;
      if (row < a.rows) {
        float gw = 1.0f;
        if (a.w_global) gw = __ldg(a.w_global + (a.w_per_row ? row : 0));
        for (int c = 0; c < own; ++c) {
          const int64_t tok = static_cast<int64_t>(w.tt) * kBN + sp * own + c;
          if (tok >= a.m) break;
          float val = 0.0f;
          for (int q = 0; q < splits; ++q) val += part[(q * own + c) * 128];
          if (a.x_global) val = __fmul_rn(val, __fmul_rn(__ldg(a.x_global + tok), gw));
          const __nv_bfloat16 b = __float2bfloat16_rn(val);
          a.out[tok * a.rows + row] = *reinterpret_cast<const uint16_t*>(&b);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <int kFmt, int kBN>
cudaError_t launch_t(const MxGemmArgs& a, const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& lw,
                     const CUtensorMap& lx, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr size_t smem = smem_bytes(kFmt, kBN);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_mx_gemm<kFmt, kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.t_tiles;
  int64_t grid = tiles * a.splits;
  if (a.splits == 1 && grid > num_sms) grid = num_sms;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_gemm<kFmt, kBN>, a, w, x, lw, lx);
}

template <int kFmt>
cudaError_t launch_f(const MxGemmArgs& a, const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& lw,
                     const CUtensorMap& lx, int num_sms, cudaStream_t stream) {
  switch (mx_token_tile(a.m)) {
    case 16: return launch_t<kFmt, 16>(a, w, x, lw, lx, num_sms, stream);
    case 32: return launch_t<kFmt, 32>(a, w, x, lw, lx, num_sms, stream);
    case 64: return launch_t<kFmt, 64>(a, w, x, lw, lx, num_sms, stream);
    default: return launch_t<kFmt, 128>(a, w, x, lw, lx, num_sms, stream);
  }
}

}  // namespace

int mx_token_tile(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128; }

cudaError_t launch_mx_gemm(int fmt, const MxGemmArgs& a, const CUtensorMap& w, const CUtensorMap& x,
                           const CUtensorMap& lora_w, const CUtensorMap& lora_x, int num_sms, cudaStream_t stream) {
  return fmt == kMxFp4 ? launch_f<kMxFp4>(a, w, x, lora_w, lora_x, num_sms, stream)
                       : launch_f<kNvFp4>(a, w, x, lora_w, lora_x, num_sms, stream);
}

}  // namespace qlora
