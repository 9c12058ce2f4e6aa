// mx_stream.cu -- the product of two microscaled 4-bit operands for few tokens
// (at most 64) on tcgen05's block-scaled instructions (sm_100a).
//
//   out[t, n] = bf16( gx[t] gw[n] sum_k x[t, k] w[n, k]  +  lora_x[t] . lora_w[n] )
//
// x and w are e2m1 codes times block scales (E8M0 per 32 or E4M3 per 16), gx
// and gw the global scales of NVFP4.  The tensor core multiplies by the block
// scales itself and sums in fp32, so nothing is expanded: per 256 elements of
// the contraction a stage holds 128 bytes of codes per row and the scale tiles,
// which tcgen05.cp moves to TMEM.  The weight is the M operand (128 rows), the
// tokens the N operand.  The rank-r term is a bf16 x bf16 product accumulated
// into the same TMEM tile (64 ranks a step); its activation side arrives in two
// bf16 parts (bf16_parts.cuh) that meet the same weight tile, and with global
// scales divided by gx gw.
//
// The weight's bytes bound it, so every SM has to stream all the time: the steps
// of all row tiles are dealt to the SMs in equal runs (mx_runs.cuh).
// The first stages' weight tiles are requested before the kernel that quantises
// the activations has ended.  22016 x 8192 MXFP4, 16 tokens: 22.8 us with the
// quantiser, 4.2 TB/s; the last product is issued when 15 us of weight have been
// read, the rest is the launch before and the joining behind.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_format.cuh"
#include "mx_ptx.cuh"
#include "mx_runs.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 6 * 32;            // warp 0 TMA, warp 1 MMA, warps 2..5 epilogue
constexpr int kABytes = 128 * 128;          // 128 rows x 256 codes (or 64 ranks)
// A step is two pieces of 256 of the contraction (of 64 ranks), one stage: issuing
// the waits, the election and the commit of a stage costs 270 of the 650 cycles
// that a piece takes, and 512 make the weight rows runs of 256 bytes.
constexpr int kSub = 2;

__host__ __device__ constexpr int atoms_of(int fmt) { return fmt == kMxFp4 ? 2 : 4; }
__host__ __device__ constexpr int piece_bytes(int fmt, int bn) { return kABytes + bn * 128 + 2 * atoms_of(fmt) * 512; }
__host__ __device__ constexpr int stream_stage(int fmt, int bn) { return kSub * piece_bytes(fmt, bn); }
__host__ __device__ constexpr int stream_stages(int fmt, int bn) { return (224 * 1024 - 2048) / stream_stage(fmt, bn); }
__host__ __device__ constexpr size_t stream_smem(int fmt, int bn) {
  return 1024 + static_cast<size_t>(stream_stages(fmt, bn)) * stream_stage(fmt, bn) + 512;
}
__host__ __device__ constexpr uint32_t stream_cols(int fmt, int bn) {
  const int need = 2 * bn + 2 * 4 * atoms_of(fmt);
  uint32_t c = 32;
  while (static_cast<int>(c) < need) c *= 2;
  return c;
}

template <int kFmt, int kBN>
__global__ void __launch_bounds__(kThreads, 1)
k_mx_stream(const MxGemmArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
            const __grid_constant__ CUtensorMap lwmap, const __grid_constant__ CUtensorMap lxmap) {
  constexpr int kStages = stream_stages(kFmt, kBN);
  constexpr int kStageBytes = stream_stage(kFmt, kBN), kPiece = piece_bytes(kFmt, kBN);
  constexpr int kAtoms = atoms_of(kFmt);
  constexpr uint32_t kCols = stream_cols(kFmt, kBN);
  constexpr uint32_t kSfa = 2 * kBN, kSfb = kSfa + 4 * kAtoms;      // TMEM columns of the scales

  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_gen + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;      // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = warp_index();
  const int lane = threadIdx.x & 31;
  // steps of a tile: ksteps of 512, then the rank-r ones of 64 (two pieces of activations, one of weight)
  static_assert(kSub == 2);
  const int ksteps = (a.ksteps + kSub - 1) / kSub, per_tile = ksteps + a.lora_steps;
  const int64_t total = static_cast<int64_t>(a.m_tiles) * per_tile;
  const int runs = static_cast<int>(gridDim.x);
  const int64_t begin = run_begin(total, static_cast<int>(blockIdx.x), runs);
  const int64_t end = run_begin(total, static_cast<int>(blockIdx.x) + 1, runs);
  const int tile0 = static_cast<int>(begin / per_tile), step0 = static_cast<int>(begin - static_cast<int64_t>(tile0) * per_tile);
  const int nsteps = static_cast<int>(end - begin);

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
  if (warp == 0 && elect_one()) {
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    // weight side of step (tile, j) into a stage, with the stage's byte count
    auto load_w = [&](int stage, int tile, int j) {
      uint8_t* sA = smem_gen + stage * kStageBytes;
      if (j < ksteps) {
        const int pieces = min(kSub, a.ksteps - j * kSub);
        const int atoms = min(kSub * kAtoms, static_cast<int>(a.kt) - j * (kSub * kAtoms));      // of all pieces
        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(pieces * (kABytes + kBN * 128) + 2 * atoms * 512));
#pragma unroll
        for (int p = 0; p < kSub; ++p)
          if (p < pieces) {
            tma_load_2d(sA + p * kPiece, &wmap, (j * kSub + p) * 128, tile * 128, &full[stage]);
            bulk_load(sA + p * kPiece + kABytes + kBN * 128,
                      a.w_scales + (static_cast<int64_t>(tile) * a.kt + (j * kSub + p) * kAtoms) * 512,
                      static_cast<uint32_t>(min(kAtoms, atoms - p * kAtoms) * 512), &full[stage]);
          }
      } else {
        const int r0 = (j - ksteps) * 64;
        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(kABytes + 2 * kBN * 128));
        if (a.lora_mn) {
          tma_load_2d(sA, &lwmap, tile * 128, r0, &full[stage]);
          tma_load_2d(sA + 8192, &lwmap, tile * 128 + 64, r0, &full[stage]);
        } else {
          tma_load_2d(sA, &lwmap, r0, tile * 128, &full[stage]);
        }
      }
    };
    auto load_x = [&](int stage, int j) {
      uint8_t* sB = smem_gen + stage * kStageBytes + kABytes;
      if (j < ksteps) {
        const int pieces = min(kSub, a.ksteps - j * kSub);
        const int atoms = min(kSub * kAtoms, static_cast<int>(a.kt) - j * (kSub * kAtoms));
#pragma unroll
        for (int p = 0; p < kSub; ++p)
          if (p < pieces) {
            tma_load_2d(sB + p * kPiece, &xmap, (j * kSub + p) * 128, 0, &full[stage]);
            bulk_load(sB + p * kPiece + kBN * 128 + kAtoms * 512,
                      a.x_scales + static_cast<int64_t>(j * kSub + p) * (kAtoms * 512),
                      static_cast<uint32_t>(min(kAtoms, atoms - p * kAtoms) * 512), &full[stage]);
          }
      } else {
#pragma unroll
        for (int p = 0; p < 2; ++p) tma_load_2d(sB + p * kPiece, &lxmap, (j - ksteps) * 128 + p * 64, 0, &full[stage]);
      }
    };
    const int early = min(kStages, nsteps);
    int tile = tile0, j = step0;
    for (int i = 0; i < early; ++i) {
      if (elect_one()) load_w(i, tile, j);
      __syncwarp();
      if (++j == per_tile) { j = 0; ++tile; }
    }
    // the activations come from the kernel before this one
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int jx = step0;
    for (int i = 0; i < early; ++i) {
      if (elect_one()) load_x(i, jx);
      __syncwarp();
      if (++jx == per_tile) jx = 0;
    }
    uint32_t stage = early == kStages ? 0 : early, phase = early == kStages ? 1 : 0;
    for (int i = early; i < nsteps; ++i) {
      if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err)) break;
      if (elect_one()) {
        load_w(static_cast<int>(stage), tile, j);
        load_x(static_cast<int>(stage), j);
      }
      __syncwarp();
      if (++j == per_tile) { j = 0; ++tile; }
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0, seg = 0;
    const uint32_t lora_idesc = idesc_bf16(128, kBN, a.lora_mn != 0, false);
    const uint64_t desc0 = smem_desc_sw128(smem0, 16, 1024);         // + (byte offset >> 4)
    const uint64_t sdesc0 = smem_desc_scales(smem0);
    int j = step0;
    bool fresh = true;
    for (int i = 0; i < nsteps; ++i) {
      const uint32_t ab = seg & 1u;
      if (fresh && !mbar_wait_warp(&acc_empty[ab], ((seg >> 1) & 1u) ^ 1u, a.err)) break;
      if (!mbar_wait_warp(&full[stage], phase, a.err)) break;
      tc_fence_after();
      const uint32_t d = tmem + ab * kBN;
      const uint32_t off = stage * (kStageBytes >> 4);
      const uint64_t ad = desc0 + off, bd = ad + (kABytes >> 4);
      const bool last = j == per_tile - 1 || i == nsteps - 1;        // of this run's part of the tile
      if (elect_one()) {
        if (j < ksteps) {
          const int pieces = min(kSub, a.ksteps - j * kSub);
          const int atoms = min(kSub * kAtoms, static_cast<int>(a.kt) - j * (kSub * kAtoms));
          const int slices = static_cast<int>(min(static_cast<int64_t>(4 * kSub), (a.k - static_cast<int64_t>(j) * (256 * kSub) + 63) / 64));
#pragma unroll
          for (int p = 0; p < kSub; ++p)
            if (p < pieces) {
              const uint64_t sa = sdesc0 + off + ((p * kPiece + kABytes + kBN * 128) >> 4), sb = sa + (kAtoms * 512 >> 4);
#pragma unroll
              for (int t = 0; t < kAtoms; ++t)
                if (p * kAtoms + t < atoms) {
                  tmem_cp_scales(tmem + kSfa + 4 * t, sa + t * 32);
                  tmem_cp_scales(tmem + kSfb + 4 * t, sb + t * 32);
                }
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (p * 4 + q < slices) {
                  const uint32_t acc = !fresh || p + q != 0 ? 1u : 0u;
                  const uint64_t x = ad + (p * kPiece >> 4) + q * 2, y = bd + (p * kPiece >> 4) + q * 2;
                  if (kFmt == kMxFp4)
                    mma_mxf4_ss(d, x, y, idesc_mxf4(128, kBN, true, 2u * (q & 1)), tmem + kSfa + 4 * (q >> 1),
                                tmem + kSfb + 4 * (q >> 1), acc);
                  else
                    mma_nvf4_ss(d, x, y, idesc_mxf4(128, kBN, false, 0), tmem + kSfa + 4 * q, tmem + kSfb + 4 * q, acc);
                }
            }
        } else {
          // A K = 16 slice: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
          const uint64_t la = a.lora_mn ? smem_desc_sw128(smem0, 8192, 1024) + off : ad;
          const uint32_t step = a.lora_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mma_bf16_ss(d, la + q * step, bd + (p * kPiece >> 4) + q * 2, lora_idesc, !fresh || p + q != 0 ? 1u : 0u);
        }
        mma_commit(&empty[stage]);
        if (last) mma_commit(&acc_full[ab]);
      }
      __syncwarp();
      fresh = last;
      if (last) ++seg;
      if (++j == per_tile) j = 0;
      if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
  } else {
    // ------------------------------------------------ epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");      // x_global and the zeroed counters
    const int quarter = warp & 3, rl = quarter * 32 + lane;
    const int m = static_cast<int>(a.m);
    // lane t: the global scales of tokens t and t + 32
    float gx0 = 1.0f, gx1 = 1.0f;
    if (kFmt == kNvFp4) {
      if (lane < m) gx0 = __ldcg(a.x_global + lane);
      if (lane + 32 < m) gx1 = __ldcg(a.x_global + lane + 32);
    }
    constexpr int kChunk = kBN < 32 ? kBN : 32;
    const int64_t slot_floats = static_cast<int64_t>(m) * 128;
    int tile = tile0, j = step0, left = nsteps;
    for (uint32_t seg = 0; left > 0; ++seg, ++tile, j = 0) {
      const int steps = min(per_tile - j, left);
      left -= steps;
      const uint32_t ab = seg & 1u;
      const bool whole = steps == per_tile;
      const int64_t row = static_cast<int64_t>(tile) * 128 + rl;
      const bool row_ok = row < a.rows;
      // all that does not need the products, before waiting for them
      Parts p{};
      uint32_t* counter = a.counters + tile * 4 + quarter;
      bool alone = false;                    // the other runs' parts are there
      if (!whole) {
        p = parts_of(a.slots + rl, slot_floats, total, static_cast<int64_t>(tile) * per_tile, per_tile, runs);
        alone = others_counted(counter, p.n);
      }
      MxRowScale gw = {1.0f, 1.0f};
      if (kFmt == kNvFp4 && row_ok) gw = mx_row_scale(__ldg(a.w_global + (a.w_per_row ? row : 0)));
      auto store = [&](int t, float v) {
        if (kFmt == kNvFp4) v = mx_scaled(v, __shfl_sync(0xFFFFFFFFu, t < 32 ? gx0 : gx1, t & 31), gw);
        if (!row_ok) return;
        const __nv_bfloat16 b = __float2bfloat16_rn(v);
        a.out[t * a.rows + row] = *reinterpret_cast<const uint16_t*>(&b);
      };
      if (!mbar_wait_warp(&acc_full[ab], (seg >> 1) & 1u, a.err)) break;
      tc_fence_after();
      if (!whole && !alone && left == 0) alone = others_counted(counter, p.n);
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + ab * kBN;
      float* mine = my_slot(a.slots, slot_floats, tile == tile0) + rl;
#pragma unroll 1
      for (int cc = 0; cc * kChunk < m; ++cc) {
        uint32_t v[kChunk];
        if constexpr (kChunk == 32) tmem_ld32(taddr + cc * 32, v);
        else tmem_ld16(taddr, v);
        tmem_wait_ld();
        float f[kChunk];
#pragma unroll
        for (int c = 0; c < kChunk; ++c) f[c] = __uint_as_float(v[c]);
        if (alone) add_parts<kChunk>(p, static_cast<int>(blockIdx.x) - p.c0, cc * kChunk, m, f);
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          const int t = cc * kChunk + c;
          if (t < m) {
            if (whole || alone) store(t, f[c]);
            else mine[t * 128] = f[c];
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[ab]);
      // each warp counts its own 32 rows, so no warp waits for another
      if (!whole && !alone && count_part(counter, p.n)) join_columns(p, m, store);
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <int kFmt, int kBN>
cudaError_t launch_t(const MxGemmArgs& a, const MxMaps& m, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr size_t smem = stream_smem(kFmt, kBN);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_mx_stream<kFmt, kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t steps = static_cast<int64_t>(a.m_tiles) * ((a.ksteps + kSub - 1) / kSub + a.lora_steps);
  int grid = num_sms < kMxMaxRuns ? num_sms : kMxMaxRuns;
  if (steps < grid) grid = static_cast<int>(steps);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_mx_stream<kFmt, kBN>, a, m.w, m.x, m.lora_w, m.lora_x);
}

template <int kFmt>
cudaError_t launch_f(int token_tile, const MxGemmArgs& a, const MxMaps& m, int num_sms, cudaStream_t stream) {
  switch (token_tile) {
    case 16: return launch_t<kFmt, 16>(a, m, num_sms, stream);
    case 32: return launch_t<kFmt, 32>(a, m, num_sms, stream);
    default: return launch_t<kFmt, 64>(a, m, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_mx_stream(int fmt, int token_tile, const MxGemmArgs& a, const MxMaps& m, int num_sms,
                             cudaStream_t stream) {
  return fmt == kMxFp4 ? launch_f<kMxFp4>(token_tile, a, m, num_sms, stream)
                       : launch_f<kNvFp4>(token_tile, a, m, num_sms, stream);
}

}  // namespace qlora
