// mx_few.cu -- the product of a microscaled 4-bit weight with at most 16 tokens,
// the tokens' quantisation included, in one launch (sm_100a).  The formula and
// the operands are those of mx_stream.cu.
//
// For a token or a few the time is the weight's bytes plus whatever the launch
// does before and after them, so nothing of that is spread over kernels: every CTA
// quantises the tokens itself (they are 2 m k bytes, read from L2) into the operand
// that stays in shared memory, while its first weight tiles are on the way, and
// takes whole rows, so that no partial sum leaves it.  A row's unit is 32 rows
// (one lane quarter of the accumulator, one column of a scale tile); the units
// are dealt evenly, up to eight at a time.
//
// The scales that an MMA reads start at a multiple of four TMEM columns (any other
// column is a misaligned address), so units keep their place in their tile of 128
// rows: a product covers whole tiles, and what its rows outside the CTA's units
// hold is never looked at.  They read whatever lies around the stage.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mx.h"
#include "mx_encode.cuh"
#include "mx_ptx.cuh"

namespace qlora {
namespace {

constexpr int kQuantWarps = 8;                       // warps 2..9; they are the epilogue too
constexpr int kThreads = 64 + 32 * kQuantWarps;      // warp 0 TMA, warp 1 MMA
constexpr int kUnits = 8;                            // 32-row units of a chunk at most
constexpr int kMaxStages = 12;
constexpr size_t kSmem = 224 * 1024;

constexpr int kTiles = 3;                            // 128-row tiles that eight units touch at most
constexpr uint32_t kPad = 3 * 4096;                  // a tile begins up to three units before its chunk

__host__ __device__ constexpr int atoms_of(int fmt) { return fmt == kMxFp4 ? 2 : 4; }
// Tokens' scale bytes of a step: 16 bytes a token and scale tile, of which four
// are used (the copies of 32 rows run on into the next ones).
__host__ __device__ constexpr int token_scales(int fmt, int n) { return atoms_of(fmt) * n * 16; }

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

template <int kFmt, int kN>
__global__ void __launch_bounds__(kThreads, 1)
k_mx_few(const MxFewArgs a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap lwmap,
         const __grid_constant__ CUtensorMap lxmap) {
  constexpr int kAtoms = atoms_of(kFmt);
  constexpr uint32_t kAcc = kTiles * kN;             // columns of one accumulator set
  constexpr uint32_t kSfw = 2 * kAcc, kSfx = kSfw + 4 * kTiles * kAtoms;
  constexpr uint32_t kCols = 256;
  constexpr int kSx = token_scales(kFmt, kN);
  static_assert(kSfx + 4 * kAtoms <= kCols);

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kMaxStages + 6];
  __shared__ uint32_t s_amax[16];
  __shared__ float s_g[16];
  __shared__ uint32_t tmem_slot;
  const uint32_t smem0 = ((smem_u32(smem_raw) + 1023u) & ~1023u) + kPad;
  uint8_t* smem_gen = smem_raw + (smem0 - smem_u32(smem_raw));
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* x_full = bars + 2 * kMaxStages;          // the quantised tokens (kQuantWarps * 32 arrivals)
  uint64_t* l_full = x_full + 1;                     // the rank-r activations (TMA)
  uint64_t* acc_full = l_full + 1;                   // [2]
  uint64_t* acc_empty = acc_full + 2;                // [2]

  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int stages = a.stages;
  const uint32_t stage_bytes = static_cast<uint32_t>(a.stage_bytes);
  const uint32_t x_off = stage_bytes * stages;       // tokens' codes, scales, rank-r activations
  const uint32_t sx_off = x_off + a.ksteps * (kN * 128), l_off = (sx_off + a.ksteps * kSx + 512u + 1023u) & ~1023u;
  // this CTA's units, in chunks of nearly equal size
  // (the first `more` CTAs have one more than the others)
  const int total_units = static_cast<int>((a.rows + 31) / 32), cta = static_cast<int>(blockIdx.x);
  const int least = total_units / static_cast<int>(gridDim.x), more = total_units - least * static_cast<int>(gridDim.x);
  const int u0 = cta * least + min(cta, more), units = least + (cta < more ? 1 : 0);
  const int chunks = a.chunks;
  const int per_chunk = a.ksteps + a.lora_steps;
  struct Chunk {
    int unit;                                        // first
    int n, tile, tiles, col;                         // units, first row tile of its scales, how many, first column
  };
  auto chunk_of = [&](int c) {
    Chunk k;
    // chunk c has one unit more than the last ones while c is below the remainder
    const int each = units / chunks, left = units - each * chunks;
    k.unit = u0 + each * c + min(c, left);
    k.n = each + (c < left ? 1 : 0);
    k.tile = k.unit >> 2;
    k.col = k.unit & 3;
    k.tiles = (k.col + k.n + 3) >> 2;
    return k;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(x_full, kQuantWarps * 32);
    mbar_init(l_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kQuantWarps * 32);
    }
    fence_barrier_init();
  }
  if (threadIdx.x < 16) s_amax[threadIdx.x] = 0u;
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp == 0 && elect_one()) tma_prefetch_desc(&wmap);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // With a rank-r term the kernel before this one is the one that makes it, which
  // began after everything else; without, nothing may be read before its end.
  if (a.lora_steps == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    uint32_t stage = 0, phase = 0;
    bool alive = true;
    for (int c = 0; c < chunks && alive; ++c) {
      const Chunk k = chunk_of(c);
      for (int j = 0; j < per_chunk; ++j) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1u, a.err)) { alive = false; break; }
        uint8_t* sA = smem_gen + stage * stage_bytes;
        if (elect_one()) {
          if (j < a.ksteps) {
            const int atoms = min(kAtoms, static_cast<int>(a.kt) - j * kAtoms);
            const uint32_t sbytes = static_cast<uint32_t>(atoms * 512);
            mbar_arrive_expect_tx(&full[stage], k.n * 4096 + k.tiles * sbytes);
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
              if (i < k.n) tma_load_2d(sA + i * 4096, &wmap, j * 128, (k.unit + i) * 32, &full[stage]);
            uint8_t* sS = sA + a.units * 4096;
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
              if (i < k.tiles) bulk_load(sS + i * (kAtoms * 512), a.w_scales + ((static_cast<int64_t>(k.tile) + i) * a.kt + j * kAtoms) * 512,
                        sbytes, &full[stage]);
          } else {
            mbar_arrive_expect_tx(&full[stage], k.n * 4096);
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
              if (i < k.n) tma_load_2d(sA + i * 4096, &lwmap, (j - a.ksteps) * 64, (k.unit + i) * 32, &full[stage]);
          }
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(stages)) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (a.lora_steps != 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (elect_one()) {
        mbar_arrive_expect_tx(l_full, static_cast<uint32_t>(2 * a.lora_steps) * kN * 128);
        for (int i = 0; i < 2 * a.lora_steps; ++i) tma_load_2d(smem_gen + l_off + i * (kN * 128), &lxmap, i * 64, 0, l_full);
      }
      __syncwarp();
    }
    uint32_t stage = 0, phase = 0;
    const uint64_t desc0 = smem_desc_sw128(smem0, 16, 1024);         // + (byte offset >> 4)
    const uint64_t sdesc0 = smem_desc_scales(smem0);
    bool alive = mbar_wait_warp(x_full, 0, a.err);
    for (int c = 0; c < chunks && alive; ++c) {
      const Chunk k = chunk_of(c);
      const uint32_t d = tmem + (c & 1) * kAcc;
      if (!mbar_wait_warp(&acc_empty[c & 1], ((c >> 1) & 1u) ^ 1u, a.err)) break;
      for (int j = 0; j < per_chunk; ++j) {
        if (!mbar_wait_warp(&full[stage], phase, a.err)) { alive = false; break; }
        if (j == a.ksteps && c == 0 && !mbar_wait_warp(l_full, 0, a.err)) { alive = false; break; }
        tc_fence_after();
        const uint32_t off = stage * (stage_bytes >> 4);
        const uint64_t ad = desc0 + off - k.col * (4096 >> 4);       // the first tile's first row
        if (elect_one()) {
          if (j < a.ksteps) {
            const uint64_t sw = sdesc0 + off + a.units * (4096 >> 4), sx = sdesc0 + ((sx_off + j * kSx) >> 4);
            const uint64_t bd = desc0 + ((x_off + j * (kN * 128)) >> 4);
            const int atoms = min(kAtoms, static_cast<int>(a.kt) - j * kAtoms);
#pragma unroll
            for (int t = 0; t < kAtoms; ++t)
              if (t < atoms) {
                tmem_cp_scales(tmem + kSfx + 4 * t, sx + t * kN);
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                  if (i < k.tiles) tmem_cp_scales(tmem + kSfw + 4 * (t * kTiles + i), sw + (i * kAtoms + t) * 32);
              }
            const int slices = static_cast<int>(min(static_cast<int64_t>(4), (a.k - static_cast<int64_t>(j) * 256 + 63) / 64));
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q < slices) {
                const uint32_t acc = (j | q) != 0 ? 1u : 0u;
                const int t = kFmt == kMxFp4 ? q >> 1 : q;
                const uint32_t id = kFmt == kMxFp4 ? 2u * (q & 1) : 0u;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                  if (i >= k.tiles) break;
                  const uint32_t sf = tmem + kSfw + 4 * (t * kTiles + i);
                  if (kFmt == kMxFp4)
                    mma_mxf4_ss(d + i * kN, ad + i * 1024 + q * 2, bd + q * 2, idesc_mxf4(128, kN, true, id), sf,
                                tmem + kSfx + 4 * t, acc);
                  else
                    mma_nvf4_ss(d + i * kN, ad + i * 1024 + q * 2, bd + q * 2, idesc_mxf4(128, kN, false, id), sf,
                                tmem + kSfx + 4 * t, acc);
                }
              }
          } else {
            const uint64_t bd = desc0 + ((l_off + (j - a.ksteps) * (2 * kN * 128)) >> 4);
#pragma unroll
            for (int p = 0; p < 2; ++p)                                  // the activations' two bf16 parts
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                  if (i < k.tiles)
                    mma_bf16_ss(d + i * kN, ad + i * 1024 + q * 2, bd + p * (kN * 128 >> 4) + q * 2,
                                idesc_bf16(128, kN, false, false), 1u);
          }
          mma_commit(&empty[stage]);
          if (j == per_chunk - 1) mma_commit(&acc_full[c & 1]);
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(stages)) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------ the tokens: quantise into shared memory
    const int tid = threadIdx.x - 64;
    const int m = a.m, per_row = a.ksteps * 8;       // 32 elements a task, whole steps
    const int tasks = m * per_row;
    auto load = [&](int i) {
      const int t = i / per_row;
      const int64_t c = static_cast<int64_t>(i - t * per_row) * 32;
      const uint16_t* row = a.x + static_cast<int64_t>(t) * a.k;
      const int64_t limit = (m - t) * a.k;
      return a.vec ? load32<true, true>(row, c, a.k, limit) : load32<false, true>(row, c, a.k, limit);
    };
    Elems32 first = {};
    if (tid < tasks) first = load(tid);
    if (kFmt == kNvFp4) {
      for (int i = tid; i < tasks; i += kQuantWarps * 32) {
        const Elems32 e = i == tid ? first : load(i);
        uint32_t mag = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) mag = max(mag, finite_mag8(e.q[q]));
        atomicMax(&s_amax[i / per_row], mag);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kQuantWarps * 32) : "memory");
      if (tid < m) s_g[tid] = mx_global_scale(s_amax[tid] << 16);
      asm volatile("bar.sync 1, %0;" ::"n"(kQuantWarps * 32) : "memory");
    }
    for (int i = tid; i < tasks; i += kQuantWarps * 32) {
      const Elems32 e = i == tid ? first : load(i);
      const int t = i / per_row, b = i - t * per_row;                  // 32-element piece of the row
      const float inv_g = kFmt == kNvFp4 ? mx_pow2_inverse(s_g[t]) : 1.0f;
      uint32_t scales;
      const uint4 codes = encode32<kFmt>(e, inv_g, scales);
      const uint32_t dst = x_off + (b >> 3) * (kN * 128) + sw128_offset(static_cast<uint32_t>(t), static_cast<uint32_t>(b & 7));
      *reinterpret_cast<uint4*>(smem_gen + dst) = codes;
      // its blocks are 4a + k of the step's: scale tile a, byte k
      uint8_t* sd = smem_gen + sx_off + (b >> 3) * kSx + t * 16;
      if (kFmt == kMxFp4) sd[((b >> 2) & 1) * (kN * 16) + (b & 3)] = static_cast<uint8_t>(scales);
      else *reinterpret_cast<uint16_t*>(sd + ((b >> 1) & 3) * (kN * 16) + 2 * (b & 1)) = static_cast<uint16_t>(scales);
    }
    fence_proxy_async_smem();
    mbar_arrive(x_full);
    // ------------------------------------------------ epilogue: warps 2..5 take tiles 0 and 2, warps 6..9 tile 1
    const int quarter = warp & 3;
    for (int c = 0; c < chunks; ++c) {
      const Chunk k = chunk_of(c);
      // the weight's global scale before waiting for the products (it may be as late as
      // X: no read-only load)
      MxRowScale gw = {1.0f, 1.0f};
      auto load_gw = [&](int i) {              // (a tile's rows may lie behind the last one, past 32 bits too)
        const int64_t row = static_cast<int64_t>(k.unit + i * 4 + quarter - k.col) * 32 + lane;
        if (kFmt == kNvFp4 && row < a.rows) gw = mx_row_scale(a.w_global[a.w_per_row ? row : 0]);
      };
      const int i0 = warp >= 6 ? 1 : 0;
      load_gw(i0);
      if (!mbar_wait(&acc_full[c & 1], (c >> 1) & 1u, a.err)) break;
      tc_fence_after();
      for (int i = i0; i < k.tiles; i += 2) {
        const int unit = i * 4 + quarter - k.col;
        if (unit < 0 || unit >= k.n) continue;
        uint32_t v[kN];
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (c & 1) * kAcc + i * kN;
        if constexpr (kN == 8) tmem_ld8(taddr, v);
        else tmem_ld16(taddr, v);
        tmem_wait_ld();
        const int row = (k.unit + unit) * 32 + lane;
        if (row < a.rows) {
          if (a.w_per_row && i != i0) load_gw(i);
#pragma unroll
          for (int t = 0; t < kN; ++t)
            if (t < m) {
              float y = __uint_as_float(v[t]);
              if (kFmt == kNvFp4) y = mx_scaled(y, s_g[t], gw);
              const __nv_bfloat16 b = __float2bfloat16_rn(y);
              a.out[static_cast<int64_t>(t) * a.rows + row] = *reinterpret_cast<const uint16_t*>(&b);
            }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[c & 1]);
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

// Shared memory behind the weight's stages.
size_t tokens_bytes(int fmt, int n, int ksteps, int lora_steps) {
  return (static_cast<size_t>(ksteps) * (n * 128 + token_scales(fmt, n)) + 512 + 1023) / 1024 * 1024 +
         static_cast<size_t>(2 * lora_steps) * n * 128;
}

template <int kFmt, int kN>
cudaError_t launch_t(MxFewArgs a, const MxMaps& m, int num_sms, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(k_mx_few<kFmt, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t units = (a.rows + 31) / 32;
  const int64_t grid = units < num_sms ? units : num_sms;
  const int64_t most = (units + grid - 1) / grid;                      // of one CTA
  a.chunks = static_cast<int>((most + kUnits - 1) / kUnits);           // the others have one unit less: chunks of one at least
  a.units = static_cast<int>((most + a.chunks - 1) / a.chunks);
  a.stage_bytes = a.units * 4096 + 3 * atoms_of(kFmt) * 512;
  // the last stage's tiles have to end inside the allocation, whatever of them the
  // chunk's units fill
  const size_t behind = tokens_bytes(kFmt, kN, a.ksteps, a.lora_steps);
  const size_t reach = static_cast<size_t>(kTiles) * 16384, room = kSmem - 1024 - kPad;
  a.stages = 0;
  while (a.stages < kMaxStages && (a.stages + 1) * static_cast<size_t>(a.stage_bytes) + behind <= room &&
         a.stages * static_cast<size_t>(a.stage_bytes) + reach <= room)
    ++a.stages;
  if (a.stages < 2) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_mx_few<kFmt, kN>, a, m.w, m.lora_w, m.lora_x);
}

}  // namespace

// Where one launch is faster than the quantiser's and the streamed product's, by a
// model of both in us on 148 SMs.  Here a chunk's step of 256 (or of 64 ranks) costs
// `step` and `unit` for each of its units, or `bytes` a unit at least (4.3 KB at an
// SM's share of memory bandwidth), quantising `quant` per 1024 elements, waiting for X
// A^T 0.5; there a tile's step of 256 costs `stream` (of 64 ranks a third of it), and
// the second kernel and the joining 5.5.  Both were timed at 720 calls (512 to 22016
// rows, 512 to 16384 columns, 1 to 16 tokens, rank 0 to 256): what the model takes is
// 0.2% (MXFP4) and 0.3% (NVFP4) slower than the faster one on average and 10% at most.
// MXFP4, one token: 22016 x 8192: 18.4 us here, 21.0 there; 4096 x 4096: 8.0 and 9.0;
// 8192 x 8192: 13.7 both; 8192 x 16384: 25.0 and 18.3.
int mx_few_tile(int fmt, int64_t rows, int64_t m, int64_t k, int lora_steps, int num_sms) {
  if (m > 16 || m * k > kMxFewElements) return 0;
  const int n = m <= 8 ? 8 : 16, ksteps = static_cast<int>((k + 255) / 256);
  if (tokens_bytes(fmt, n, ksteps, lora_steps) > kMxFewShared) return 0;
  struct Costs {
    double step, unit, bytes, quant, stream;
  };
  const Costs c = fmt == kMxFp4 ? Costs{0.30, 0.045, 0.100, 0.12, 0.42} : Costs{0.40, 0.033, 0.127, 0.19, 0.45};
  const int64_t units = (rows + 31) / 32, most = (units + num_sms - 1) / num_sms, chunks = (most + kUnits - 1) / kUnits;
  const double per = static_cast<double>(most) / chunks;
  const double step = c.step + c.unit * per > c.bytes * per ? c.step + c.unit * per : c.bytes * per;
  const double here = chunks * (ksteps + lora_steps) * step + c.quant * m * k / 1024 + (lora_steps ? 0.5 : 0.0);
  const double there = 5.5 + c.stream * static_cast<double>((rows + 127) / 128) * (ksteps + 0.34 * lora_steps) / num_sms;
  return here < there ? n : 0;
}

cudaError_t launch_mx_few(int fmt, int token_tile, const MxFewArgs& a, const MxMaps& m, int num_sms, cudaStream_t stream) {
  if (fmt == kMxFp4)
    return token_tile == 8 ? launch_t<kMxFp4, 8>(a, m, num_sms, stream) : launch_t<kMxFp4, 16>(a, m, num_sms, stream);
  return token_tile == 8 ? launch_t<kNvFp4, 8>(a, m, num_sms, stream) : launch_t<kNvFp4, 16>(a, m, num_sms, stream);
}

}  // namespace qlora
