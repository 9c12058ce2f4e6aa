// mx_xa.cu -- X A^T of the LoRA branch for few tokens (sm_100a).
//
// XA [m, r] = X [m, k] A^T, A [r, k]: 2 r k bytes of A and 2 m k of X for 2 m r k
// operations, so it is all latency and spread.  A cluster of eight CTAs takes 16
// ranks x 16 tokens, an eighth of k each; every warp multiplies its share with
// m16n8k16 (bf16 in, fp32 sums), the warps of a CTA meet in shared memory and the
// CTAs in the first one's, both summed in a fixed order.  It runs beside the
// quantisation of X, and finds NVFP4's global scale of a token by itself.  16
// tokens of 22016, rank 64: 4 to 5 us more than the product without the term.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bf16_parts.cuh"
#include "mx.h"
#include "mx_encode.cuh"
#include "mx_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kCluster = 8;

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1) k_mx_xa(const MxXaArgs a) {
  __shared__ float part[kWarps][16][17];       // per warp, then (CTA 0) per CTA of the cluster
  __shared__ float joined[kCluster][16][17];
  __shared__ uint32_t s_amax[16];              // the first CTA's: largest finite magnitude of each token
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x < 16) s_amax[threadIdx.x] = 0u;
  __syncthreads();
  cluster_sync();                              // the first CTA runs before the others write to it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_rank();
  const int r0 = static_cast<int>(blockIdx.x) / kCluster * 16, m0 = static_cast<int>(blockIdx.y) * 16;

  // 64 columns a step; a lane's 16 bytes of a row are columns 8t .. 8t+7 of each
  // 32: the same order in both operands, so any order will do for the sum.
  const int steps = static_cast<int>(a.k / 64), lanes = kCluster * kWarps;
  float d[2][4] = {};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint32_t mag_a = 0, mag_b = 0;               // of tokens g and g + 8
  const bool ra = r0 + g < a.r, rb = r0 + g + 8 < a.r, ta = m0 + g < a.m, tb = m0 + g + 8 < a.m;
  const uint4* pa = reinterpret_cast<const uint4*>(a.a + (r0 + g) * a.k) + t;
  const uint4* pb = reinterpret_cast<const uint4*>(a.a + (r0 + g + 8) * a.k) + t;
  const uint4* xa = reinterpret_cast<const uint4*>(a.x + (m0 + g) * a.k) + t;
  const uint4* xb = reinterpret_cast<const uint4*>(a.x + (m0 + g + 8) * a.k) + t;
#pragma unroll 2
  for (int s = static_cast<int>(rank) * kWarps + warp; s < steps; s += lanes) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = s * 8 + h * 4;
      const uint4 wa = ra ? __ldg(pa + o) : zero, wb = rb ? __ldg(pb + o) : zero;
      const uint4 va = ta ? __ldg(xa + o) : zero, vb = tb ? __ldg(xb + o) : zero;
      if (a.all_div) {
        mag_a = max(mag_a, finite_mag8(va));
        mag_b = max(mag_b, finite_mag8(vb));
      }
      // columns 8t .. 8t+7 of a row feed two products of 16
      const uint32_t a0[4] = {wa.x, wb.x, wa.y, wb.y}, a1[4] = {wa.z, wb.z, wa.w, wb.w};
      const uint32_t p0[2] = {va.x, va.y}, p1[2] = {va.z, va.w}, q0[2] = {vb.x, vb.y}, q1[2] = {vb.z, vb.w};
      mma_16x8x16(d[0], a0, p0);
      mma_16x8x16(d[0], a1, p1);
      mma_16x8x16(d[1], a0, q0);
      mma_16x8x16(d[1], a1, q1);
    }
  }
  // d[n][i]: rank g (+8 for i >= 2), token 8n + 2t + (i & 1)
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = d[n][i];
  if (a.all_div) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      mag_a = max(mag_a, __shfl_xor_sync(0xFFFFFFFFu, mag_a, o));
      mag_b = max(mag_b, __shfl_xor_sync(0xFFFFFFFFu, mag_b, o));
    }
    if (t == 0) {
      atomic_max_cluster(cluster_map(smem_u32(&s_amax[g]), 0), mag_a);
      atomic_max_cluster(cluster_map(smem_u32(&s_amax[g + 8]), 0), mag_b);
    }
  }
  __syncthreads();
  const int rr = (threadIdx.x >> 4) & 15, tt = threadIdx.x & 15;
  float v = 0.0f;
  if (threadIdx.x < 256) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w][rr][tt];
    st_cluster_f32(cluster_map(smem_u32(&joined[rank][rr][tt]), 0), v);
  }
  cluster_sync();
  if (rank != 0 || threadIdx.x >= 256) return;
  v = 0.0f;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) v += joined[c][rr][tt];
  asm volatile("griddepcontrol.wait;" ::: "memory");         // a reader of this kernel's end may rely on the one before
  const int rank_row = r0 + rr, tok = m0 + tt;
  if (tok >= a.m) return;
  if (a.xa && rank_row < a.r) a.xa[static_cast<int64_t>(tok) * a.r + rank_row] = v;
  if (rank_row < a.rpad) {
    v = __fmul_rn(a.s, v);
    // one divisor after the other: their product may be below what a float holds
    if (a.all_div) v = __fdiv_rn(__fmul_rn(v, mx_pow2_inverse(mx_global_scale(s_amax[tt] << 16))), a.all_div[0]);
    const BfParts p = bf16_parts(v);
    uint16_t* dst = a.sxa + static_cast<int64_t>(tok) * (2 * a.rpad) + (rank_row >> 6) * 128 + (rank_row & 63);
    dst[0] = bf16_bits(p.first);
    dst[64] = bf16_bits(p.second);
  }
}

}  // namespace

cudaError_t launch_mx_xa(const MxXaArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rpad / 16 * kCluster), static_cast<unsigned>((a.m + 15) / 16));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.first ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_xa, a);
}

}  // namespace qlora
