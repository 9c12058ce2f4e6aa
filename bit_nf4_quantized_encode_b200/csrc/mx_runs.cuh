// mx_runs.cuh -- steps of a kernel's tiles dealt to its CTAs in equal runs, and
// the joining of a tile that several runs share.
//
// The tiles' steps are numbered one tile after the other; run c (CTA c of G) has
// steps [total c / G, total (c + 1) / G).  A run's part of a tile that it does not
// have whole goes to one of its two slots in the work buffer (its first tile's, or
// its last one's); the warp that completes the count of its rows of the tile sums
// the parts in the order of the runs, so results do not depend on who that is.
// Writing a part, making it visible, counting it and reading the others take 4 to
// 5 us at the end of a run.  The run behind usually has counted its part of a tile
// long before, with its first steps: a warp that finds all others counted sums
// them with its own values and writes nothing (0.6 us).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace qlora {

__device__ __forceinline__ int64_t run_begin(int64_t total, int c, int runs) { return total * c / runs; }
// The run that has a step.
__device__ __forceinline__ int run_of(int64_t total, int64_t step, int runs) {
  return static_cast<int>(((step + 1) * runs - 1) / total);
}

// The parts of the tile of steps [s0, s0 + per_tile): runs c0 .. c0 + n - 1.
struct Parts {
  int c0, n;
  const float* first;          // run c0's part at this thread's place
  int64_t skip, next;          // to run c0 + 1's, and from each of those to the next
};
__device__ __forceinline__ Parts parts_of(const float* slots, int64_t slot_floats, int64_t total, int64_t s0, int per_tile,
                                          int runs) {
  Parts p;
  p.c0 = run_of(total, s0, runs);
  p.n = run_of(total, s0 + per_tile - 1, runs) - p.c0 + 1;
  // run c0 may have begun in an earlier tile: this one is its last then
  const int which = run_begin(total, p.c0, runs) < s0 ? 1 : 0;
  p.first = slots + (static_cast<int64_t>(p.c0) * 2 + which) * slot_floats;
  p.skip = (2 - which) * slot_floats;
  p.next = 2 * slot_floats;
  return p;
}
__device__ __forceinline__ float* my_slot(float* slots, int64_t slot_floats, bool first_tile) {
  return slots + (static_cast<int64_t>(blockIdx.x) * 2 + (first_tile ? 0 : 1)) * slot_floats;
}

// Whether all parts but this warp's are counted (one load, acquired).
__device__ __forceinline__ bool others_counted(const uint32_t* counter, int n) {
  uint32_t v = 0;
  if ((threadIdx.x & 31) == 0) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
  const bool all = __shfl_sync(0xFFFFFFFFu, v, 0) == static_cast<uint32_t>(n - 1);
  __syncwarp();                              // the other lanes' reads come after the acquired one
  return all;
}

// Adds the other parts of columns t0 .. t0 + kT - 1 below m to this run's `mine`,
// everything in the order of the runs.
template <int kT>
__device__ __forceinline__ void add_parts(const Parts& p, int me, int t0, int m, float (&mine)[kT]) {
  const float* rest = p.first + p.skip - p.next;
  float sum[kT];
#pragma unroll
  for (int i = 0; i < kT; ++i) sum[i] = 0.0f;
#pragma unroll 1
  for (int c = 0; c < p.n; ++c) {
    if (c == me) {
#pragma unroll
      for (int i = 0; i < kT; ++i) sum[i] += mine[i];
      continue;
    }
    const float* part = (c == 0 ? p.first : rest + c * p.next) + t0 * 128;
    float v[kT];
#pragma unroll
    for (int i = 0; i < kT; ++i) v[i] = t0 + i < m ? __ldcg(part + i * 128) : 0.0f;
#pragma unroll
    for (int i = 0; i < kT; ++i) sum[i] += v[i];
  }
#pragma unroll
  for (int i = 0; i < kT; ++i) mine[i] = sum[i];
}

// Counts this warp's part of a tile (its stores before are visible to whoever
// completes the count); true in the warp that does.
__device__ __forceinline__ bool count_part(uint32_t* counter, int n) {
  __threadfence();
  __syncwarp();
  uint32_t before = 0;
  if ((threadIdx.x & 31) == 0) before = atomicAdd(counter, 1u);
  const bool last = __shfl_sync(0xFFFFFFFFu, before, 0) == static_cast<uint32_t>(n - 1);
  if (last) __threadfence();
  return last;
}

// Sums the parts' columns 0 .. m-1 (128 floats apart), kT columns and kC parts at
// a time, in the order of the runs, and hands on each column's sum.
template <int kT, int kC, typename F>
__device__ __forceinline__ void join_parts(const Parts& p, int m, const F& store) {
  const float* rest = p.first + p.skip - p.next;         // part c >= 1 is at rest + c * next
#pragma unroll 1
  for (int t0 = 0; t0 < m; t0 += kT) {
    float sum[kT];
#pragma unroll
    for (int i = 0; i < kT; ++i) sum[i] = 0.0f;
#pragma unroll 1
    for (int c0 = 0; c0 < p.n; c0 += kC) {
      float v[kC][kT];
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < kT; ++i)
          v[c][i] = c0 + c < p.n && t0 + i < m ? __ldcg((c0 + c == 0 ? p.first : rest + (c0 + c) * p.next) + (t0 + i) * 128)
                                               : 0.0f;
#pragma unroll
      for (int c = 0; c < kC; ++c)
#pragma unroll
        for (int i = 0; i < kT; ++i) sum[i] += v[c][i];
    }
#pragma unroll
    for (int i = 0; i < kT; ++i)
      if (t0 + i < m) store(t0 + i, sum[i]);
  }
}
// Several parts are read at once, more of them the fewer the columns are.
template <typename F>
__device__ __forceinline__ void join_columns(const Parts& p, int m, const F& store) {
  if (m <= 2) join_parts<2, 16>(p, m, store);
  else if (m <= 8) join_parts<8, 4>(p, m, store);
  else join_parts<16, 2>(p, m, store);
}

}  // namespace qlora
