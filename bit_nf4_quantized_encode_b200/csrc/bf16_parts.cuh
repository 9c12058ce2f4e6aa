// bf16_parts.cuh -- a float as the sum of two bf16 numbers (sm_100a): what a bf16
// product takes instead of a rounded operand where eight bits would show.
#pragma once
#include <cuda_bf16.h>

namespace qlora {

struct BfParts {
  float first, second;
};
// v rounded to bf16 and what that leaves out, rounded too: for v in [1, 2) the
// first is off by 2^-8 at most, so the second by 2^-17.  Nothing is left out of an
// infinity or a NaN (inf - inf would make one of the other).
__device__ __forceinline__ BfParts bf16_parts(float v) {
  BfParts p;
  p.first = __bfloat162float(__float2bfloat16_rn(v));
  const float left = __fsub_rn(v, p.first);
  p.second = (__float_as_uint(p.first) & 0x7F800000u) == 0x7F800000u ? 0.0f : __bfloat162float(__float2bfloat16_rn(left));
  return p;
}
// The bits of a bf16 value.
__device__ __forceinline__ uint16_t bf16_bits(float v) { return static_cast<uint16_t>(__float_as_uint(v) >> 16); }

}  // namespace qlora
