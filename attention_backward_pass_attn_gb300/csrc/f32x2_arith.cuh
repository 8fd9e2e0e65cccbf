// f32x2_arith.cuh -- the packed product and sum beside f32x2.cuh's multiply-add.
// A header of its own: the plain attention kernels include that one, and need
// neither.
#pragma once

#include "f32x2.cuh"

namespace attn {

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace attn
