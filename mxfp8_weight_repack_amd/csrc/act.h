// act.h -- the gated activation's arithmetic.
#pragma once
#include <hip/hip_runtime.h>

namespace sshdp {

// The sigmoid: off by at most (1.25 |x| + 6) 2^-24 of itself for x under 0 (the rounding of the
// exponent x log2(e) and of log2(e) grow with x: 1.23 of them), 2^-21 over it; 0 from about -88
// on, where it leaves float32's normal range.  Four instructions: a gated tile has 32 of them
// a lane at its end.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

__device__ __forceinline__ float swiglu(float gate, float up) { return gate * sigmoid(gate) * up; }

}  // namespace sshdp
