// act.h -- the gated activation's arithmetic.
#pragma once
#include <hip/hip_runtime.h>

namespace sshdp {

// exp(x) for |x| up to 88 (as there further out), to 2 steps of float32: the rounding of
// x log2(e), which would cost |x| / 2 steps, is multiplied back in.
__device__ __forceinline__ float exp_near(float x) {
  x = __builtin_amdgcn_fmed3f(x, -88.f, 88.f);
  constexpr float L = 1.44269504f, l = 1.92596299e-8f;        // log2(e) and what float32 leaves of it
  const float hi = x * L, lo = fmaf(x, l, fmaf(x, L, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return fmaf(e * lo, 0.693147181f, e);
}

// The sigmoid, to 2^-21 of itself; 0 for x under -87, where it leaves float32's normal range.
__device__ __forceinline__ float sigmoid(float x) {
  return x < -87.f ? 0.f : __builtin_amdgcn_rcpf(1.f + exp_near(-x));
}

__device__ __forceinline__ float swiglu(float gate, float up) { return gate * sigmoid(gate) * up; }

}  // namespace sshdp
