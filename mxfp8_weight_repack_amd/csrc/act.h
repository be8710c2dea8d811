// act.h -- the gated activation's arithmetic.
#pragma once
#include <hip/hip_runtime.h>

namespace sshdp {

// ln 2^-126: under it the sigmoid leaves float32's normal range.
constexpr float kSigmoidLeast = -87.3365f;

// The sigmoid: off by at most (1.25 |x| + 6) 2^-24 of itself for x under 0 (the rounding of the
// exponent x log2(e) and of log2(e) grow with x: 1.23 of them), 2^-21 over it, as long as it is a
// normal float32 number: under kSigmoidLeast it is less than 2^-126, or 0.  Four instructions: a
// gated tile has 32 (of 128 rows) or 64 (of 256) of them a lane at its end, and its sums are not
// nearer than that.
__device__ __forceinline__ float sigmoid_near(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// The same within 2^-21 down to there, and 0 below: what the exponent's rounding and log2(e)'s
// leave out is multiplied back in.  For where memory is what takes the time.
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float L = 1.44269504f, l = 1.92596299e-8f;        // log2(e) and what float32 leaves of it
  const float y = __builtin_amdgcn_fmed3f(-x, -88.f, 88.f), hi = y * L, lo = fmaf(y, l, fmaf(y, L, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return x < kSigmoidLeast ? 0.f : __builtin_amdgcn_rcpf(1.f + fmaf(e * lo, 0.693147181f, e));
}

}  // namespace sshdp
