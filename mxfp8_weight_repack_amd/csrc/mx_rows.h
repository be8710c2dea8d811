// mx_rows.h -- pieces shared by the kernels that quantise rows 8 elements per lane.
//
// A lane owns 8 consecutive elements (one or two 16-byte loads, one 8-byte store
// of codes) and 4 consecutive lanes, aligned to 4, one 32-element MX block.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace sshdp {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4r_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2r_t __attribute__((ext_vector_type(2)));
typedef float f32x2r_t __attribute__((ext_vector_type(2)));

// 8 consecutive elements at element index i of a float32 or bfloat16 array.
template <bool BF16>
struct Raw8;
template <>
struct Raw8<true> {
  u32x4r_t w;
};
template <>
struct Raw8<false> {
  u32x4r_t w[2];
};

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void *p, int64_t i) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.w = *reinterpret_cast<const u32x4r_t *>(static_cast<const uint16_t *>(p) + i);
  } else {
    const u32x4r_t *q = reinterpret_cast<const u32x4r_t *>(static_cast<const float *>(p) + i);
    r.w[0] = q[0];
    r.w[1] = q[1];
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw8<BF16> &r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16) {
      v[2 * j] = __uint_as_float(r.w[j] << 16);
      v[2 * j + 1] = __uint_as_float(r.w[j] & 0xFFFF0000u);
    } else {
      v[j] = __uint_as_float(r.w[0][j]);
      v[4 + j] = __uint_as_float(r.w[1][j]);
    }
  }
}

// To the array's type, bfloat16 by round to nearest even.
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> pack8(const float (&v)[8]) {
  Raw8<BF16> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (BF16) {
      r.w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2r_t{v[2 * j], v[2 * j + 1]}, bf16x2r_t));
    } else {
      r.w[0][j] = __float_as_uint(v[j]);
      r.w[1][j] = __float_as_uint(v[4 + j]);
    }
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t i, const Raw8<BF16> &r) {
  if constexpr (BF16) {
    __builtin_nontemporal_store(r.w, reinterpret_cast<u32x4r_t *>(static_cast<uint16_t *>(p) + i));
  } else {
    u32x4r_t *q = reinterpret_cast<u32x4r_t *>(static_cast<float *>(p) + i);
    __builtin_nontemporal_store(r.w[0], q);
    __builtin_nontemporal_store(r.w[1], q + 1);
  }
}

// Largest |x| bit pattern of the 4 aligned lanes' 8 elements each (NaN above Inf).
// Every lane of the wave must call it.
__device__ __forceinline__ uint32_t mx_amax4(const float (&v)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  a = max(a, (uint32_t)__shfl_xor((int)a, 1));
  a = max(a, (uint32_t)__shfl_xor((int)a, 2));
  return a;
}

// The 8 E4M3FN codes of v under scale byte sb.
__device__ __forceinline__ u32x2_t mx_encode8(const float (&v)[8], uint32_t sb) {
  return u32x2_t{mx_encode4(make_float4(v[0], v[1], v[2], v[3]), sb),
                 mx_encode4(make_float4(v[4], v[5], v[6], v[7]), sb)};
}

}  // namespace sshdp
