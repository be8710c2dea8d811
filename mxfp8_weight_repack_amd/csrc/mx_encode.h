// mx_encode.h -- G of values in registers by the scaled conversions of gfx950, which divide by the
// scale on the way (one instruction for two codes; tested against the codes' definition for every
// bfloat16 value under each of the 248 scales that a block may have, and for float32 values at,
// beside and between the rounding borders under each).
#pragma once
#include <hip/hip_runtime.h>

#include "mx_rows.h"

namespace sshdp {

typedef short i16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// 4 codes of float32 values; `scale` has the block's exponent.
__device__ __forceinline__ uint32_t mx_cvt4(float a, float b, float c, float d, float scale) {
  i16x2_t o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, a, b, scale, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, o);
}

// 4 codes of two words of bfloat16 pairs.
__device__ __forceinline__ uint32_t mx_cvt4_bf16(uint32_t p, uint32_t q, float scale) {
  i16x2_t o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2r_t, p), scale, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2r_t, q), scale, true);
  return __builtin_bit_cast(uint32_t, o);
}

__device__ __forceinline__ float mx_scale_float(uint32_t sb) { return __uint_as_float(sb << 23); }

// Codes in a block holding NaN or infinity are all 0x7F.
__device__ __forceinline__ uint32_t mx_or_nan(uint32_t codes, uint32_t sb) { return sb == 0xFFu ? 0x7F7F7F7Fu : codes; }

// A lane's 8 codes and its block's scale byte, 4 aligned lanes a block.  Every lane of the
// wave must call it.
__device__ __forceinline__ u32x2_t mx_codes4(const float (&v)[8], uint32_t &sb) {
  sb = mx_scale_byte(mx_amax4(v));
  const float s = mx_scale_float(sb);
  return u32x2_t{mx_or_nan(mx_cvt4(v[0], v[1], v[2], v[3], s), sb), mx_or_nan(mx_cvt4(v[4], v[5], v[6], v[7], s), sb)};
}

// The larger magnitudes of two words of bfloat16 pairs, half by half (`m` has no signs).
__device__ __forceinline__ uint32_t mx_max_bf16(uint32_t m, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m),
                                                                __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu)));
}

// The same of 8 elements as loaded.
template <bool BF16>
__device__ __forceinline__ u32x2_t mx_codes4_raw(const Raw8<BF16> &r, uint32_t &sb) {
  if constexpr (BF16) {
    uint32_t m = mx_max_bf16(mx_max_bf16(mx_max_bf16(r.w[0] & 0x7FFF7FFFu, r.w[1]), r.w[2]), r.w[3]);
    uint32_t a = max(m << 16, m & 0xFFFF0000u);
    a = max(a, (uint32_t)__shfl_xor((int)a, 1));
    a = max(a, (uint32_t)__shfl_xor((int)a, 2));
    sb = mx_scale_byte(a);
    const float s = mx_scale_float(sb);
    return u32x2_t{mx_or_nan(mx_cvt4_bf16(r.w[0], r.w[1], s), sb), mx_or_nan(mx_cvt4_bf16(r.w[2], r.w[3], s), sb)};
  } else {
    float v[8];
    unpack8<BF16>(r, v);
    return mx_codes4(v, sb);
  }
}

// 16 codes of a lane's 16 elements and its block's scale byte, 2 aligned lanes a block.  Every
// lane of the wave must call it.
__device__ __forceinline__ u32x4r_t mx_codes2(const float (&v)[16], uint32_t &sb) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));      // quad_perm [1, 0, 3, 2]
  sb = mx_scale_byte(a);
  const float s = mx_scale_float(sb);
  u32x4r_t c;
#pragma unroll
  for (int j = 0; j < 4; ++j) c[j] = mx_or_nan(mx_cvt4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s), sb);
  return c;
}

// The same of 16 elements as loaded.
template <bool BF16>
__device__ __forceinline__ u32x4r_t mx_codes2_raw(const Raw8<BF16> (&r)[2], uint32_t &sb) {
  if constexpr (BF16) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = mx_max_bf16(m, r[j >> 2].w[j & 3]);
    uint32_t a = max(m << 16, m & 0xFFFF0000u);
    a = max(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));
    sb = mx_scale_byte(a);
    const float s = mx_scale_float(sb);
    u32x4r_t c;
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = mx_or_nan(mx_cvt4_bf16(r[j >> 1].w[2 * (j & 1)], r[j >> 1].w[2 * (j & 1) + 1], s), sb);
    return c;
  } else {
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      unpack8<BF16>(r[h], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[8 * h + j] = x[j];
    }
    return mx_codes2(v, sb);
  }
}

// One block's 32 codes that a lane holds alone.
struct MxColumn {
  u32x4r_t codes[2];
  uint32_t scale;
};

__device__ __forceinline__ MxColumn mx_column(const float (&v)[32]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  MxColumn o;
  o.scale = mx_scale_byte(m);
  const float s = mx_scale_float(o.scale);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    o.codes[j >> 2][j & 3] = mx_or_nan(mx_cvt4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], s), o.scale);
  return o;
}

// Two neighbouring columns' blocks, a word the two columns' bfloat16 of a row.
__device__ __forceinline__ void mx_columns_bf16(const uint32_t (&x)[32], MxColumn (&o)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = mx_max_bf16(m, x[j]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    o[h].scale = mx_scale_byte(h ? m & 0xFFFF0000u : m << 16);
    const float s = mx_scale_float(o[h].scale);
    const uint32_t pick = h ? 0x07060302u : 0x05040100u;     // rows j and j + 1 of one column
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t p = __builtin_amdgcn_perm(x[4 * j + 1], x[4 * j], pick), q = __builtin_amdgcn_perm(x[4 * j + 3], x[4 * j + 2], pick);
      o[h].codes[j >> 2][j & 3] = mx_or_nan(mx_cvt4_bf16(p, q, s), o[h].scale);
    }
  }
}

// Two 16-byte chunks a lane, 32 bytes apart from lane to lane, exchanged within 4 aligned lanes
// so that each of two stores writes 64 bytes in a row: store k takes the chunks of the lanes
// 2 k and 2 k + 1, and chunk lane & 3 of them.  Every lane of the four must call it.
__device__ __forceinline__ void mx_in_runs(const u32x4r_t &lo, const u32x4r_t &hi, int lane, u32x4r_t (&w)[2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // quad_perm [0, 0, 1, 1] and [2, 2, 3, 3]: two lanes a source, one a half
    const int a0 = __builtin_amdgcn_mov_dpp((int)lo[j], 0x50, 0xF, 0xF, true), a1 = __builtin_amdgcn_mov_dpp((int)hi[j], 0x50, 0xF, 0xF, true);
    const int b0 = __builtin_amdgcn_mov_dpp((int)lo[j], 0xFA, 0xF, 0xF, true), b1 = __builtin_amdgcn_mov_dpp((int)hi[j], 0xFA, 0xF, 0xF, true);
    w[0][j] = (uint32_t)(lane & 1 ? a1 : a0);
    w[1][j] = (uint32_t)(lane & 1 ? b1 : b0);
  }
}

// A column's 128 rows of codes from the 4 lanes (aligned to 4) that hold its 4 blocks: lane l's
// is block l (stored lane by lane the gradients' 26624 x 1408 columns took 18 us each, in runs
// 11).  `at`: block 0's place; `blocks`: how many of the 4 are stored.
__device__ __forceinline__ void mx_store_column(const MxColumn &c, uint8_t *at, int blocks, int lane) {
  const int l = lane & 3;
  u32x4r_t w[2];
  mx_in_runs(c.codes[0], c.codes[1], l, w);
  u32x4r_t *d = reinterpret_cast<u32x4r_t *>(at + 16 * l);
  if ((l >> 1) < blocks) __builtin_nontemporal_store(w[0], d);
  if (2 + (l >> 1) < blocks) __builtin_nontemporal_store(w[1], d + 4);
}

}  // namespace sshdp
