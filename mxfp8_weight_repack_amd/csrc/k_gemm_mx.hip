// k_gemm_mx.hip -- MXFP8 products on gfx950's matrix cores.
//
//   out[m][n] = sum over blocks kb of 2^(ea(m, kb) + eb(n, kb)) * sum over the
//   block's 32 k of a(m, k) b(n, k)   (+ addend[m][n]),
//
// a, b E4M3 values, ea, eb the blocks' E8M0 exponents.
//
// bfloat16 output: v_mfma_scale_f32_16x16x128_f8f6f4 (16 x 16 outputs, 128 k, i.e.
// 4 blocks) takes codes and exponent bytes as they lie in memory.  It adds each 8
// consecutive k's products in fixed point, cut off at 2^-14 of their largest
// (measured: about 1.4e-5 of the result, rms), and those sums in float32: far
// below bfloat16's half step of 2^-9 to 2^-8, but not a float32 sum.  So float32
// output converts the codes, scale included and exactly, to bfloat16
// (v_cvt_scalef32_pk_bf16_fp8: 4 significant bits, and bfloat16 has float32's
// exponents) and uses v_mfma_f32_16x16x32_bf16, whose sums are float32's (measured
// 5e-9 to 1.2e-7), at half the matrix rate.
//
// Operand layout, lane l = 16 g + r: row (or column) r of the 16.  The 8-bit
// instruction takes the lane's 16-byte chunks g and 4 + g of the 128 k, and for its
// scale the byte of block g.  The bfloat16 form uses the same chunks, 8 bytes per
// instruction: which 8 k they are does not matter as long as both operands agree.
// Chunk g lies in block g / 2, chunk 4 + g in block 2 + g / 2.  The result holds
// rows 4 g + 0..3 of column r.  The first operand is B (n) and the second A (m), so
// a lane ends up with 4 consecutive n of one m.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"

namespace sshdp {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// Index of the scale byte of row `r`'s block kb in a matrix with KB blocks a row.
__device__ __forceinline__ int64_t scale_index(int layout, int64_t r, int64_t kb, int64_t KB) {
  if (layout == SSHDP_SCALE_ROWMAJOR) return r * KB + kb;
  if (layout == SSHDP_SCALE_TILE32X4) return ((r >> 5) * (KB >> 2) + (kb >> 2)) * 128 + (r & 31) * 4 + (kb & 3);
  return (r >> 5) * KB + kb;
}

// 8 codes (two words) times 2^(byte - 127), as bfloat16, exact.  The conversion reads
// the scale's exponent bits, so byte << 23 is E8M0 from 2^-127 (0) to NaN (255).
__device__ __forceinline__ bf16x8_t to_bf16(int w0, int w1, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  bf16x2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true)};
  return __builtin_bit_cast(bf16x8_t, v);
}

// One wave, one 16 x 16 block of the output, operands straight from memory.
template <bool NN, bool BF16>
__global__ __launch_bounds__(64) void k_gemm_mx_16(GemmMx p, int64_t tiles_n) {
  const int l = threadIdx.x, r = l & 15, g = l >> 4;
  const int64_t m = blockIdx.x / tiles_n * 16 + r, n = blockIdx.x % tiles_n * 16 + r;
  const bool in_m = m < p.m, in_n = n < p.n;
  const int64_t KB = p.k >> 5;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k0 = 0; k0 < p.k; k0 += 128) {
    i32x8_t a = {0, 0, 0, 0, 0, 0, 0, 0}, b = a;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = k0 + 64 * h + 16 * g;          // K % 32 == 0: a chunk is in or out as a whole
      if (k < p.k && in_m) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(p.a + m * p.k + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[4 * h + j] = (int)v[j];
      }
      if (k < p.k && in_n) {
        if (NN) {
#pragma unroll
          for (int j = 0; j < 16; ++j) b[4 * h + (j >> 2)] |= (int)p.b[(k + j) * p.n + n] << (8 * (j & 3));
        } else {
          const u32x4_t v = *reinterpret_cast<const u32x4_t *>(p.b + n * p.k + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) b[4 * h + j] = (int)v[j];
        }
      }
    }
    auto scale_a = [&](int64_t kb) -> int {            // 2^-127 beside codes that are all zero
      return kb < KB && in_m ? p.as[scale_index(p.la, m, kb, KB)] : 0;
    };
    auto scale_b = [&](int64_t kb) -> int {
      if (!(kb < KB && in_n)) return 0;
      return NN ? p.bs[kb * (p.n >> 5) + (n >> 5)] : p.bs[scale_index(p.lb, n, kb, KB)];
    };
    const int64_t kb = k0 >> 5;
    if (BF16) {
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, acc, 0, 0, 0, scale_b(kb + g), 0, scale_a(kb + g));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int sa = scale_a(kb + 2 * h + (g >> 1)), sb = scale_b(kb + 2 * h + (g >> 1));
#pragma unroll
        for (int j = 4 * h; j < 4 * h + 4; j += 2)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(to_bf16(b[j], b[j + 1], sb), to_bf16(a[j], a[j + 1], sa), acc,
                                                        0, 0, 0);
      }
    }
  }
  // every lane takes part in the matrix instructions: none may sink below the branch
  asm volatile("" : "+v"(acc));
  const int64_t n0 = blockIdx.x % tiles_n * 16 + 4 * g;
  if (!in_m) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n0 + j >= p.n) break;
    const int64_t e = m * p.ld + n0 + j;
    float v = acc[j];
    if (p.addend) v += p.addend[e];
    if (BF16) static_cast<uint16_t *>(p.out)[e] = (uint16_t)pk_bf16(v, 0.f);
    else static_cast<float *>(p.out)[e] = v;
  }
}

}  // namespace

int64_t gemm_mx_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_gemm_mx(const GemmMx &g, void *, hipStream_t s) {
  const int64_t tm = (g.m + 15) / 16, tn = (g.n + 15) / 16;
  const dim3 grid((unsigned)(tm * tn)), block(64);
  if (g.nn && g.bf16) hipLaunchKernelGGL((k_gemm_mx_16<true, true>), grid, block, 0, s, g, tn);
  else if (g.nn) hipLaunchKernelGGL((k_gemm_mx_16<true, false>), grid, block, 0, s, g, tn);
  else if (g.bf16) hipLaunchKernelGGL((k_gemm_mx_16<false, true>), grid, block, 0, s, g, tn);
  else hipLaunchKernelGGL((k_gemm_mx_16<false, false>), grid, block, 0, s, g, tn);
  return hipGetLastError();
}

}  // namespace sshdp
