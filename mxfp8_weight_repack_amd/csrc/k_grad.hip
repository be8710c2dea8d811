// k_grad.hip -- the global gradient norm over a plan's units, and clipping.
//
//   s = sum of g^2 over every unit element, norm = sqrt(s),
//   coef = max_norm / norm if norm > max_norm, else 1;  out = g * coef.
//
// Two launches: the partial sums (one double per workgroup), and the scaling,
// whose every workgroup first adds the partials up in one fixed order, so no
// atomics, no third launch and the same bits each time.  Squares are formed and
// added in float64: no finite float32 gradient overflows or vanishes, and at 4
// bytes read per element the two float64 operations are far below the memory
// time.  Bound by HBM: 4 bytes read, then 4 read and 4 written per element (5e8 elements:
// 327 us = 6.2 TB/s for the sums, 741 us = 5.4 TB/s for the scaling; a copy reaches 4.8).
// A block of 262400 elements is bound by its two launches: 2.8 and 3.8 us, 11 a call.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"

namespace sshdp {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGradThreads = 256;
// Workgroups of both kernels at most: 8 per CU (256 threads each) fill the CUs'
// wave slots; each takes every gridDim.x-th chunk.
constexpr int64_t kGradGroups = 2048;

// Sum over the workgroup, in lane then wave order; every thread gets it.
__device__ __forceinline__ double group_sum(double v, double *sm) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) sm[w] = v;
  __syncthreads();
  return ((sm[0] + sm[1]) + (sm[2] + sm[3]));
}

__device__ __forceinline__ void add_squares(double &s, const f32x4_t &v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) s = fma((double)v[j], (double)v[j], s);
}

// Elements [base, base + n) split into a head up to a 16-byte boundary, whole
// 16-byte words and a tail (head and tail under 4 elements each).
__device__ __forceinline__ void split4(const GChunk &c, int &head, int &words) {
  head = (int)min<int64_t>((4 - (c.base & 3)) & 3, c.n);
  words = (c.n - head) >> 2;
}

__global__ __launch_bounds__(kGradThreads) void k_grad_partials(const GChunk *chunks, int64_t n, const float *g,
                                                                double *partials) {
  __shared__ double sm[kGradThreads / 64];
  const int t = threadIdx.x;
  double s = 0.0;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const GChunk c = chunks[i];
    int head, words;
    split4(c, head, words);
    const f32x4_t *q = reinterpret_cast<const f32x4_t *>(g + c.base + head);
    f32x4_t v[kChunk / (4 * kGradThreads)];
#pragma unroll
    for (int k = 0; k < kChunk / (4 * kGradThreads); ++k) {
      const int w = t + k * kGradThreads;
      v[k] = w < words ? q[w] : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    if (t < head) {
      const double x = g[c.base + t];
      s = fma(x, x, s);
    }
    const int done = head + 4 * words;
    if (t < c.n - done) {
      const double x = g[c.base + done + t];
      s = fma(x, x, s);
    }
#pragma unroll
    for (int k = 0; k < kChunk / (4 * kGradThreads); ++k) add_squares(s, v[k]);
  }
  s = group_sum(s, sm);
  if (t == 0) partials[blockIdx.x] = s;
}

// The partials' sum: thread t adds parts t, t + 256, ..., then lanes, then waves.
__device__ __forceinline__ double total(const double *parts, int64_t n_parts, double *sm) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n_parts; i += kGradThreads) s += parts[i];
  return group_sum(s, sm);
}

__global__ __launch_bounds__(kGradThreads) void k_grad_total(const double *parts, int64_t n_parts, double *sumsq) {
  __shared__ double sm[kGradThreads / 64];
  const double s = total(parts, n_parts, sm);
  if (threadIdx.x == 0) *sumsq = s;
}

__global__ __launch_bounds__(kGradThreads) void k_grad_scale(const GChunk *chunks, int64_t n, const float *g,
                                                             float *out, const double *parts, int64_t n_parts,
                                                             float max_norm, float *stats) {
  __shared__ double sm[kGradThreads / 64];
  const double norm = sqrt(total(parts, n_parts, sm));
  const float coef = norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.0f;
  const int t = threadIdx.x;
  if (blockIdx.x == 0 && t == 0) {
    stats[0] = (float)norm;
    stats[1] = coef;
  }
  if (coef == 1.0f && out == g) return;              // uniform: nothing to change in place
  // last chunks first: they are what the norm's pass left in the last-level cache
  for (int64_t i = n - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
    const GChunk c = chunks[i];
    int head, words;
    split4(c, head, words);
    const f32x4_t *q = reinterpret_cast<const f32x4_t *>(g + c.base + head);
    f32x4_t *o = reinterpret_cast<f32x4_t *>(out + c.base + head);
    f32x4_t v[kChunk / (4 * kGradThreads)];
#pragma unroll
    for (int k = 0; k < kChunk / (4 * kGradThreads); ++k) {
      const int w = t + k * kGradThreads;
      if (w < words) v[k] = q[w];
    }
#pragma unroll
    for (int k = 0; k < kChunk / (4 * kGradThreads); ++k) {
      const int w = t + k * kGradThreads;
      if (w < words) __builtin_nontemporal_store(f32x4_t{v[k][0] * coef, v[k][1] * coef, v[k][2] * coef, v[k][3] * coef}, o + w);
    }
    if (t < head) out[c.base + t] = g[c.base + t] * coef;
    const int done = head + 4 * words;
    if (t < c.n - done) out[c.base + done + t] = g[c.base + done + t] * coef;
  }
}

unsigned grad_grid(int64_t chunks) { return (unsigned)std::max<int64_t>(1, std::min(chunks, kGradGroups)); }

}  // namespace

int64_t grad_partials(int64_t chunks) { return grad_grid(chunks); }

hipError_t launch_grad_partials(const sshdp_plan &p, const float *g, double *partials, hipStream_t s) {
  const int64_t n = (int64_t)p.gchunks.size();
  hipLaunchKernelGGL(k_grad_partials, dim3(grad_grid(n)), dim3(kGradThreads), 0, s, p.d.gchunks, n, g, partials);
  return hipGetLastError();
}

hipError_t launch_grad_total(const sshdp_plan &p, const double *partials, double *sumsq, hipStream_t s) {
  hipLaunchKernelGGL(k_grad_total, dim3(1), dim3(kGradThreads), 0, s, partials,
                     grad_partials((int64_t)p.gchunks.size()), sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const sshdp_plan &p, const float *g, float *out, const double *parts, int64_t n_parts,
                             float max_norm, float *stats, hipStream_t s) {
  const int64_t n = (int64_t)p.gchunks.size();
  hipLaunchKernelGGL(k_grad_scale, dim3(grad_grid(n)), dim3(kGradThreads), 0, s, p.d.gchunks, n, g, out, parts,
                     n_parts, max_norm, stats);
  return hipGetLastError();
}

}  // namespace sshdp
