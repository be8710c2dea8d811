// k_act.hip -- the gated activation and its gradient, with G along the rows, along the
// columns, or both.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "act.h"
#include "moe.h"
#include "mx_encode.h"

namespace sshdp {
namespace {

// One element's results: the gradients of gate and up, and the activation.
struct Act {
  float dg, du, h;
};
__device__ __forceinline__ Act act_grad(float dh, float g, float u) {
  const float s = sigmoid(g), silu = g * s;
  return {dh * u * (s * fmaf(g, 1.f - s, 1.f)), dh * silu, silu * u};
}

// Rows in use, whatever the offsets hold.
__device__ __forceinline__ int64_t rows_in_use(const sshdp_swiglu_grad &a) {
  return a.offsets ? min((int64_t)max(a.offsets[a.groups], 0), a.rows) : a.rows;
}

__device__ __forceinline__ void put_rows(const sshdp_mx_out &o, const float (&v)[8], int64_t e, bool in, int lane) {
  if (!o.codes) return;
  uint32_t sb;
  const u32x2_t c = mx_codes4(v, sb);
  if (!in) return;
  *reinterpret_cast<u32x2_t *>(o.codes + e) = c;
  if ((lane & 3) == 0) o.scales[e >> 5] = (uint8_t)sb;
}

// One column's 4 blocks by 4 lanes, from element e on.
__device__ __forceinline__ void put_column(const sshdp_mx_out &o, const float (&v)[32], int64_t e, int blocks, int lane) {
  const MxColumn c = mx_column(v);
  mx_store_column(c, o.codes_t + e, blocks, lane);
  if ((lane & 3) < blocks) o.scales_t[(e >> 5) + (lane & 3)] = (uint8_t)c.scale;
}

// Along the rows alone: 8 elements a lane.  Bound by HBM: dgate and dup of 24576 x 1408 42 us, 6.7
// TB/s (by the tiles below 47; 6 x 704 2.9 and 4.4).
__global__ __launch_bounds__(256) void k_act_rows(sshdp_swiglu_grad a) {
  const int64_t runs = rows_in_use(a) * (a.cols >> 3);   // a multiple of 4: a block's lanes leave together
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < runs; i += (int64_t)gridDim.x * 256) {
    float d[8] = {}, g[8], u[8], dg[8], du[8], h[8];
    if (a.dh) unpack8<true>(load8<true>(a.dh, i * 8), d);
    unpack8<true>(load8<true>(a.gate, i * 8), g);
    unpack8<true>(load8<true>(a.up, i * 8), u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Act r = act_grad(d[j], g[j], u[j]);
      dg[j] = r.dg;
      du[j] = r.du;
      h[j] = r.h;
    }
    put_rows(a.dgate, dg, i * 8, true, threadIdx.x);
    put_rows(a.dup, du, i * 8, true, threadIdx.x);
    put_rows(a.h, h, i * 8, true, threadIdx.x);
  }
}

constexpr int kActRows = 128, kActCols = 64;         // tile of one workgroup

// Columns too: a lane computes 16 elements of 2 rows, stores their codes (the scales of the two
// in one store) and keeps the three results; one result after the other goes through LDS, from
// which a lane takes 32 rows of one column.  LDS columns are rotated by the row group, so the 4
// groups that a wave reads at one step fall on different banks.  Tiles go along the rows, all
// XCDs side by side: 24558 x 1408, all ten outputs, 95 to 97 us, 4.0 TB/s (79 back to back, part
// of the inputs still in the last-level cache), each XCD in an eighth of the rows 107; two or four
// neighbouring tiles on an XCD, and ordinary stores in place of nontemporal ones, change nothing.
// Bound by HBM and by the number of store instructions: with 8 elements a lane and a store for
// each row's scales 102 to 111 us.
__global__ __launch_bounds__(256) void k_act_tiles(sshdp_swiglu_grad a, uint32_t tiles_c) {
  constexpr int NP = kActRows / 64;
  __shared__ __align__(16) float sm[kActRows][kActCols];
  const int t = threadIdx.x;
  const int64_t r0 = blockIdx.x / tiles_c * (int64_t)kActRows, c0 = blockIdx.x % tiles_c * (int64_t)kActCols;
  const int64_t used = rows_in_use(a);
  if (r0 >= used) return;
  const int lc = (t & 3) * 16, lr = t >> 2;
  const bool in_c = c0 + lc < a.cols;
  const void *src[3] = {a.dh, a.gate, a.up};
  Raw8<true> raw[NP][3][2];
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int64_t r = r0 + lr + 64 * p;
      raw[p][k][0] = raw[p][k][1] = Raw8<true>{};
      if (in_c && r < used && src[k]) {
        raw[p][k][0] = load8<true>(src[k], r * a.cols + c0 + lc);
        raw[p][k][1] = load8<true>(src[k], r * a.cols + c0 + lc + 8);
      }
    }
  const sshdp_mx_out *out[3] = {&a.dgate, &a.dup, &a.h};
  float v[3][NP][16];                                // dgate, dup, h
  uint32_t sbs[3] = {0, 0, 0};                       // lane p of 4: the scales of its row of pass p
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float d[8], g[8], u[8];
      unpack8<true>(raw[p][0][h], d);
      unpack8<true>(raw[p][1][h], g);
      unpack8<true>(raw[p][2][h], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Act r = act_grad(d[j], g[j], u[j]);
        v[0][p][8 * h + j] = r.dg;
        v[1][p][8 * h + j] = r.du;
        v[2][p][8 * h + j] = r.h;
      }
    }
    const int rr = lr + 64 * p;
    const int64_t e = (r0 + rr) * a.cols + c0 + lc;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (!out[k]->codes) continue;
      uint32_t sb;
      const u32x4r_t x = mx_codes2(v[k][p], sb);
      if (in_c && r0 + rr < used) __builtin_nontemporal_store(x, reinterpret_cast<u32x4r_t *>(out[k]->codes + e));
      // the row's two scale bytes, in all of its 4 lanes
      uint32_t q = sb << (8 * ((t & 3) >> 1));
      q |= (uint32_t)__builtin_amdgcn_mov_dpp((int)q, 0x4E, 0xF, 0xF, true);      // quad_perm [2, 3, 0, 1]
      if ((t & 3) == p) sbs[k] = q;
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    typedef uint16_t u16u_t __attribute__((aligned(1)));
    const int64_t r = r0 + lr + 64 * (t & 3);
    if (!out[k]->codes || (t & 3) >= NP || r >= used) continue;
    uint8_t *d = out[k]->scales + r * (a.cols >> 5) + (c0 >> 5);
    if (c0 + 32 < a.cols) *reinterpret_cast<u16u_t *>(d) = (uint16_t)sbs[k];
    else *d = (uint8_t)sbs[k];
  }
  const int grp = t & 3, c = t >> 2;
  const int64_t e = (c0 + c) * a.rows + r0;
  const int blocks = (int)min<int64_t>(4, (used - r0 + 31) / 32);
  bool first = true;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (!out[k]->codes_t) continue;
    if (!first) __syncthreads();                     // the one before has been read
    first = false;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int rr = lr + 64 * p;
      float4 *q = reinterpret_cast<float4 *>(&sm[rr][lc ^ (16 * (rr >> 5))]);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = make_float4(v[k][p][4 * i], v[k][p][4 * i + 1], v[k][p][4 * i + 2], v[k][p][4 * i + 3]);
    }
    __syncthreads();
    if (c0 + c >= a.cols) continue;
    float x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = sm[32 * grp + j][c ^ (16 * grp)];
    put_column(*out[k], x, e, blocks, t);
  }
}

}  // namespace

hipError_t launch_swiglu_grad(const sshdp_swiglu_grad &a, hipStream_t s) {
  if (a.dgate.codes_t || a.dup.codes_t || a.h.codes_t) {
    const int64_t tc = (a.cols + kActCols - 1) / kActCols, tr = (a.rows + kActRows - 1) / kActRows;
    hipLaunchKernelGGL(k_act_tiles, dim3((unsigned)(tr * tc)), dim3(256), 0, s, a, (uint32_t)tc);
  } else {
    const int64_t runs = a.rows * (a.cols / 8);
    hipLaunchKernelGGL(k_act_rows, dim3((unsigned)std::min<int64_t>((runs + 255) / 256, 1 << 20)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace sshdp
