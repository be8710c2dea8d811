// k_rows.hip -- MXFP8 quantisation of any matrix (along rows, along columns, or
// both), and the residual RMS norm with MXFP8 output and its gradient.
//
// All of them are bound by HBM: each element is read once and each result
// written once, in 16-byte loads and 8- or 16-byte stores.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx_rows.h"

namespace sshdp {
namespace {

// ------------------------------------------------------------------ along rows

// 16384 x 8192: bfloat16 74 us = 5.4 TB/s, float32 115 us = 5.8 TB/s.
// One 8-element run per lane; a row is cols / 8 runs and 4 of them one block, so
// runs of all rows are numbered through and blocks never leave their 4 lanes.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quant_rows(const void *src, int64_t runs, int runs_per_row, int64_t ld,
                                                    uint8_t *codes, uint8_t *scales) {
  // `runs` is a multiple of 4, so a block's lanes leave the loop together and the
  // shuffles of the others never need them
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < runs; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / runs_per_row;
    const int64_t at = row * ld + (i - row * runs_per_row) * 8;
    float v[8];
    unpack8<BF16>(load8<BF16>(src, at), v);
    const uint32_t sb = mx_scale_byte(mx_amax4(v));
    *reinterpret_cast<u32x2_t *>(codes + i * 8) = mx_encode8(v, sb);
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)sb;
  }
}

// --------------------------------------------------- along columns, or both ways

constexpr int kQtRows = 128, kQtCols = 128;          // tile of one workgroup

// A 128 x 128 tile goes through LDS in src's own type.  Reading it: a row's 128 elements
// are 16 lanes' 8 each (full 256- or 512-byte lines).  Along columns a lane then takes two
// neighbouring columns' 32 rows, one LDS read a row, so a block is one lane's and needs no
// exchange; 4 consecutive lanes take the 4 row groups of a column pair, i.e. 128
// consecutive bytes of codes_t.  LDS columns are rotated by the row group (element (r, c)
// sits at column c ^ S * (r / 32), S = 32 of bfloat16 or 16 of float32), so the 4 groups
// that a wave reads at one step fall on different banks.  Rows past the end count as zeros.
// Both ways of 4093 x 8192 bfloat16: 28 us = 5.2 TB/s; columns of 8192 x 2048 float32: 19 us
// = 4.4 TB/s, of which a copy's time is 17.5.
template <bool BF16, bool ROWS>
__global__ __launch_bounds__(256) void k_quant_tiles(const void *src, int64_t rows, int64_t cols, int64_t ld,
                                                     uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                                     uint8_t *scales_t, int64_t tiles_c) {
  constexpr int ES = BF16 ? 2 : 4, ROT = BF16 ? 32 : 16;
  __shared__ __align__(16) char sm[kQtRows * kQtCols * ES];
  const int t = threadIdx.x;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = tr * kQtRows, c0 = tc * kQtCols;
  const int lc = (t & 15) * 8, lr = t >> 4;
  const bool in_c = c0 + lc < cols;                   // cols % 32 == 0: whole blocks in or out
  Raw8<BF16> raw[kQtRows / 16];
#pragma unroll
  for (int p = 0; p < kQtRows / 16; ++p) {
    const int64_t r = r0 + lr + 16 * p;
    raw[p] = Raw8<BF16>{};
    if (in_c && r < rows) raw[p] = load8<BF16>(src, r * ld + c0 + lc);
  }
#pragma unroll
  for (int p = 0; p < kQtRows / 16; ++p) {
    const int rr = lr + 16 * p;
    *reinterpret_cast<Raw8<BF16> *>(sm + (rr * kQtCols + (lc ^ ((rr >> 5) * ROT))) * ES) = raw[p];
    if (ROWS) {
      float v[8];
      unpack8<BF16>(raw[p], v);
      const uint32_t sb = mx_scale_byte(mx_amax4(v));
      if (in_c && r0 + rr < rows) {
        const int64_t e = (r0 + rr) * cols + c0 + lc;
        *reinterpret_cast<u32x2_t *>(codes + e) = mx_encode8(v, sb);
        if ((t & 3) == 0) scales[e >> 5] = (uint8_t)sb;
      }
    }
  }
  __syncthreads();
  const int64_t rp = (rows + 31) / 32 * 32;
  const int grp = t & 3, c = (t >> 2) * 2;
  const int64_t r = r0 + 32 * grp;
  if (c0 + c >= cols || r >= rp) return;
  const char *q = sm + (32 * grp * kQtCols + (c ^ (grp * ROT))) * ES;
  float v[2][32];
  uint32_t a[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (BF16) {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(q + j * kQtCols * ES);
      v[0][j] = __uint_as_float(w << 16);
      v[1][j] = __uint_as_float(w & 0xFFFF0000u);
    } else {
      const float2 w = *reinterpret_cast<const float2 *>(q + j * kQtCols * ES);
      v[0][j] = w.x;
      v[1][j] = w.y;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) a[h] = max(a[h], __float_as_uint(v[h][j]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t sb = mx_scale_byte(a[h]);
    u32x4r_t w[2];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j >> 2][j & 3] = mx_encode4(make_float4(v[h][4 * j], v[h][4 * j + 1], v[h][4 * j + 2], v[h][4 * j + 3]), sb);
    if (sb == 0xFFu && r + 32 > rows) {               // the missing rows' codes stay 0 in a NaN block too
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (r + j >= rows) w[j >> 4][(j >> 2) & 3] &= ~(0xFFu << (8 * (j & 3)));
    }
    const int64_t e = (c0 + c + h) * rp + r;
    u32x4r_t *o = reinterpret_cast<u32x4r_t *>(codes_t + e);
    o[0] = w[0];
    o[1] = w[1];
    scales_t[e >> 5] = (uint8_t)sb;
  }
}

// -------------------------------------------------------------- residual RMS norm

// Row layout of the norm kernels: WPR waves share a row, lane l of wave w holds
// the 8-element runs w * 64 + l + c * WPR * 64, c < NCH.  Rows of up to 512 * NCH
// elements take one wave, so a workgroup of 4 waves needs no barrier at all.
template <int WPR, int NCH>
struct RowCfg {
  static constexpr int kWpr = WPR, kNch = NCH;
  static constexpr int kThreads = WPR > 4 ? 64 * WPR : 256;
  static constexpr int kRows = kThreads / 64 / WPR;    // rows a workgroup works on at once
  // 16 waves leave a lane 128 registers: with more than 16 values of a row in them, the
  // weights and dh are read anew for each row, from the caches, and the weight gradient's
  // sums are held in LDS (4096 x 32768 bfloat16: 230 us, gradient 280; all of it in
  // registers, and spilled, 299 and 552)
  static constexpr bool kLean = WPR * NCH > 32;
};

// Run `run`'s 8 weights, 0 past the end.  They lie at any element (a norm unit's place in a
// root), so the words have an element's alignment.
template <bool WBF16>
__device__ __forceinline__ void weights(const void *weight, int run, int runs, float (&w)[8]) {
  typedef uint32_t u32x4h_t __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t u32x4w_t __attribute__((ext_vector_type(4), aligned(4)));
  Raw8<WBF16> r{};
  if (run < runs) {
    if constexpr (WBF16) {
      r.w = *reinterpret_cast<const u32x4h_t *>(static_cast<const uint16_t *>(weight) + run * 8);
    } else {
      const u32x4w_t *q = reinterpret_cast<const u32x4w_t *>(static_cast<const float *>(weight) + run * 8);
      r.w[0] = q[0];
      r.w[1] = q[1];
    }
  }
  unpack8<WBF16>(r, w);
}

// Sum over a row's lanes: a butterfly in the wave, then the waves in order.
template <int WPR>
__device__ __forceinline__ double row_sum(double v, double *sm) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if (WPR > 1) {
    const int w = threadIdx.x >> 6, first = w / WPR * WPR;
    __syncthreads();                                   // the previous row's sums have been read
    if ((threadIdx.x & 63) == 0) sm[w] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int k = 0; k < WPR; ++k) v += sm[first + k];
  }
  return v;
}

// Bound by HBM: 8191 x 8192 bfloat16 with residual, h, y and codes 104 us = 5.8 TB/s.  One row is
// bound by the launch: 4.4 us, 9 a call.  The row is held between the two passes over it;
// its sum and y's products are in float64 (what the codes' bits rest on), far below the
// memory time.
template <bool BF16, bool WBF16, class C>
__global__ __launch_bounds__(C::kThreads) void k_rmsnorm(sshdp_rmsnorm a) {
  __shared__ double sm[C::kThreads / 64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int sub = wave / C::kWpr, run0 = (wave % C::kWpr) * 64 + lane;
  const int runs = (int)(a.cols >> 3);
  float w[C::kNch][8];
  if (!C::kLean) {
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) weights<WBF16>(a.weight, run0 + c * C::kWpr * 64, runs, w[c]);
  }
  // the loop bound is the same for all waves of a workgroup (barriers inside)
  for (int64_t g = blockIdx.x; g * C::kRows < a.rows; g += gridDim.x) {
    const int64_t row = g * C::kRows + sub;
    const bool live = row < a.rows;
    float h[C::kNch][8];
    double s = 0.0;
    Raw8<BF16> rx[C::kNch], rr[C::kNch];
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      const int run = run0 + c * C::kWpr * 64;
      rx[c] = Raw8<BF16>{};
      rr[c] = Raw8<BF16>{};
      if (live && run < runs) {
        rx[c] = load8<BF16>(a.x, row * a.ld_x + run * 8);
        if (a.residual) rr[c] = load8<BF16>(a.residual, row * a.ld_residual + run * 8);
      }
    }
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      const int run = run0 + c * C::kWpr * 64;
      unpack8<BF16>(rx[c], h[c]);
      if (a.residual) {
        float r[8];
        unpack8<BF16>(rr[c], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
        const Raw8<BF16> p = pack8<BF16>(h[c]);         // h as stored is what the norm sees
        unpack8<BF16>(p, h[c]);
        if (a.h && live && run < runs) store8<BF16>(a.h, row * a.cols + run * 8, p);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma((double)h[c][j], (double)h[c][j], s);
    }
    if (C::kLean) {
#pragma unroll
      for (int c = 0; c < C::kNch; ++c) weights<WBF16>(a.weight, run0 + c * C::kWpr * 64, runs, w[c]);
    }
    s = row_sum<C::kWpr>(s, sm);
    const double rstd = 1.0 / sqrt(s / (double)a.cols + (double)a.eps);
    if (a.rstd && live && run0 == 0) a.rstd[row] = (float)rstd;
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      const int run = run0 + c * C::kWpr * 64;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (float)((double)h[c][j] * rstd * (double)w[c][j]);
      if (a.codes) {
        const uint32_t sb = mx_scale_byte(mx_amax4(y));
        if (live && run < runs) {
          const int64_t e = row * a.cols + run * 8;
          *reinterpret_cast<u32x2_t *>(a.codes + e) = mx_encode8(y, sb);
          if ((lane & 3) == 0) a.scales[e >> 5] = (uint8_t)sb;
        }
      }
      if (a.y && live && run < runs) store8<BF16>(a.y, row * a.cols + run * 8, pack8<BF16>(y));
    }
  }
}

// --------------------------------------------------------------------- its gradient

// A lane's own 8 sums of chunk c in LDS.
__device__ __forceinline__ void get_dw(const float4 *sums, int c, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 x = sums[(2 * c + h) * blockDim.x + threadIdx.x];
    v[4 * h] = x.x, v[4 * h + 1] = x.y, v[4 * h + 2] = x.z, v[4 * h + 3] = x.w;
  }
}
__device__ __forceinline__ void put_dw(float4 *sums, int c, const float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    sums[(2 * c + h) * blockDim.x + threadIdx.x] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
}

// The sum of N values in pairs: log2(N) roundings to a value, where a chain takes up to N.
template <int N>
__device__ __forceinline__ float pair_sum(float (&v)[N]) {
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] += v[k + n];
  return v[0];
}

// dweight of 32 columns from c0 on: 64 threads' rows of 8 columns each, then the threads in
// pairs.
template <bool BF16>
__device__ __forceinline__ void column_grads(const sshdp_rmsnorm_grad &a, int c0) {
  __shared__ float sums[64][33];
  const int t = threadIdx.x, c = (t & 3) * 8, sl = t >> 2;
  float s[8] = {};
  for (int64_t row = sl; row < a.rows; row += 64) {
    const int64_t e = row * a.cols + c0 + c;
    float dy[8], h[8];
    unpack8<BF16>(load8<BF16>(a.dy, e), dy);
    unpack8<BF16>(load8<BF16>(a.h, e), h);
    const float rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = fmaf(dy[j], h[j] * rstd, s[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[sl][c + j] = s[j];
  __syncthreads();
  if (t >= 32) return;
  const float v = a.first ? 0.f : a.dweight[c0 + t];
  float d[64];
#pragma unroll
  for (int k = 0; k < 64; ++k) d[k] = sums[k][t];
  a.dweight[c0 + t] = v + pair_sum(d);
}

// Workgroups keep their columns' weight-gradient sums in registers over all their
// rows and leave one partial row each; k_dweight adds the partial rows.  Bound by HBM: 8191 x
// 8192 bfloat16 with dh 96 us = 5.6 TB/s, and 7 us of partial rows.
//
// ONCE, for few rows: no partial rows and no second launch.  Workgroups from `row_groups` on
// take 32 columns each and add their weight gradient over all rows, read a second time (the
// rows' statistics are not needed for it: rstd is given).
template <bool BF16, bool WBF16, class C, bool ONCE>
__global__ __launch_bounds__(C::kThreads) void k_rmsnorm_grad(sshdp_rmsnorm_grad a, float *partials, int row_groups) {
  __shared__ double sm[C::kThreads / 64];
  if (ONCE && blockIdx.x >= (unsigned)row_groups) {
    column_grads<BF16>(a, (int)(blockIdx.x - row_groups) * 32);
    return;
  }
  __shared__ float4 sums[C::kLean ? C::kNch * 2 * C::kThreads : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int sub = wave / C::kWpr, run0 = (wave % C::kWpr) * 64 + lane;
  const int runs = (int)(a.cols >> 3);
  float w[C::kNch][8], dw[C::kNch][8];
#pragma unroll
  for (int c = 0; c < C::kNch; ++c) {
    const int run = run0 + c * C::kWpr * 64;
    if (!C::kLean) weights<WBF16>(a.weight, run, runs, w[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[c][j] = 0.f;
    if (C::kLean) put_dw(sums, c, dw[c]);
  }
  for (int64_t g = blockIdx.x; g * C::kRows < a.rows; g += row_groups) {
    const int64_t row = g * C::kRows + sub;
    const bool live = row < a.rows;
    Raw8<BF16> ry[C::kNch], rh[C::kNch], rd[C::kNch];
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      const int run = run0 + c * C::kWpr * 64;
      ry[c] = Raw8<BF16>{};
      rh[c] = Raw8<BF16>{};
      rd[c] = Raw8<BF16>{};
      if (live && run < runs) {
        const int64_t e = row * a.cols + run * 8;
        ry[c] = load8<BF16>(a.dy, e);
        rh[c] = load8<BF16>(a.h, e);
        if (!C::kLean && a.dh) rd[c] = load8<BF16>(a.dh, e);
      }
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      float dy[8], h[8];
      unpack8<BF16>(ry[c], dy);
      unpack8<BF16>(rh[c], h);
      if (C::kLean) {
        weights<WBF16>(a.weight, run0 + c * C::kWpr * 64, runs, w[c]);
        get_dw(sums, c, dw[c]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h[j] * rstd;
        s = fmaf(w[c][j] * dy[j], xhat, s);
        dw[c][j] = fmaf(dy[j], xhat, dw[c][j]);
      }
      if (C::kLean) put_dw(sums, c, dw[c]);
    }
    const float mean = (float)(row_sum<C::kWpr>((double)s, sm) / (double)a.cols);
#pragma unroll
    for (int c = 0; c < C::kNch; ++c) {
      const int run = run0 + c * C::kWpr * 64;
      float dy[8], h[8], dx[8];
      if (C::kLean) {
        weights<WBF16>(a.weight, run, runs, w[c]);
        if (a.dh && live && run < runs) rd[c] = load8<BF16>(a.dh, row * a.cols + run * 8);
      }
      unpack8<BF16>(ry[c], dy);
      unpack8<BF16>(rh[c], h);
      unpack8<BF16>(rd[c], dx);                          // zeros without dh
#pragma unroll
      for (int j = 0; j < 8; ++j) dx[j] = fmaf(rstd, fmaf(-mean, h[j] * rstd, w[c][j] * dy[j]), dx[j]);
      if (live && run < runs) store8<BF16>(a.dx, row * a.cols + run * 8, pack8<BF16>(dx));
    }
  }
  if (ONCE) return;
  // one partial row per workgroup: its waves' rows are added in wave order
  if (C::kRows > 1) {
    __shared__ float4 part[C::kRows > 1 ? C::kRows - 1 : 1][C::kNch][2][64];
#pragma unroll
    for (int c = 0; c < C::kNch; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (sub) part[sub - 1][c][h][lane] = make_float4(dw[c][4 * h], dw[c][4 * h + 1], dw[c][4 * h + 2], dw[c][4 * h + 3]);
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int c = 0; c < C::kNch; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < C::kRows - 1; ++k) {
          const float4 v = part[k][c][h][lane];
          dw[c][4 * h] += v.x;
          dw[c][4 * h + 1] += v.y;
          dw[c][4 * h + 2] += v.z;
          dw[c][4 * h + 3] += v.w;
        }
  }
#pragma unroll
  for (int c = 0; c < C::kNch; ++c) {
    const int run = run0 + c * C::kWpr * 64;
    if (C::kLean) get_dw(sums, c, dw[c]);
    if (run < runs) {
      float4 *p = reinterpret_cast<float4 *>(partials + (int64_t)blockIdx.x * a.cols + run * 8);
      p[0] = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
      p[1] = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
    }
  }
}

// dweight = (first ? 0 : dweight) + sum of the partial rows: 32 columns per
// workgroup, 32 row slices added in pairs.
__global__ __launch_bounds__(1024) void k_dweight(const float *partials, int64_t n, int64_t cols, int first,
                                                  float *dweight) {
  __shared__ float sm[32][33];
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;      // cols % 32 == 0
  float s = 0.f;
  for (int64_t i = sl; i < n; i += 32) s += partials[i * cols + col];
  sm[sl][c] = s;
  __syncthreads();
  if (sl == 0) {
    const float v = first ? 0.f : dweight[col];
    float d[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) d[k] = sm[k][c];
    dweight[col] = v + pair_sum(d);
  }
}

using R1x1 = RowCfg<1, 1>;
using R1x2 = RowCfg<1, 2>;
using R1x4 = RowCfg<1, 4>;
using R4x2 = RowCfg<4, 2>;
using R4x4 = RowCfg<4, 4>;
using R16x2 = RowCfg<16, 2>;
using R16x3 = RowCfg<16, 3>;
using R16x4 = RowCfg<16, 4>;

// Calls f with the row layout for `cols`: the fewest waves per row whose
// registers hold it.
template <class F>
void with_rows(int64_t cols, F f) {
  if (cols <= 512) f(R1x1{});
  else if (cols <= 1024) f(R1x2{});
  else if (cols <= 2048) f(R1x4{});
  else if (cols <= 4096) f(R4x2{});
  else if (cols <= 8192) f(R4x4{});
  else if (cols <= 16384) f(R16x2{});
  else if (cols <= 24576) f(R16x3{});
  else f(R16x4{});
}

constexpr int64_t kNormGroups = 2048;                  // workgroups of the forward at most
// Workgroups of the backward, each leaving a partial row of the weight gradient, at most:
// two per CU keep HBM busy, and each more is a row written and read back (8191 x 8192
// bfloat16: 103 us; 256 108, 1024 110).
constexpr int64_t kGradGroups = 512;
constexpr int64_t kOnceRows = 1024;

template <class C>
int64_t norm_groups(int64_t rows, int64_t most) {
  return std::max<int64_t>(1, std::min((rows + C::kRows - 1) / C::kRows, most));
}

template <class C>
hipError_t rmsnorm(const sshdp_rmsnorm &a, hipStream_t s) {
  const dim3 grid((unsigned)norm_groups<C>(a.rows, kNormGroups)), block(C::kThreads);
  const bool b = a.dtype == SSHDP_DTYPE_BF16, wb = a.weight_dtype == SSHDP_DTYPE_BF16;
  if (b && wb) hipLaunchKernelGGL((k_rmsnorm<true, true, C>), grid, block, 0, s, a);
  else if (b) hipLaunchKernelGGL((k_rmsnorm<true, false, C>), grid, block, 0, s, a);
  else if (wb) hipLaunchKernelGGL((k_rmsnorm<false, true, C>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_rmsnorm<false, false, C>), grid, block, 0, s, a);
  return hipGetLastError();
}

// Up to 1024 rows a second reading costs less than a second launch (bfloat16, 33 x 2048: 4.9
// us a call against 7.5, 512 x 8192 9.6 against 18.9, 1024 x 8192 18.1 against 19.3; 2048 x
// 8192 33.8 against 25.8).
// Not over dy itself: it is read by other workgroups while dx is written.
template <class C>
bool norm_grad_once(const sshdp_rmsnorm_grad &a) {
  return C::kThreads == 256 && a.rows <= kOnceRows && a.dx != a.dy;
}

template <class C, bool ONCE>
hipError_t rmsnorm_grad(const sshdp_rmsnorm_grad &a, float *partials, hipStream_t s) {
  const int groups = (int)norm_groups<C>(a.rows, kGradGroups);
  const dim3 grid((unsigned)(groups + (ONCE ? a.cols / 32 : 0))), block(C::kThreads);
  const bool b = a.dtype == SSHDP_DTYPE_BF16, wb = a.weight_dtype == SSHDP_DTYPE_BF16;
  if (b && wb) hipLaunchKernelGGL((k_rmsnorm_grad<true, true, C, ONCE>), grid, block, 0, s, a, partials, groups);
  else if (b) hipLaunchKernelGGL((k_rmsnorm_grad<true, false, C, ONCE>), grid, block, 0, s, a, partials, groups);
  else if (wb) hipLaunchKernelGGL((k_rmsnorm_grad<false, true, C, ONCE>), grid, block, 0, s, a, partials, groups);
  else hipLaunchKernelGGL((k_rmsnorm_grad<false, false, C, ONCE>), grid, block, 0, s, a, partials, groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows(const void *src, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                             uint8_t *scales, hipStream_t s) {
  const int64_t runs = rows * (cols / 8);
  const dim3 grid((unsigned)std::min<int64_t>((runs + 255) / 256, 1 << 20)), block(256);
  if (bf16) hipLaunchKernelGGL((k_quant_rows<true>), grid, block, 0, s, src, runs, (int)(cols / 8), ld, codes, scales);
  else hipLaunchKernelGGL((k_quant_rows<false>), grid, block, 0, s, src, runs, (int)(cols / 8), ld, codes, scales);
  return hipGetLastError();
}

hipError_t launch_quant_tiles(const void *src, bool bf16, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                              uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, hipStream_t s) {
  const int64_t tiles_c = (cols + kQtCols - 1) / kQtCols;
  const dim3 grid((unsigned)((rows + kQtRows - 1) / kQtRows * tiles_c)), block(256);
#define SSHDP_QT(B, R) \
  hipLaunchKernelGGL((k_quant_tiles<B, R>), grid, block, 0, s, src, rows, cols, ld, codes, scales, codes_t, scales_t, \
                     tiles_c)
  if (bf16 && codes) SSHDP_QT(true, true);
  else if (bf16) SSHDP_QT(true, false);
  else if (codes) SSHDP_QT(false, true);
  else SSHDP_QT(false, false);
#undef SSHDP_QT
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const sshdp_rmsnorm &a, hipStream_t s) {
  hipError_t e = hipSuccess;
  with_rows(a.cols, [&](auto c) { e = rmsnorm<decltype(c)>(a, s); });
  return e;
}

int64_t rmsnorm_partials(int64_t rows, int64_t cols) {
  int64_t n = 0;
  with_rows(cols, [&](auto c) {
    using C = decltype(c);
    n = norm_groups<C>(rows, kGradGroups);
  });
  return n;
}

hipError_t launch_rmsnorm_backward(const sshdp_rmsnorm_grad &a, float *partials, hipStream_t s) {
  hipError_t e = hipSuccess;
  bool once = false;
  if (a.rows)
    with_rows(a.cols, [&](auto c) {
      using C = decltype(c);
      once = norm_grad_once<C>(a);
      if constexpr (C::kThreads == 256) {
        if (once) e = rmsnorm_grad<C, true>(a, nullptr, s);
      }
      if (!once) e = rmsnorm_grad<C, false>(a, partials, s);
    });
  if (e != hipSuccess || once) return e;
  hipLaunchKernelGGL(k_dweight, dim3((unsigned)(a.cols / 32)), dim3(1024), 0, s, partials,
                     a.rows ? rmsnorm_partials(a.rows, a.cols) : 0, a.cols, a.first, a.dweight);
  return hipGetLastError();
}

}  // namespace sshdp
