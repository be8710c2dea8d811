// k_gemm_grouped.hip -- MXFP8 products grouped by expert: consecutive rows of A with each
// expert's own B, the gated pair of them with the activation and G behind, and the weight
// gradients over each expert's rows.
//
// How many rows an expert has is known on the device alone.  A launch has as many workgroups
// as any distribution may need; each finds its expert and tile from the offsets (one load and
// a sum over the wave's lanes for 64 experts) and those left over end at once.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "act.h"
#include "gemm_mx.h"
#include "moe.h"
#include "mx_encode.h"

namespace sshdp {
namespace {

// Expert e's rows, inside the matrix whatever the offsets hold.
__device__ __forceinline__ void rows_of(const int32_t *offsets, int groups, int rows, int e, int &first, int &n) {
  first = n = 0;
  if (e >= groups) return;
  if (!offsets) {
    n = rows;
    return;
  }
  // both ends are brought inside before they are subtracted: the difference cannot overflow
  first = min(max(offsets[e], 0), rows);
  n = max(min(max(offsets[e + 1], 0), rows) - first, 0);
}

// Sum of the lanes up to this one, within rows of 16 and then from row to row.
__device__ __forceinline__ int scan_lanes(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);      // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);      // row_bcast 15: rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);      // row_bcast 31: rows 2 and 3
  return x;
}

struct Found {
  int e, first, rows;                                // the expert and its rows
  int at;                                            // which of its pieces
};

// 64 experts' rows, one a lane, in pieces of PIECE, one expert after the other.
template <int PIECE>
struct Pieces {
  int e0, first, n, mine, upto;                      // upto: of the experts e0 to the lane's

  __device__ __forceinline__ Pieces(const int32_t *offsets, int groups, int rows, int e0_) : e0(e0_) {
    rows_of(offsets, groups, rows, e0 + (threadIdx.x & 63), first, n);
    mine = (n + PIECE - 1) / PIECE;
    upto = scan_lanes(mine);
  }
  __device__ __forceinline__ int all() const { return __builtin_amdgcn_readlane(upto, 63); }
  // Piece `at` of them, the same for every lane; false past the last one.
  __device__ __forceinline__ bool find(int at, Found &f) const {
    const uint64_t past = __ballot(upto > at);
    if (!past) return false;
    const int l = __builtin_ctzll(past);
    f.e = e0 + l;
    f.first = __builtin_amdgcn_readlane(first, l);
    f.rows = __builtin_amdgcn_readlane(n, l);
    f.at = at - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(mine, l));
    return true;
  }
};

// A workgroup's tile: XCD i % 8 takes one contiguous eighth of an order that goes through the
// experts, and through each one's tiles in strips of 4 along its rows, so the workgroups an
// XCD runs at once share an expert's panels.
template <int TM>
__device__ __forceinline__ bool find_tile(const GemmGrouped &g, int tiles_n, Found &f, int &tn) {
  const int rows = (int)g.p.m;
  const Pieces<TM> head(g.offsets, g.groups, rows, 0);  // up to 64 experts are read once
  int64_t pieces = head.all();
  for (int e0 = 64; e0 < g.groups; e0 += 64) pieces += Pieces<TM>(g.offsets, g.groups, rows, e0).all();
  // the launch has a workgroup for every tile of offsets that do not run backwards; experts whose
  // rows overlap have more pieces than an int counts
  const int total = (int)min(pieces * tiles_n, (int64_t)gridDim.x);
  const int id = blockIdx.x, q = total >> 3, rem = total & 7, x = id & 7;
  if (id >= total) return false;
  const int pos = x * q + min(x, rem) + (id >> 3);
  // tiles_n tiles to each of an expert's row pieces, taken strip by strip
  if (!head.find(pos / tiles_n, f)) {
    int at = pos / tiles_n - head.all(), e0 = 64;
    for (; e0 < g.groups; e0 += 64) {
      const Pieces<TM> some(g.offsets, g.groups, rows, e0);
      if (some.find(at, f)) break;
      at -= some.all();
    }
    if (e0 >= g.groups) return false;
  }
  const int tiles_m = (f.rows + TM - 1) / TM, in = pos - (pos / tiles_n - f.at) * tiles_n;
  const int strip = in / (4 * tiles_n), rest = in - strip * 4 * tiles_n, h = min(4, tiles_m - 4 * strip);
  tn = rest / h;
  f.at = 4 * strip + rest - tn * h;
  return true;
}

// The expert's part of the operands.
__device__ __forceinline__ void take_rows(GemmMx &p, const GemmMx &a, const Found &f, bool nn) {
  p.m = f.rows;
  p.a = a.a + f.first * a.k;
  p.as = a.as + f.first * (a.k >> 5);
  const int64_t block = a.lb == SSHDP_SCALE_BLOCK32X32 ? 1024 : 32;
  p.b = a.b + f.e * (a.n * a.k);
  p.bs = a.bs + f.e * (a.n * a.k / block);
}

// A gated tile's end.  A wave holds its columns' gates in the first half of its n fragments
// and their ups in the second, so the activation needs no exchange, and a block of 32 columns
// is two fragments of the four lanes that share a row.
template <class C>
__device__ __forceinline__ void finish_gated(const GemmGrouped &g, const GemmMx &p, char *smem, int64_t n0, int64_t m0, int first,
                                             int wn, int wm, int t, const f32x4_t (&acc)[C::FP][C::FQ]) {
  constexpr int HP = C::FP / 2, FQ = C::FQ, HN = C::TN / 2, WN2 = HN / C::WN;   // columns of a tile, of a wave
  const int r = t & 15, gq = t >> 4 & 3;
  if (g.gate) {
    // gates in the tile's first half of columns, ups in the second
    uint16_t *lt = reinterpret_cast<uint16_t *>(smem);
    constexpr int LP = C::TN + 8, CH = C::TN / 8;
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        const f32x4_t &v = acc[i][j];
        const int c = (i < HP ? 0 : HN) + wn * WN2 + 16 * (i % HP) + 4 * gq;
        *reinterpret_cast<uint2 *>(lt + (wm * (C::TM / C::WM) + 16 * j + r) * LP + c) =
            make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
      }
    __syncthreads();
    for (int id = t; id < C::TM * CH; id += C::NT) {
      const int row = id / CH, c = (id - row * CH) * 8, cc = c & (HN - 1);
      if (m0 + row >= p.m || n0 + cc >= p.n) continue;      // whole chunks: n is a multiple of 32
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(lt + row * LP + c);
      uint16_t *o = (c < HN ? g.gate : g.up) + (first + m0 + row) * p.n + n0 + cc;
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t *>(o));
    }
    __syncthreads();
  }
  if (!g.codes) return;
  // codes and scales of the tile in LDS, then 16 codes and a row's scales a lane
  constexpr int CP = HN + 16, SB = HN / 32;
  uint8_t *lc = reinterpret_cast<uint8_t *>(smem), *ls = lc + C::TM * CP;
#pragma unroll
  for (int j = 0; j < FQ; ++j)
#pragma unroll
    for (int b = 0; b < HP / 2; ++b) {
      float h[8];
      uint32_t a = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float gate = acc[2 * b + (k >> 2)][j][k & 3];
        h[k] = gate * sigmoid_near(gate) * acc[HP + 2 * b + (k >> 2)][j][k & 3];
        a = max(a, __float_as_uint(h[k]) & 0x7FFFFFFFu);
      }
      const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);   // the lanes 16 apart
      a = max(x[0], x[1]);
      const auto y = __builtin_amdgcn_permlane32_swap(a, a, false, false);   // and 32
      const uint32_t sb = mx_scale_byte(max(y[0], y[1]));
      const float sf = mx_scale_float(sb);
      const uint32_t c[2] = {mx_or_nan(mx_cvt4(h[0], h[1], h[2], h[3], sf), sb), mx_or_nan(mx_cvt4(h[4], h[5], h[6], h[7], sf), sb)};
      const int row = wm * (C::TM / C::WM) + 16 * j + r, col = wn * WN2 + 32 * b;
      *reinterpret_cast<uint32_t *>(lc + row * CP + col + 4 * gq) = c[0];
      *reinterpret_cast<uint32_t *>(lc + row * CP + col + 16 + 4 * gq) = c[1];
      if (gq == 0) ls[row * SB + (col >> 5)] = (uint8_t)sb;
    }
  __syncthreads();
  for (int id = t; id < C::TM * (HN / 16); id += C::NT) {
    const int row = id / (HN / 16), c = (id - row * (HN / 16)) * 16;
    if (m0 + row >= p.m || n0 + c >= p.n) continue;
    *reinterpret_cast<u32x4_t *>(g.codes + (first + m0 + row) * p.n + n0 + c) =
        *reinterpret_cast<const u32x4_t *>(lc + row * CP + c);
  }
  for (int id = t; id < C::TM * SB; id += C::NT) {
    const int row = id / SB, b = id - row * SB;
    if (m0 + row < p.m && n0 + 32 * b < p.n)
      g.scales[(first + m0 + row) * (p.n >> 5) + (n0 >> 5) + b] = ls[id];
  }
}

// bfloat16 addend into a tile's sums, 4 columns of a row a lane, a row block's words in flight
// together (more of them would not fit beside a 256-tile's sums); rows past the end read the
// last one's.
template <class C>
__device__ __forceinline__ void add_bf16(const GemmMx &p, const uint16_t *addend, int64_t n0, int64_t m0, int wn, int wm, int t,
                                         f32x4_t (&acc)[C::FP][C::FQ]) {
  const int64_t mw = m0 + wm * (C::TM / C::WM) + (t & 15), nw = n0 + wn * (C::TN / C::WN) + 4 * (t >> 4 & 3);
  const bool whole = n0 + C::TN <= p.n;
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) {
    const uint16_t *row = addend + min(mw + 16 * j, p.m - 1) * p.ld + nw;
    u32x2e_t w[C::FP];
#pragma unroll
    for (int i = 0; i < C::FP; ++i) {
      w[i] = u32x2e_t{0, 0};
      if (whole || nw + 16 * i + 4 <= p.n) {
        w[i] = *reinterpret_cast<const u32x2e_t *>(row + 16 * i);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (nw + 16 * i + k < p.n) w[i][k >> 1] |= (uint32_t)row[16 * i + k] << (16 * (k & 1));
      }
    }
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][j][k] += __uint_as_float(k & 1 ? w[i][k >> 1] & 0xFFFF0000u : w[i][k >> 1] << 16);
#pragma unroll
    for (int i = 0; i < C::FP; ++i) asm volatile("" : "+v"(acc[i][j])::"memory");
  }
}

// A tile of an expert's rows, bfloat16 or codes out.  Bound by the wait for operands at each step and,
// in 256-tiles, by what one workgroup a CU has nothing to hide behind: its first operands and its
// end (8 us of the 37 of a gated tile with K 2048).  24558 slots of 64 experts, operands from HBM:
// gated 2 x 1408 x 2048 with both kept 218 to 229 us (283 GFLOP, 606 MB; matrix cores 37% busy),
// by 128-tiles 245; input gradient, K 2048 and 1408 columns, 124 to 131 us (142 GFLOP, 311 MB; 37%).
// Workgroups that stay and walk the tiles lose to the hardware's dealing: 146 us for the gradient.
// The 8-bit instruction's cut is a choice: with float32 sums the gated pair takes 1.3 times as long
// (351 against 266 us after a write through the caches).  Of 37 million codes of h 59000 then move
// over a rounding border no more, and h is no nearer: 2.65e-2 of itself from its value with
// either, which is G's own rounding.
template <class C, bool NN, bool SHORT, Form F>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPS, C::WPS))) void k_group8(GemmGrouped g, int tiles_n) {
  __shared__ __align__(1024) char smem[C::LDS];
  Found f;
  int tn;
  if (!find_tile<C::TM>(g, tiles_n, f, tn)) return;
  GemmPart p;
  static_cast<GemmMx &>(p) = g.p;
  take_rows(p, g.p, f, NN);
  if (F == kGated) {
    p.b2 = g.b2 + (p.b - g.p.b);
    p.b2s = g.b2s + (p.bs - g.p.bs);
  }
  const int64_t n0 = (int64_t)tn * (F == kGated ? C::TN / 2 : C::TN), m0 = (int64_t)f.at * C::TM;
  const Loader<C, NN, F> ld(p, n0, m0, 0, (int)((p.k + kRowB - 1) / kRowB));
  const int wn = ld.wave / C::WM, wm = ld.wave % C::WM;
  f32x4_t acc[C::FP][C::FQ];
  sums8<C, NN, SHORT>(ld, smem, acc);
  __syncthreads();
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  if constexpr (F == kGated) {
    finish_gated<C>(g, p, smem, n0, m0, f.first, wn, wm, t_end, acc);
  } else {
    const int64_t out = f.first * p.ld;
    p.out = static_cast<uint16_t *>(p.out) + out;
    if (g.addend16) add_bf16<C>(p, g.addend16 + out, n0, m0, wn, wm, t_end, acc);
    store_tile_bf16<C>(p, smem, n0, m0, wn, wm, t_end, acc);
  }
}

// The same with float32 out, in float32 sums at half the matrix rate.
template <class C, bool NN, bool SHORT>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPS, C::WPS))) void k_group16(GemmGrouped g, int tiles_n) {
  __shared__ __align__(1024) char smem[C::LDS];
  Found f;
  int tn;
  if (!find_tile<C::TM>(g, tiles_n, f, tn)) return;
  GemmMx p = g.p;
  take_rows(p, g.p, f, NN);
  const int64_t n0 = (int64_t)tn * C::TN, m0 = (int64_t)f.at * C::TM;
  const Loader<C, NN> ld(p, n0, m0, 0, (int)((p.k + kRowB - 1) / kRowB));
  const int wn = ld.wave / C::WM, wm = ld.wave % C::WM;
  f32x4_t acc[C::FP][C::FQ];
  sums16<C, NN, SHORT>(ld, smem, acc);
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  const int64_t out = f.first * p.ld;
  p.out = static_cast<float *>(p.out) + out;
  if (p.addend) p.addend += out;
  store_tile_f32<C>(p, n0, m0, wn, wm, t_end, acc);
}

// A tile's rows in memory's order, through LDS: 4 columns a lane, whole lines an instruction.
// Straight from the sums' layout, 64 bytes of 16 rows an instruction, HBM gave 2.7 TB/s (64
// gradients of 1408 x 2048 over 26624 rows: 555 us).
template <class C>
struct RowOrder {
  static constexpr int LP = C::TN + 4, PER = C::NT * 4 / C::TN, N = C::TM / PER;   // rows an instruction; of them
  static_assert(C::TM * LP * 4 <= C::LDS, "the tile fits the stages");
  const GemmMx &p;
  const int64_t n;
  const int row;
  const int64_t m0;

  __device__ __forceinline__ RowOrder(const GemmMx &p_, int64_t n0, int64_t m0_, int t)
      : p(p_), n(n0 + (t * 4) % C::TN), row(t * 4 / C::TN), m0(m0_) {}

  __device__ __forceinline__ void load(const float *src, f32x4_t (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t m = m0 + row + i * PER;
      v[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (m >= p.m || n >= p.n) continue;
      const float *q = src + m * p.ld + n;
      if (n + 4 <= p.n) {
        v[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4e_t *>(q));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < p.n) v[i][k] = q[k];
      }
    }
  }

  // Of a tile that lies inside: exactly N loads.
  __device__ __forceinline__ void load_whole(const float *src, f32x4_t (&v)[N]) const {
    const float *q = src + (m0 + row) * p.ld + n;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4e_t *>(q + i * PER * p.ld));
  }

  // The sums to LDS, by the threads that have them; a barrier comes before store.
  static __device__ __forceinline__ void put(char *smem, int wn, int wm, int t, const f32x4_t (&acc)[C::FP][C::FQ]) {
    float *lt = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int j = 0; j < C::FQ; ++j)
#pragma unroll
      for (int i = 0; i < C::FP; ++i)
        *reinterpret_cast<f32x4_t *>(lt + (wm * (C::TM / C::WM) + 16 * j + (t & 15)) * LP + wn * (C::TN / C::WN) + 16 * i +
                                     4 * (t >> 4 & 3)) = acc[i][j];
  }

  // LDS + v to the output.
  __device__ __forceinline__ void store(const char *smem, int t, const f32x4_t (&v)[N]) const {
    const float *lt = reinterpret_cast<const float *>(smem);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t m = m0 + row + i * PER;
      if (m >= p.m || n >= p.n) continue;
      const f32x4_t x = *reinterpret_cast<const f32x4_t *>(lt + (row + i * PER) * LP + (t * 4) % C::TN) + v[i];
      float *o = static_cast<float *>(p.out) + m * p.ld + n;
      if (n + 4 <= p.n) {
        __builtin_nontemporal_store(x, reinterpret_cast<f32x4e_t *>(o));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < p.n) o[k] = x[k];
      }
    }
  }
};

// Weight gradients: tile `pos` of all experts', one expert's after the other's, each one's in
// strips of 4 along m.
template <class C>
struct ColumnTile {
  GemmPart p;
  int64_t n0, m0;

  __device__ __forceinline__ ColumnTile(const GemmGrouped &g, int pos, int tiles_m, int tiles_n) {
    const int tiles = tiles_m * tiles_n, e = pos / tiles, in = pos - e * tiles;
    const int strip = in / (4 * tiles_n), rest = in - strip * 4 * tiles_n, h = min(4, tiles_m - 4 * strip);
    n0 = (int64_t)(rest / h) * C::TN;
    m0 = (int64_t)(4 * strip + rest % h) * C::TM;
    int first, n;
    rows_of(g.offsets, g.groups, (int)g.p.k, e, first, n);
    static_cast<GemmMx &>(p) = g.p;
    p.pitch = g.p.k;
    p.start = first & ~31;
    p.k = n & ~31;
    const int64_t out = e * p.m * p.ld;
    p.out = static_cast<float *>(p.out) + out;
    if (p.addend) p.addend += out;
  }
  __device__ __forceinline__ int steps() const { return (int)((p.k + kRowB - 1) / kRowB); }
  // an expert without rows leaves what is there
  __device__ __forceinline__ bool nothing() const { return !p.k && p.addend == p.out; }
};

template <class C>
__device__ __forceinline__ void column_sums(const ColumnTile<C> &t, char *smem, f32x4_t (&acc)[C::FP][C::FQ]) {
  if (t.p.k) {
    const Loader<C, false, kRange> ld(t.p, t.n0, t.m0, 0, t.steps());
    sums16<C, false, false, true>(ld, smem, acc);
  } else {
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}

template <class C>
__device__ __forceinline__ void column_addend(const ColumnTile<C> &t, const RowOrder<C> &rows, f32x4_t (&add)[RowOrder<C>::N]) {
  if (t.p.addend) {
    rows.load(t.p.addend, add);
  } else {
#pragma unroll
    for (int i = 0; i < RowOrder<C>::N; ++i) add[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}

// Where XCD x's tiles of all experts' begin, in an order of one expert's after the other's: the
// eighths are of equal work, a tile's being its steps and as much as kTileWork more for what
// every tile moves.  Experts' rows differ many times over; eighths of equal numbers of tiles
// take as long as the one with the most rows (410 to 455 against 368 to 418 us; at a unit of 2,
// 12 and 24 for the rest 401, 401 and 413).
constexpr int kTileWork = 6;
__device__ __forceinline__ int xcd_begin(const GemmGrouped &g, int tiles, int x) {
  if (x == 0) return 0;
  if (x == 8) return tiles * g.groups;
  const int lane = threadIdx.x & 63;
  auto work_of = [&](int e) __attribute__((always_inline)) {
    int first, n;
    rows_of(g.offsets, g.groups, (int)g.p.k, e, first, n);
    return e < g.groups ? kTileWork + (n + kRowB - 1) / kRowB : 0;
  };
  int total = 0;
  for (int e0 = 0; e0 < g.groups; e0 += 64) total += __builtin_amdgcn_readlane(scan_lanes(work_of(e0 + lane)), 63);
  const int64_t target = (int64_t)total * x;          // in eighths of a unit
  int64_t base = 0;
  for (int e0 = 0; e0 < g.groups; e0 += 64) {
    const int mine = work_of(e0 + lane), upto = scan_lanes(mine);
    const uint64_t past = __ballot(8 * (base + upto) > target);
    if (past) {
      const int l = __builtin_ctzll(past), c = __builtin_amdgcn_readlane(mine, l);
      const int64_t in = target - 8 * (base + __builtin_amdgcn_readlane(upto, l) - c);
      return (e0 + l) * tiles + (int)(in * tiles / (8 * c));
    }
    base += __builtin_amdgcn_readlane(upto, 63);
  }
  return tiles * g.groups;
}

// A workgroup walks its XCD's tiles, two workgroups a CU.  The addend comes in behind the first
// two stages' operands, while the first products are made; experts of a few hundred rows leave
// little more time than that.  Bound by HBM and by the turns of reading, multiplying and writing:
// 64 gradients of 1408 x 2048 over 24558 rows, added to what was there, 369 us (1.56 GB, 4.2 TB/s;
// 142 GFLOP, matrix cores 19% busy).
template <class C>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WPS, C::WPS))) void k_group_columns(GemmGrouped g, int tiles_m,
                                                                                            int tiles_n) {
  __shared__ __align__(1024) char smem[C::LDS];
  const int x = blockIdx.x & 7, end = xcd_begin(g, tiles_m * tiles_n, x + 1), step = (int)(gridDim.x + 7 - x) >> 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int pos = xcd_begin(g, tiles_m * tiles_n, x) + ((int)blockIdx.x >> 3); pos < end; pos += step) {
    const ColumnTile<C> tile(g, pos, tiles_m, tiles_n);
    if (tile.nothing()) continue;
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    const RowOrder<C> rows(tile.p, tile.n0, tile.m0, t);
    f32x4_t add[RowOrder<C>::N], acc[C::FP][C::FQ];
    if (tile.p.k && tile.p.addend && tile.m0 + C::TM <= tile.p.m && tile.n0 + C::TN <= tile.p.n) {
      const Loader<C, false, kRange> ld(tile.p, tile.n0, tile.m0, 0, tile.steps());
      sums16<C, false, false, true, RowOrder<C>::N>(ld, smem, acc, [&]() __attribute__((always_inline)) { rows.load_whole(tile.p.addend, add); });
    } else {
      column_addend<C>(tile, rows, add);
      column_sums<C>(tile, smem, acc);
    }
    __syncthreads();
    RowOrder<C>::put(smem, wave / C::WM, wave % C::WM, t, acc);
    __syncthreads();
    rows.store(smem, t, add);
    __syncthreads();                                 // read before the next tile's stages are written
  }
}

// ----------------------------------------------------------------- a few rows an expert
//
// Bound by reading the experts' B once.  A workgroup makes 16 rows of one expert by 64 rows of
// B (gated: 32 of each matrix): its W waves share K, a wave has 4 steps of all of them in
// flight at once, straight from memory to registers, and its sums meet the others' in LDS.
// The products are float32 sums whatever the output: the conversions that takes cost nothing
// beside the reads.  For bfloat16 output (and gated), where any scale is allowed, rows with elements
// that bfloat16 does not hold exactly are multiplied as codes, as tiles multiply all.  Looking for
// them takes 0.1 to 0.3 us; a wave that has some goes over its operands again (two experts of 16
// rows, all such: 20 us instead of 13.5).  16 tokens of 6 choices, 64 experts, gated 2 x 1408 x
// 2048: 47 to 52 us for the 302 MB of the 50 experts in use, 5.8 to 6.4 TB/s.
constexpr int kFewSteps = 4, kFewFrags = 4;
// Scale bytes under which every code is a normal bfloat16 number: 2^-9 2^(10 - 127) = 2^-126 and
// 1.75 2^8 2^(246 - 127) < 2^128.
constexpr uint32_t kBf16Least = 10, kBf16Most = 246;

template <Form F, bool BF16, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_group_few(GemmGrouped g, int blocks_n) {
  constexpr int S = kFewSteps, NF = kFewFrags;
  typedef uint32_t u32x4u_t __attribute__((ext_vector_type(4), aligned(1)));   // scales lie at any address
  typedef uint32_t u32u_t __attribute__((aligned(1)));
  __shared__ __align__(16) f32x4_t part[W][NF][64];
  Found f;
  int block;
  if (!find_tile<16>(g, blocks_n, f, block)) return;
  GemmPart p;
  static_cast<GemmMx &>(p) = g.p;
  take_rows(p, g.p, f, false);
  if (F == kGated) {
    p.b2 = g.b2 + (p.b - g.p.b);
    p.b2s = g.b2s + (p.bs - g.p.bs);
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const int KB = (int)(p.k >> 5), m0 = 16 * f.at, rows = min(16, f.rows - m0);
  const int64_t n0 = (int64_t)block * (F == kGated ? 32 : 64);
  // fragment i: 16 rows of B from n on
  auto column = [&](int i) __attribute__((always_inline)) { return n0 + 16 * (F == kGated ? i & 1 : i); };
  // Rows past the end are past their resource, chunks past K are sent there: both read as zeros.
  auto resource = [&](const uint8_t *base, int64_t n) __attribute__((always_inline)) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, (int)(n * p.k), kBufWord3);
  };
  const __amdgpu_buffer_rsrc_t ra = resource(p.a + m0 * p.k, rows);
  __amdgpu_buffer_rsrc_t rb[NF];
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    const int64_t n = column(i), left = max(min<int64_t>(p.n - n, 16), (int64_t)0);
    rb[i] = resource((F == kGated && i >= 2 ? p.b2 : p.b) + (left ? n * p.k : 0), left);
  }
  // word j: a row's blocks kb + 4 j .. + 3, ones (beside codes of zero) past the end
  struct Words {
    uint32_t w[S];
  };
  auto row_scales = [&](const uint8_t *s, int layout, int64_t row) __attribute__((always_inline)) {
    if (layout == SSHDP_SCALE_TILE32X4) return s + (row >> 5) * (KB >> 2) * 128 + (row & 31) * 4;
    return s + (layout == SSHDP_SCALE_ROWMAJOR ? row : row >> 5) * KB;
  };
  auto word = [&](const uint8_t *s, bool tile, int at) __attribute__((always_inline)) {
    const int n = min(KB - at, 4);
    const uint8_t *b = s + (tile ? (at >> 2) * 128 : at);
    uint32_t v = 0x7F7F7F7Fu;
    if (n == 4) v = *reinterpret_cast<const u32u_t *>(b);
    else for (int i = 0; i < n; ++i) v ^= (uint32_t)(b[i] ^ 0x7F) << (8 * i);
    return v;
  };
  auto scales = [&](const uint8_t *s, int layout, int64_t row, int kb) __attribute__((always_inline)) {
    const bool tile = layout == SSHDP_SCALE_TILE32X4;
    s = row_scales(s, layout, row);
    Words v{};
    if (kb + 4 * S <= KB && !tile) {
      const u32x4_t x = *reinterpret_cast<const u32x4u_t *>(s + kb);
#pragma unroll
      for (int j = 0; j < S; ++j) v.w[j] = x[j];
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) v.w[j] = word(s, tile, kb + 4 * j);
    }
    return v;
  };
  auto b_row = [&](int i) __attribute__((always_inline)) { return min(column(i) + r, p.n - 1); };
  auto b_scales = [&](int i) __attribute__((always_inline)) { return F == kGated && i >= 2 ? p.b2s : p.bs; };
  const int64_t a_row = m0 + min(r, rows - 1);
  f32x4_t acc[NF];
#pragma unroll
  for (int i = 0; i < NF; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // The byte of the lane's chunk in half h of a step: its block is 2 h + q / 2.
  auto byte = [&](uint32_t w, int h) __attribute__((always_inline)) { return (w >> (8 * (2 * h + (q >> 1)))) & 0xFFu; };
  auto any_code = [](const u32x4_t &c) __attribute__((always_inline)) { return (c[0] | c[1] | c[2] | c[3]) & 0x7F7F7F7Fu; };
  auto multiply = [&](const u32x4_t &x, uint32_t ea, const u32x4_t (&z)[NF], const uint32_t (&eb)[NF]) __attribute__((always_inline)) {
    const u32x4_t y[2] = {to_bf16((int)x[0], (int)x[1], ea), to_bf16((int)x[2], (int)x[3], ea)};
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      acc[i] = mma_bf16(to_bf16((int)z[i][0], (int)z[i][1], eb[i]), y[0], acc[i]);
      acc[i] = mma_bf16(to_bf16((int)z[i][2], (int)z[i][3], eb[i]), y[1], acc[i]);
    }
  };
  auto load = [&](__amdgpu_buffer_rsrc_t rs, int c, int from) __attribute__((always_inline)) {
    const int k0 = from * 32 + 16 * q, left = (int)p.k - k0, voff = r * (int)p.k + k0;
    return __builtin_bit_cast(u32x4_t,
                              __builtin_amdgcn_raw_buffer_load_b128(rs, 64 * c < left ? voff + 64 * c : INT32_MAX - 15, 0, 0));
  };
  uint32_t small = 0;                                // codes of elements under bfloat16's normal numbers
  for (int kb = 4 * S * wave; kb < KB; kb += 4 * S * W) {
    u32x4_t a[2 * S], b[NF][2 * S];
    Words wa, wb[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      wb[i] = scales(b_scales(i), p.lb, b_row(i), kb);
#pragma unroll
      for (int c = 0; c < 2 * S; ++c) b[i][c] = load(rb[i], c, kb);
    }
    wa = scales(p.as, SSHDP_SCALE_ROWMAJOR, a_row, kb);
#pragma unroll
    for (int c = 0; c < 2 * S; ++c) a[c] = load(ra, c, kb);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t least = 255;                            // of the scale bytes
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t z[NF];
        uint32_t eb[NF], ea = byte(wa.w[s], h);
        least = min(least, ea);
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          z[i] = b[i][2 * s + h];
          eb[i] = byte(wb[i].w[s], h);
          least = min(least, eb[i]);
        }
        multiply(a[2 * s + h], ea, z, eb);
      }
    }
    if (BF16 && __any(least < kBf16Least)) {         // blocks of zeros, as a rule
#pragma unroll
      for (int c = 0; c < 2 * S; ++c) {
        small |= byte(wa.w[c >> 1], c & 1) < kBf16Least ? any_code(a[c]) : 0;
#pragma unroll
        for (int i = 0; i < NF; ++i) small |= byte(wb[i].w[c >> 1], c & 1) < kBf16Least ? any_code(b[i][c]) : 0;
      }
    }
  }
  // an element from 2^128 on makes sums infinite or NaN
  uint32_t most = small ? 0x7F800000u : 0;
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) most = max(most, __float_as_uint(acc[i][k]) & 0x7FFFFFFFu);
  if (BF16 && __any(most >= 0x7F800000u)) {
    // Some of the wave's elements are outside bfloat16's range, or NaN: its steps once more, each
    // multiplied as codes too, which the 8-bit instruction takes under every scale.  The rows of A
    // and of B with such elements take those sums, the others come out as they were.
#pragma unroll
    for (int i = 0; i < NF; ++i) acc[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int kb = 4 * S * wave; kb < KB; kb += 4 * S * W) {
      for (int at = kb; at < min(kb + 4 * S, KB); at += 4) {
        u32x4_t x[2], z[2][NF];
        uint32_t xw = word(row_scales(p.as, SSHDP_SCALE_ROWMAJOR, a_row), false, at), zw[NF];
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = load(ra, h, at);
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          zw[i] = word(row_scales(b_scales(i), p.lb, b_row(i)), p.lb == SSHDP_SCALE_TILE32X4, at);
#pragma unroll
          for (int h = 0; h < 2; ++h) z[h][i] = load(rb[i], h, at);
        }
        // whether a chunk has such an element; then the rows of the 16 that have one, a bit each
        auto beyond = [&](const u32x4_t &c, uint32_t e) __attribute__((always_inline)) {
          return any_code(c) && (e < kBf16Least || (e > kBf16Most && e != 255));
        };
        auto rows_of_lanes = [](bool any) __attribute__((always_inline)) {
          const uint64_t v = __ballot(any);
          const uint32_t o = (uint32_t)v | (uint32_t)(v >> 32);
          return (o | o >> 16) & 0xFFFFu;
        };
        auto codes = [](const u32x4_t &u, const u32x4_t &v) __attribute__((always_inline)) {
          return i32x8_t{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
        };
        const uint32_t of_a = rows_of_lanes(beyond(x[0], byte(xw, 0)) || beyond(x[1], byte(xw, 1)));
        uint32_t of_b[NF];
        f32x4_t any[NF];
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          of_b[i] = rows_of_lanes(beyond(z[0][i], byte(zw[i], 0)) || beyond(z[1][i], byte(zw[i], 1)));
          any[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes(z[0][i], z[1][i]), codes(x[0], x[1]), acc[i], 0, 0, 0,
                                                                    (int)(zw[i] >> (8 * q)), 0, (int)(xw >> (8 * q)));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t eb[NF];
#pragma unroll
          for (int i = 0; i < NF; ++i) eb[i] = byte(zw[i], h);
          multiply(x[h], byte(xw, h), z[h], eb);
        }
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][k] = (of_a >> r | of_b[i] >> (4 * q + k)) & 1 ? any[i][k] : acc[i][k];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NF; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  auto total = [&](int i) __attribute__((always_inline)) {
    f32x4_t v = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][i][lane];
    return v;
  };
  p.m = rows;
  const int64_t out = f.first + m0;
  if constexpr (F == kGated) {
    if (wave) return;
    float h[8];
    uint32_t m = 0;
    const int64_t e = (out + r) * p.n + n0 + 4 * q;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const f32x4_t gate = total(c), up = total(2 + c);
      if (g.gate && r < rows) {
        *reinterpret_cast<uint2 *>(g.gate + e + 16 * c) = make_uint2(pk_bf16(gate[0], gate[1]), pk_bf16(gate[2], gate[3]));
        *reinterpret_cast<uint2 *>(g.up + e + 16 * c) = make_uint2(pk_bf16(up[0], up[1]), pk_bf16(up[2], up[3]));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[4 * c + k] = gate[k] * sigmoid(gate[k]) * up[k];
        m = max(m, __float_as_uint(h[4 * c + k]) & 0x7FFFFFFFu);
      }
    }
    if (!g.codes) return;
    const auto x = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(x[0], x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    const uint32_t sb = mx_scale_byte(max(y[0], y[1]));
    if (r >= rows) return;
    const float sf = mx_scale_float(sb);
    *reinterpret_cast<uint32_t *>(g.codes + e) = mx_or_nan(mx_cvt4(h[0], h[1], h[2], h[3], sf), sb);
    *reinterpret_cast<uint32_t *>(g.codes + e + 16) = mx_or_nan(mx_cvt4(h[4], h[5], h[6], h[7], sf), sb);
    if (q == 0) g.scales[(out + r) * (p.n >> 5) + block] = (uint8_t)sb;
  } else {
    for (int i = wave; i < NF; i += W) {
      f32x4_t v = total(i);
      const int64_t n = column(i) + 4 * q, e = out * p.ld;
      if (BF16) {
        p.out = static_cast<uint16_t *>(g.p.out) + e;
        if (g.addend16 && r < rows) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + k < p.n) v[k] += __uint_as_float((uint32_t)g.addend16[e + r * p.ld + n + k] << 16);
        }
        store_bf16(p, r, n, v);
      } else {
        if (g.p.addend) p.addend = g.p.addend + e;
        store_f32(p, static_cast<float *>(g.p.out) + e, r, n, v);
      }
    }
  }
}

template <class C, bool NN, Form F>
hipError_t group_rows(const GemmGrouped &g, hipStream_t s) {
  const int cols = grouped_cols(g.form, C::TM), tn = (int)((g.p.n + cols - 1) / cols);
  const dim3 grid((unsigned)grouped_tiles(g.form, g.groups, g.p.m, g.p.n, C::TM)), block(C::NT);
  auto launch = [&](auto sh) {
    constexpr bool SHORT = decltype(sh)::value;
    if (g.bf16) hipLaunchKernelGGL((k_group8<C, NN, SHORT, F>), grid, block, 0, s, g, tn);
    else if constexpr (C::TM == 128 && F == kWhole) hipLaunchKernelGGL((k_group16<C, NN, SHORT>), grid, block, 0, s, g, tn);
  };
  if (gemm_short(g.p.k)) launch(std::true_type{});
  else launch(std::false_type{});
  return hipGetLastError();
}

template <Form F, bool BF16>
hipError_t group_few(const GemmGrouped &g, hipStream_t s) {
  const int cols = grouped_cols(g.form, 16), blocks = (int)((g.p.n + cols - 1) / cols);
  const dim3 grid((unsigned)grouped_tiles(g.form, g.groups, g.p.m, g.p.n, 16));
  if (g.p.k <= 2048) hipLaunchKernelGGL((k_group_few<F, BF16, 4>), grid, dim3(256), 0, s, g, blocks);
  else hipLaunchKernelGGL((k_group_few<F, BF16, 8>), grid, dim3(512), 0, s, g, blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_grouped(const GemmGrouped &g, hipStream_t s) {
  if (g.form == kColumns) {
    // what the CUs hold at once: every XCD has its share whatever the number of tiles
    const int tm = (int)((g.p.m + 127) / 128), tn = (int)((g.p.n + 127) / 128);
    hipLaunchKernelGGL((k_group_columns<T128>), dim3(512), dim3(T128::NT), 0, s, g, tm, tn);
    return hipGetLastError();
  }
  const int tile = grouped_tile(g.form, g.groups, g.p.m, g.p.n, g.p.k, g.bf16);
  if (tile == 16) {
    if (g.form == kRowsGated) return group_few<kGated, true>(g, s);
    return g.bf16 ? group_few<kWhole, true>(g, s) : group_few<kWhole, false>(g, s);
  }
  const bool large = tile == 256;
  if (g.form == kRowsGated) return large ? group_rows<T256, false, kGated>(g, s) : group_rows<T128, false, kGated>(g, s);
  if (g.form == kRowsNN) return large ? group_rows<T256, true, kWhole>(g, s) : group_rows<T128, true, kWhole>(g, s);
  return large ? group_rows<T256, false, kWhole>(g, s) : group_rows<T128, false, kWhole>(g, s);
}

}  // namespace sshdp
