// k_gemm_mx.hip -- MXFP8 products: kernels of few rows, of tiles, and the join of K splits.
// Their arithmetic, operand layouts and tiles are in gemm_mx.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "gemm_mx.h"
#include "gemm_shape.h"
#include "internal.h"

namespace sshdp {
namespace {

// ------------------------------------------------------------------- few-row products

// out of p.m rows for a few m, and NN operands of fewer scale blocks than a word: bound by
// reading B once, and by the L1's rate of lines (16 rows of codes are 16 lines a load, and
// A's and the scales' are as many again).  A workgroup's W waves share 16 * NF columns n and
// split K among them, one 128-k step in W each, so together they read runs of W * 128 bytes
// of B's rows; codes go straight from memory to the matrix instructions, one step's loads in
// flight while another's are multiplied (two to four in flight were slower: fewer waves).
// MT * 16 rows of m at a time; rows past the end repeat the last one.  The waves' sums meet
// in LDS and are added in wave order.  bfloat16 and float32 output, operands from HBM: 32 x
// 2048 x 2048 6.8 and 8.4 us, 24 x 2048 x 4864 10.1 and 12.5.
template <bool NN, bool BF16, int W, int NF, int MT>
__global__ __launch_bounds__(64 * W) void k_gemm_mx_rows(GemmMx p, int64_t tiles_n, int64_t first) {
  __shared__ __align__(16) f32x4_t part[W][NF * MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t id = first + blockIdx.x;
  const int64_t nb = id % tiles_n * 16 * NF, mb = id / tiles_n * 16 * MT;
  const int KB = (int)(p.k >> 5), nk = (int)((p.k + 127) / 128);
  const uint8_t *pb[NF], *pa[MT], *sb[NF], *sa[MT];
  int tb, ta;                                        // scale bytes: block kb of the row at (kb / 4) * t + kb % 4
  auto row_scales = [](const uint8_t *s, int layout, int64_t row, int KB_, int &t) __attribute__((always_inline)) {
    t = layout == SSHDP_SCALE_TILE32X4 ? 128 : 4;
    if (layout == SSHDP_SCALE_TILE32X4) return s + (row >> 5) * (KB_ >> 2) * 128 + (row & 31) * 4;
    return s + (layout == SSHDP_SCALE_ROWMAJOR ? row : row >> 5) * KB_;
  };
  int64_t nr[NF];
#pragma unroll
  for (int i = 0; i < NF; ++i) {
    nr[i] = min(nb + 16 * i + r, p.n - 1);
    pb[i] = NN ? p.b + nr[i] : p.b + nr[i] * p.k;
    sb[i] = NN ? p.bs + (nr[i] >> 5) : row_scales(p.bs, p.lb, nr[i], KB, tb);
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t m = min(mb + 16 * j + r, p.m - 1);
    pa[j] = p.a + m * p.k;
    sa[j] = row_scales(p.as, p.la, m, KB, ta);
  }
  f32x4_t acc[NF][MT];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // Steps and chunks past K load nothing and add zeros.
  struct Step {
    i32x8_t b[NF], a[MT];
    uint32_t wb[NF], wa[MT];                         // 8-bit form: block g's byte; else blocks g / 2 and 2 + g / 2
  };
  auto fetch = [&](Step &st, int kt) __attribute__((always_inline)) {
    auto chunks = [&](const uint8_t *q) __attribute__((always_inline)) {
      i32x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)kt * 128 + 64 * h + 16 * g;
        if (k < p.k) {
          const u32x4_t x = *reinterpret_cast<const u32x4_t *>(q + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[4 * h + j] = (int)x[j];
        }
      }
      return v;
    };
    auto byte = [&](const uint8_t *s, int t, int blk) __attribute__((always_inline)) {
      const int kb = 4 * kt + blk;
      return kb < KB ? (uint32_t)s[(kb >> 2) * t + (kb & 3)] : 0u;
    };
    auto byte_nn = [&](const uint8_t *s, int blk) __attribute__((always_inline)) {
      const int kb = 4 * kt + blk;
      return kb < KB ? (uint32_t)s[(int64_t)kb * (p.n >> 5)] : 0u;
    };
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      if (NN) {
        st.b[i] = i32x8_t{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int64_t k = (int64_t)kt * 128 + 64 * (c >> 4) + 16 * g + (c & 15);
          if (k < p.k) st.b[i][c >> 2] |= (int)pb[i][k * p.n] << (8 * (c & 3));
        }
        st.wb[i] = BF16 ? byte_nn(sb[i], g) : byte_nn(sb[i], g >> 1) | byte_nn(sb[i], 2 + (g >> 1)) << 8;
      } else {
        st.b[i] = chunks(pb[i]);
        st.wb[i] = BF16 ? byte(sb[i], tb, g) : byte(sb[i], tb, g >> 1) | byte(sb[i], tb, 2 + (g >> 1)) << 8;
      }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      st.a[j] = chunks(pa[j]);
      st.wa[j] = BF16 ? byte(sa[j], ta, g) : byte(sa[j], ta, g >> 1) | byte(sa[j], ta, 2 + (g >> 1)) << 8;
    }
  };
  auto multiply = [&](const Step &st) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        if (BF16) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(st.b[i], st.a[j], acc[i][j], 0, 0, 0, (int)st.wb[i], 0,
                                                                       (int)st.wa[j]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[i][j] = mma_bf16(to_bf16(st.b[i][2 * c], st.b[i][2 * c + 1], (st.wb[i] >> (8 * (c >> 1))) & 0xFFu),
                                 to_bf16(st.a[j][2 * c], st.a[j][2 * c + 1], (st.wa[j] >> (8 * (c >> 1))) & 0xFFu),
                                 acc[i][j]);
        }
      }
  };
  Step st[2];
  fetch(st[0], wave);
  for (int k0 = wave;;) {
    fetch(st[1], k0 + W);
    multiply(st[0]);
    k0 += W;
    if (k0 >= nk) break;
    fetch(st[0], k0 + W);
    multiply(st[1]);
    k0 += W;
    if (k0 >= nk) break;
  }
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) asm volatile("" : "+v"(acc[i][j]));
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave][i * MT + j][lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < NF * MT; f += W) {
    f32x4_t v = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w][f][lane];
    const int64_t n = nb + 16 * (f / MT) + 4 * g, m = mb + 16 * (f % MT) + r;
    if (BF16) store_bf16(p, m, n, v);
    else store_f32(p, static_cast<float *>(p.out), m, n, v);
  }
}

// Up to 16 rows, K <= 1024 * W: a wave keeps its 8 steps of A in registers and walks groups
// of 16 columns, each 16 codes' slot loaded anew for the next group right after its matrix
// instructions, so B streams without a pause and A is read once a workgroup (16 rows of A per
// 16 of B are as many cache lines again).  The waves' sums of a group are added in wave order
// by one wave, in turn, while the others go on.  Bound by reading B: 1 x 28672 x 8192 42.4 us
// (5.5 TB/s), 16 rows 46.9, float32 output 42.2; split 128-tiles 54.5, 58.6 and 60.6, the
// kernel above 54 to 67; 1 x 2048 x 8192 8.3 against 10.5; a B of under 10 MB gains nothing.  Twice
// the waves with 4 steps each: up to 15% slower (16 x 12288 x 4096: 17.5 against 15.3).
constexpr int kFewSteps = 8;

template <bool BF16, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_gemm_mx_few(GemmMx p, int groups) {
  constexpr int S = kFewSteps;
  typedef uint32_t u32x4u_t __attribute__((ext_vector_type(4), aligned(1)));   // scales lie at any address
  typedef uint32_t u32u_t __attribute__((aligned(1)));
  struct Words {
    uint32_t w[S];
  };
  __shared__ __align__(16) f32x4_t part[2][W][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int KB = (int)(p.k >> 5), kb0 = 4 * S * wave;       // the wave's blocks: 4 S from kb0 on
  const bool full = kb0 + 4 * S <= KB;
  // word j: a row's blocks kb0 + 4 j .. + 3, zeros past the end
  auto scales = [&](const uint8_t *s, int layout, int64_t row) __attribute__((always_inline)) {
    const bool tile = layout == SSHDP_SCALE_TILE32X4;
    s += tile ? (row >> 5) * (KB >> 2) * 128 + (row & 31) * 4 : (layout == SSHDP_SCALE_ROWMAJOR ? row : row >> 5) * KB;
    Words v{};
    if (full && !tile) {
#pragma unroll
      for (int j = 0; j < S; j += 4) {
        const u32x4_t x = *reinterpret_cast<const u32x4u_t *>(s + kb0 + 4 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[j + i] = x[i];
      }
    } else if (full) {
#pragma unroll
      for (int j = 0; j < S; ++j) v.w[j] = *reinterpret_cast<const u32u_t *>(s + ((kb0 >> 2) + j) * 128);
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int kb = kb0 + 4 * j, n = min(KB - kb, 4);
        const uint8_t *q = s + (tile ? (kb >> 2) * 128 : kb);
        if (n == 4) v.w[j] = *reinterpret_cast<const u32u_t *>(q);
        else for (int i = 0; i < n; ++i) v.w[j] |= (uint32_t)q[i] << (8 * i);
      }
    }
    return v;
  };
  // The lane's chunk c (16 bytes) is inside K if 64 c < left; chunks past K and rows past N
  // are sent out of the resource's range, and read as zeros.
  const int k0 = kb0 * 32 + 16 * g, left = (int)p.k - k0, voff = r * (int)p.k + k0;
  auto resource = [&](int grp) __attribute__((always_inline)) {
    const int64_t rows = grp < groups ? min<int64_t>(p.n - grp * 16ll, 16) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.b + (rows ? grp * 16ll * p.k : 0)), 0,
                                             (int)(rows * p.k), kBufWord3);
  };
  auto load = [&](__amdgpu_buffer_rsrc_t rs, int c) __attribute__((always_inline)) {
    return __builtin_bit_cast(u32x4_t,
                              __builtin_amdgcn_raw_buffer_load_b128(rs, 64 * c < left ? voff + 64 * c : INT32_MAX - 15, 0, 0));
  };
  auto b_scales = [&](int grp) __attribute__((always_inline)) { return scales(p.bs, p.lb, min(grp * 16ll + r, p.n - 1)); };
  int grp = blockIdx.x;
  u32x4_t a[2 * S], b[2 * S];
  const __amdgpu_buffer_rsrc_t first = resource(grp);
#pragma unroll
  for (int c = 0; c < 2 * S; ++c) b[c] = load(first, c);
  Words wb = b_scales(grp);
  const int64_t m = min((int64_t)r, p.m - 1);               // rows past the end repeat the last one
#pragma unroll
  for (int c = 0; c < 2 * S; ++c) {
    a[c] = u32x4_t{0, 0, 0, 0};
    if (64 * c < left) a[c] = *reinterpret_cast<const u32x4_t *>(p.a + m * p.k + k0 + 64 * c);
  }
  const Words wa = scales(p.as, p.la, m);
  for (int it = 0; grp < groups; ++it) {
    const int next = grp + gridDim.x;
    const __amdgpu_buffer_rsrc_t rs = resource(next);
    Words wn = wb;
    if (next < groups) wn = b_scales(next);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (BF16) {
        i32x8_t x, y;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (int)b[2 * s + (j >> 2)][j & 3], y[j] = (int)a[2 * s + (j >> 2)][j & 3];
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, (int)(wb.w[s] >> (8 * g)), 0,
                                                               (int)(wa.w[s] >> (8 * g)));
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int h = c >> 1, e = 2 * (c & 1), sh = 8 * (2 * h + (g >> 1));
          acc = mma_bf16(to_bf16((int)b[2 * s + h][e], (int)b[2 * s + h][e + 1], (wb.w[s] >> sh) & 0xFFu),
                         to_bf16((int)a[2 * s + h][e], (int)a[2 * s + h][e + 1], (wa.w[s] >> sh) & 0xFFu), acc);
        }
      }
      b[2 * s] = load(rs, 2 * s);
      b[2 * s + 1] = load(rs, 2 * s + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    part[it & 1][wave][lane] = acc;
    // one barrier a group: a wave that adds up one half passes the next before the half is
    // written again (the barrier builtin would also wait for the loads in flight)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (wave == it % W) {
      f32x4_t v = part[it & 1][0][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) v += part[it & 1][w][lane];
      const int64_t n = grp * 16ll + 4 * g;
      if (BF16) store_bf16(p, r, n, v);
      else store_f32(p, static_cast<float *>(p.out), r, n, v);
    }
    wb = wn;
    grp = next;
  }
}

// ------------------------------------------------------------------ tiled products

// The splits' sums added in split order, 4 consecutive n per thread (1 x 8192 x 28672, eight
// splits: 51.5 us with the tiles, operands from HBM).
template <bool BF16>
__global__ __launch_bounds__(256) void k_gemm_mx_join(GemmMx p, const float *parts, int splits) {
  const int64_t n4 = (p.n + 3) & ~(int64_t)3, words = p.m * (n4 >> 2);
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / (n4 >> 2), n = (i - m * (n4 >> 2)) * 4;
    const f32x4_t *q = reinterpret_cast<const f32x4_t *>(parts) + i;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < splits; s0 += 8) {           // 8 splits' loads in flight
      f32x4_t r[8];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < splits) r[s] = q[(s0 + s) * words];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < splits) v = s0 + s ? v + r[s] : r[s];
    }
    if (BF16) store_bf16(p, m, n, v);
    else store_f32(p, static_cast<float *>(p.out), m, n, v);
  }
}

template <class C, bool NN, bool SHORT>
__global__ __launch_bounds__(C::NT * C::KG) __attribute__((amdgpu_waves_per_eu(C::WPS, C::WPS))) void k_gemm_mx8(GemmMx p, int64_t tiles_m,
                                                                                             int64_t tiles_n, int steps, float *parts) {
  __shared__ __align__(1024) char all[C::LDS];
  int64_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t n0 = tn * C::TN, m0 = tm * C::TM;
  // `steps`: of one wave group.  Groups past the last step run as many, on zeros: the
  // barriers are the whole workgroup's.
  const int grp = C::KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / C::NT) : 0;
  char *smem = all + grp * C::GROUP;
  const int kt0 = (int)blockIdx.y * C::KG * steps;
  const Loader<C, NN> ld(p, n0, m0, kt0 + grp * steps, min(steps, (int)((p.k + kRowB - 1) / kRowB) - kt0));
  const int wn = ld.wave / C::WM, wm = ld.wave % C::WM;
  constexpr int FP = C::FP, FQ = C::FQ;
  f32x4_t acc[FP][FQ];
  sums8<C, NN, SHORT>(ld, smem, acc);
  __syncthreads();

  if (C::KG > 1 && !join_groups<C>(all, grp, acc)) return;
  // the lane again, so that nothing of it is kept in registers over the loop
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  if (parts) {
    store_part<C>(p, parts, n0, m0, wn, wm, t_end & 63, acc);
    return;
  }
  store_tile_bf16<C>(p, smem, n0, m0, wn, wm, t_end, acc);
}

// Float32 output: the same tiles, stages and scale words, with operands converted to
// bfloat16 on their way from LDS to the matrix instructions.  A half step is one 16-byte
// chunk per lane (64 k): its m-side fragments stay converted while the n side's pass by,
// one converted (8 conversions) beside the previous one's 2 x FQ matrix instructions.
// 8192 x 2048 x 4096 with an addend: 117-121 us, 1.2 PFLOP/s of a bfloat16 rate of 1.38 that a
// large library product reaches here; 67 MB of addend in and as much out are 28 us of it,
// which one workgroup a CU hides only in part.
template <class C, bool NN, bool SHORT>
__global__ __launch_bounds__(C::NT * C::KG) __attribute__((amdgpu_waves_per_eu(C::WPS, C::WPS))) void k_gemm_mx16(GemmMx p, int64_t tiles_m,
                                                                                              int64_t tiles_n, int steps, float *parts) {
  __shared__ __align__(1024) char all[C::LDS];
  int64_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t n0 = tn * C::TN, m0 = tm * C::TM;
  // `steps`: of one wave group.  Groups past the last step run as many, on zeros: the
  // barriers are the whole workgroup's.
  const int grp = C::KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / C::NT) : 0;
  char *smem = all + grp * C::GROUP;
  const int kt0 = (int)blockIdx.y * C::KG * steps;
  const Loader<C, NN> ld(p, n0, m0, kt0 + grp * steps, min(steps, (int)((p.k + kRowB - 1) / kRowB) - kt0));
  const int wn = ld.wave / C::WM, wm = ld.wave % C::WM;
  constexpr int FP = C::FP, FQ = C::FQ;
  f32x4_t acc[FP][FQ];
  sums16<C, NN, SHORT>(ld, smem, acc);
  if (C::KG > 1) {
    __syncthreads();
    if (!join_groups<C>(all, grp, acc)) return;
  }
  // the lane again, so that nothing of it is kept in registers over the loop
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  if (parts) {
    store_part<C>(p, parts, n0, m0, wn, wm, t_end & 63, acc);
    return;
  }
  store_tile_f32<C>(p, n0, m0, wn, wm, t_end, acc);
}

template <class C, bool NN>
hipError_t gemm_tiled(const GemmMx &g, int splits, int steps, float *parts, hipStream_t s) {
  const int64_t tm = (g.m + C::TM - 1) / C::TM, tn = (g.n + C::TN - 1) / C::TN;
  const dim3 grid((unsigned)(tm * tn), (unsigned)splits), block(C::NT * C::KG);
  if (splits == 1) parts = nullptr;
  auto launch = [&](auto sh) {
    constexpr bool SHORT = decltype(sh)::value;
    if (g.bf16) hipLaunchKernelGGL((k_gemm_mx8<C, NN, SHORT>), grid, block, 0, s, g, tm, tn, steps, parts);
    else hipLaunchKernelGGL((k_gemm_mx16<C, NN, SHORT>), grid, block, 0, s, g, tm, tn, steps, parts);
  };
  // two wave groups take matrices of more than 4 steps only
  if constexpr (C::KG == 1) {
    if (gemm_short(g.k)) launch(std::true_type{});
    else launch(std::false_type{});
  } else {
    launch(std::false_type{});
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t words = g.m * ((g.n + 3) / 4);
  const dim3 jgrid((unsigned)std::min<int64_t>((words + 255) / 256, 8192)), jblock(256);
  if (g.bf16) hipLaunchKernelGGL((k_gemm_mx_join<true>), jgrid, jblock, 0, s, g, parts, splits);
  else hipLaunchKernelGGL((k_gemm_mx_join<false>), jgrid, jblock, 0, s, g, parts, splits);
  return hipGetLastError();
}

template <bool BF16, int W>
hipError_t gemm_few(const GemmMx &g, hipStream_t s) {
  const int groups = (int)((g.n + 15) / 16);
  // 8 waves a CU, each with 16 KB of B in flight; more groups than that are walked
  hipLaunchKernelGGL((k_gemm_mx_few<BF16, W>), dim3((unsigned)std::min(groups, 256 * 8 / W)), dim3(64 * W), 0, s, g,
                     groups);
  return hipGetLastError();
}

template <bool NN, bool BF16, int W, int NF, int MT>
hipError_t gemm_rows(const GemmMx &g, hipStream_t s) {
  const int64_t tn = (g.n + 16 * NF - 1) / (16 * NF), tm = (g.m + 16 * MT - 1) / (16 * MT);
  const int64_t most = 1 << 22;                        // a launch has under 2^32 threads: outputs past that take several
  for (int64_t first = 0; first < tm * tn; first += most) {
    const dim3 grid((unsigned)std::min(tm * tn - first, most));
    hipLaunchKernelGGL((k_gemm_mx_rows<NN, BF16, W, NF, MT>), grid, dim3(64 * W), 0, s, g, tn, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// What either output type may need.
int64_t gemm_mx_workspace(int64_t m, int64_t n, int64_t k, bool nn) {
  int splits = 1;
  for (const bool bf16 : {false, true}) splits = std::max(splits, gemm_shape_of(m, n, k, nn, bf16).splits);
  return splits > 1 ? splits * m * ((n + 3) / 4 * 4) * (int64_t)sizeof(float) : 0;
}

hipError_t launch_gemm_mx(const GemmMx &g, void *ws, hipStream_t s) {
  const GemmShape sh = gemm_shape_of(g.m, g.n, g.k, g.nn, g.bf16);
  float *parts = static_cast<float *>(ws);
  if (sh.tile == 16) {
    const int waves = gemm_few_waves(g.k);
    if (g.bf16) return waves == 2 ? gemm_few<true, 2>(g, s) : waves == 4 ? gemm_few<true, 4>(g, s) : gemm_few<true, 8>(g, s);
    return waves == 2 ? gemm_few<false, 2>(g, s) : waves == 4 ? gemm_few<false, 4>(g, s) : gemm_few<false, 8>(g, s);
  }
  if (sh.tile == 256)
    return g.nn ? gemm_tiled<T256, true>(g, sh.splits, sh.steps, parts, s)
                : gemm_tiled<T256, false>(g, sh.splits, sh.steps, parts, s);
  if (sh.groups == 2)
    return g.nn ? gemm_tiled<T128K, true>(g, sh.splits, sh.steps, parts, s)
                : gemm_tiled<T128K, false>(g, sh.splits, sh.steps, parts, s);
  if (sh.tile == 128)
    return g.nn ? gemm_tiled<T128, true>(g, sh.splits, sh.steps, parts, s)
                : gemm_tiled<T128, false>(g, sh.splits, sh.steps, parts, s);
  if (g.nn) return g.bf16 ? gemm_rows<true, true, 4, 1, 1>(g, s) : gemm_rows<true, false, 4, 1, 1>(g, s);
  const int rows = gemm_rows_block(g.m);
  if (rows == 16) return g.bf16 ? gemm_rows<false, true, 8, 1, 1>(g, s) : gemm_rows<false, false, 8, 1, 1>(g, s);
  if (rows == 32) return g.bf16 ? gemm_rows<false, true, 8, 1, 2>(g, s) : gemm_rows<false, false, 8, 1, 2>(g, s);
  return g.bf16 ? gemm_rows<false, true, 8, 2, 4>(g, s) : gemm_rows<false, false, 8, 2, 4>(g, s);
}

}  // namespace sshdp
