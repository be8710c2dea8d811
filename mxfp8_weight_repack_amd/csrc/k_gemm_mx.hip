// k_gemm_mx.hip -- MXFP8 products on gfx950's matrix cores.
//
//   out[m][n] = sum over blocks kb of 2^(ea(m, kb) + eb(n, kb)) * sum over the
//   block's 32 k of a(m, k) b(n, k)   (+ addend[m][n]),
//
// a, b E4M3 values, ea, eb the blocks' E8M0 exponents.
//
// bfloat16 output: v_mfma_scale_f32_16x16x128_f8f6f4 (16 x 16 outputs, 128 k, i.e.
// 4 blocks) takes codes and exponent bytes as they lie in memory.  It adds each 8
// consecutive k's products in fixed point, cut off at 2^-14 of the binade of their largest,
// and those sums in float32: a group is off by less than 7 * 2^-14 of its largest product
// (measured about 1.4e-5 rms of a result of random operands, against bfloat16's half step of
// 2^-9 to 2^-8).  That is relative to the products: where they cancel it may pass the
// rounding of the small result, and it is no float32 sum.  So float32
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
#include <type_traits>

#include "gemm_shape.h"
#include "internal.h"

namespace sshdp {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// the output's rows start at any element: its words have an element's alignment, which costs
// the memory pipes little (4096 x 8191 x 2048: bfloat16 70 us, element by element 97; aligned rows of 8192: 64)
typedef uint32_t u32x4e_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2e_t __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4e_t __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kBufWord3 = 0x00020000;                // raw gfx9-family buffer resource

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

// 8 codes (two words) times 2^(byte - 127), as bfloat16, exact.  The conversion reads
// the scale's exponent bits, so byte << 23 is E8M0 from 2^-127 (0) to NaN (255).
__device__ __forceinline__ u32x4_t to_bf16(int w0, int w1, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  bf16x2_t v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false),
                   __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true)};
  return __builtin_bit_cast(u32x4_t, v);
}

__device__ __forceinline__ f32x4_t mma_bf16(const u32x4_t &p, const u32x4_t &q, const f32x4_t &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, p), __builtin_bit_cast(bf16x8_t, q), c, 0, 0, 0);
}

// Four consecutive n of one row m: float32 result, the addend joined in.
__device__ __forceinline__ void store_f32(const GemmMx &p, float *out, int64_t m, int64_t n, f32x4_t v) {
  if (m >= p.m || n >= p.n) return;
  const int64_t e = m * p.ld + n;
  if (n + 4 <= p.n) {
    if (p.addend) v += *reinterpret_cast<const f32x4e_t *>(p.addend + e);
    *reinterpret_cast<f32x4e_t *>(out + e) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.n) out[e + k] = p.addend ? v[k] + p.addend[e + k] : v[k];
  }
}

__device__ __forceinline__ void store_bf16(const GemmMx &p, int64_t m, int64_t n, const f32x4_t &v) {
  if (m >= p.m || n >= p.n) return;
  uint16_t *o = static_cast<uint16_t *>(p.out) + m * p.ld + n;
  const uint32_t x = pk_bf16(v[0], v[1]), y = pk_bf16(v[2], v[3]);
  if (n + 4 <= p.n) {
    *reinterpret_cast<u32x2e_t *>(o) = u32x2e_t{x, y};
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.n) o[k] = (uint16_t)((k < 2 ? x : y) >> (16 * (k & 1)));
  }
}

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
//
// A workgroup makes a TN x TM block of the output (n x m), its waves WN x WM of them
// (TN / WN) x (TM / WM) each, 128 k per step.  Operands go from memory to LDS with
// buffer loads (no registers in between), two stages, each 128-byte row's 16-byte
// chunks XOR-swizzled; the buffer resources end with the operand's last row, so
// rows past it read as zeros, and chunks past K are sent out of range.
//
// Scales: every 4 steps a thread loads one row's 16 scale bytes (4 steps x 4
// blocks), four steps ahead, and a 4 x 4 byte transpose across the lanes 16 and 32
// apart turns each step's 4 bytes into the word the matrix instruction wants: lane
// 16 g + r holds block g's byte of the rows r, 16 + r, 32 + r, 48 + r of its 64-row
// group, picked by the instruction's byte select.
//
// 8192 x 28672 x 8192, bfloat16: 1.43-1.66 ms, 2.3-2.7 PFLOP/s (the clock falls with the data's
// activity), matrix cores busy 68 to 71% of the time.  The rest is operand latency beyond the L2
// (with every load a hit: 1.32 ms) and the scales (without any: 1.38 ms).

constexpr int kRowB = kGemmStep;                     // bytes (= k) of a stage row

// KG groups of WN x WM waves make the same tile over KG parts of its K and add their sums
// in LDS: where there are too few tiles to give every CU two workgroups, a second group takes
// the place of the second workgroup (1999 x 2048 x 8192 NN, operands in the last-level cache:
// 43.9 us, one group 50.3; 26 us at the large product's rate).  Both groups pass the one
// barrier of a step, so they wait for their loads at the same time: matrix cores are 28%
// busy, LDS 17%, and with operands from HBM the same product takes 54 us.
template <int TN_, int TM_, int WN_, int WM_, int KG_>
struct Tile {
  static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_, NW = WN * WM, NT = 64 * NW, KG = KG_, NST = 2;
  static constexpr int FP = TN / WN / 16, FQ = TM / WM / 16;     // 16-row fragments of a wave: n side, m side
  static constexpr int SEGP = TN * kRowB, SEGQ = TM * kRowB, STAGE = SEGP + SEGQ;
  static constexpr int NIP = SEGP / 1024 / NW, NIQ = SEGQ / 1024 / NW;   // buffer loads per wave and stage
  static constexpr int GRPS = (TN + TM) / 64;                   // 64-row scale groups, n side first
  static constexpr int RING = 2 * 4 * GRPS * 64 * 4;            // scale words: 2 x 4 steps
  static constexpr int EPI = TM * (TN + 8) * 2;                 // bfloat16 output tile
  static constexpr int GROUP = NST * STAGE + RING;             // LDS of one wave group
  static constexpr int LDS = KG * GROUP > EPI ? KG * GROUP : EPI;
  static constexpr int WPS = NT * KG * (163840 / LDS) / 256;    // waves per SIMD
  static_assert(FP % 4 == 0 && FQ == 4 && NT == TN + TM, "a thread per scale row, 64-row groups");
  static_assert((NST - 1) * SEGP + SEGP / WN <= 65536, "stages are LDS read offsets");
  static_assert(KG == 1 || (KG == 2 && FP * FQ * 16 * NT <= GROUP), "the other group's sums fit its LDS");
};

// Chunk swizzle of a stage row: 8 consecutive rows, one LDS pass, hit 8 different chunks.
__device__ __forceinline__ int swz(int r) { return r & 7; }

// Bytes (row j = lane / 16, block g) -> lane 16 g + r holds block g's bytes of rows j = 0..3.
__device__ __forceinline__ uint32_t lane_transpose(uint32_t x, int lane) {
  auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);      // [0]: lanes 0..31 twice, [1]: 32..63
  x = __builtin_amdgcn_perm(a[1], a[0], lane < 32 ? 0x05040100u : 0x07060302u);
  auto b = __builtin_amdgcn_permlane16_swap(x, x, false, false);      // [0]: even rows of 16 twice, [1]: odd
  return __builtin_amdgcn_perm(b[1], b[0], lane & 16 ? 0x07030501u : 0x06020400u);
}

// The lane's number anew, for where keeping it would cost a register over the loop.
__device__ __forceinline__ int lane_again() {
  int all = -1;
  asm volatile("" : "+s"(all));
  return __builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}

// One 8-bit matrix instruction; ip, iq: byte selects of the scale words (constants once unrolled).
template <int IP, int IQ>
__device__ __forceinline__ f32x4_t mx_mma(const i32x8_t &p, const i32x8_t &q, const f32x4_t &c, int sp, int sq) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, c, 0, 0, IP, sp, IQ, sq);
}
template <int IP>
__device__ __forceinline__ f32x4_t mx_mma_q(int iq, const i32x8_t &p, const i32x8_t &q, const f32x4_t &c, int sp, int sq) {
  switch (iq) {
    case 0: return mx_mma<IP, 0>(p, q, c, sp, sq);
    case 1: return mx_mma<IP, 1>(p, q, c, sp, sq);
    case 2: return mx_mma<IP, 2>(p, q, c, sp, sq);
    default: return mx_mma<IP, 3>(p, q, c, sp, sq);
  }
}
__device__ __forceinline__ f32x4_t mx_mma_pq(int ip, int iq, const i32x8_t &p, const i32x8_t &q, const f32x4_t &c,
                                             int sp, int sq) {
  switch (ip) {
    case 0: return mx_mma_q<0>(iq, p, q, c, sp, sq);
    case 1: return mx_mma_q<1>(iq, p, q, c, sp, sq);
    case 2: return mx_mma_q<2>(iq, p, q, c, sp, sq);
    default: return mx_mma_q<3>(iq, p, q, c, sp, sq);
  }
}

// Workgroup id -> output tile.  Workgroup i runs on XCD i % 8, each with its own L2:
// each XCD gets one contiguous eighth of an order that walks the tiles in strips of
// 4 along m, so the 32 workgroups an XCD runs at once share 4 + 8 operand panels
// (8192 x 28672 x 8192: 1.43-1.44 ms; strips of 8 1.47, of 16 1.49-1.50).
__device__ __forceinline__ void tile_of(int64_t id, int64_t tiles_m, int64_t tiles_n, int64_t &tm, int64_t &tn) {
  const int64_t total = tiles_m * tiles_n, q = total >> 3, rem = total & 7, x = id & 7;
  const int64_t pos = x * q + min(x, rem) + (id >> 3);
  const int64_t strip = pos / (4 * tiles_n), in = pos - strip * 4 * tiles_n;
  const int64_t h = min<int64_t>(4, tiles_m - strip * 4);
  tn = in / h;
  tm = strip * 4 + in - tn * h;
}

// The same for the n side of NN, whose stage rows are k, TN bytes each.  A transposing read
// takes 16 bytes of 8 consecutive k rows for each 16 lanes, two such groups, 16 rows apart,
// in one LDS pass: their 16 chunks must be all different over two 128-byte halves.
template <int TN>
__device__ __forceinline__ int swz_k(int k) {
  return TN == 256 ? (k & 7) | (k >> 1 & 8) : (k >> 1 & 3) | (k >> 2 & 4);
}

// All of a workgroup's LDS accesses and loads are done, but the newest load if `newest`
// (a constant once unrolled).  The barrier builtin would wait for that one as well.
template <bool SCALES>
__device__ __forceinline__ void stage_barrier(bool newest) {
  if (SCALES && newest) asm volatile("s_waitcnt vmcnt(1) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes per lane from `bytes` of memory at base straight to LDS, lane i at dst + 16 i;
// zeros past the end.  The caller waits
// for it.  PLAIN: the compiler takes a transposing read as one that any load to LDS in
// flight may write under, and puts a wait for all of them before it (NN 8192^3: 401
// against 468 us without); as plain instructions the loads are none of its concern, and M0,
// which they take their LDS address from, is named as overwritten.
template <bool PLAIN>
__device__ __forceinline__ void dma16(const uint8_t *base, int64_t bytes, char *dst, int voff, int soff) {
  if (PLAIN) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const u32x4_t w = {(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, (uint32_t)bytes, (uint32_t)kBufWord3};
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)dst;
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff), "s"(w),
                 "s"(soff)
                 : "m0");
  } else {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, (int)bytes, kBufWord3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
  }
}

// The operand stages' addressing, shared by both matrix forms.
template <class C, bool NN>
struct Loader {
  const GemmMx &p;
  int64_t n0, m0;
  int kt0, nk, last;                                 // this workgroup's steps: kt0 .. kt0 + nk - 1; the matrix's last
  int wave, lane;
  int voffp, voffq;                                  // lane byte offsets
  bool inp, inq;                                     // whether the lane's chunk lies inside the last step
  const uint8_t *gp, *gq;
  const uint8_t *sbase;                              // scales: the wave's 64-row group ...
  int soff, xstep, xlane, xmax, xmul, xend, tshift;  // ... and the lane's address in it
  int narrow;                                        // blocks of a row too short for a 4-byte word, else 0
  static constexpr bool kEnd = NN && C::TN < 256;    // 256-tiles take no NN with N < 128 (and have no register to spare)
  bool xwords;                                       // a step's words lie apart: 4-byte loads
  uint32_t psel;

  __device__ __forceinline__ Loader(const GemmMx &p_, int64_t n0_, int64_t m0_, int kt0_, int nk_)
      : p(p_), n0(n0_), m0(m0_), kt0(kt0_), nk(nk_) {
    const int t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6) % C::NW;
    last = (int)((p.k + kRowB - 1) / kRowB) - 1;
    const int kt = (int)(p.k - (int64_t)last * kRowB);        // k of the last step (a multiple of 32)
    const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz(row);
    voffq = row * (int)p.k + chunk * 16;
    inq = chunk * 16 < kt;
    gq = p.a + m0 * p.k;
    if (NN) {
      constexpr int CPR = C::TN / 16, RPI = 64 / CPR;
      const int kr = RPI * wave + lane / CPR, c = (lane % CPR) ^ swz_k<C::TN>(kr);
      voffp = n0 + c * 16 < p.n ? kr * (int)p.n + c * 16 : INT32_MAX - 15;
      inp = true;                                     // k rows past K are past the resource
      gp = p.b + n0;
    } else {
      voffp = voffq;
      inp = inq;
      gp = p.b + n0 * p.k;
    }
    // Scales: wave = 64-row group, n side first.  A lane reads one row's 4 bytes of a step
    // at sbase + soff + min(min(step * xstep + xlane, xmax) * xmul, xend).  Rows past the end
    // repeat the last one: their codes are zeros and their results unused.
    const bool ps = wave < C::TN / 64;
    const int layout = ps ? p.lb : p.la, KB = (int)(p.k >> 5);
    const int64_t r0 = ps ? n0 + 64 * wave : m0 + 64 * (wave - C::TN / 64);
    // the group's first row, or the last row's block of 32 where the group is past the end
    const int64_t rl = (ps ? p.n : p.m) - 1, rb = min(r0, rl & ~(int64_t)31);
    const int rr = (int)min<int64_t>(lane, rl - rb);
    sbase = ps ? p.bs : p.as;
    xmul = 1;
    xlane = 0;
    xend = INT32_MAX;
    narrow = 0;
    tshift = 0;
    psel = 0;
    xwords = true;
    if (NN && ps) {
      // the group's 64 columns are two blocks: lane 16 g + r reads 4 neighbouring columns'
      // blocks in block row 4 step + g and keeps its two.  Under 4 blocks a row, that word
      // may run into the next row, and from the last one is read from before its place.
      const int NB = (int)(p.n >> 5), nb = min((int)(n0 >> 5) + 2 * wave, NB - 1), first = max(min(nb, NB - 4), 0);
      sbase += first;
      soff = 0;
      xstep = 4;
      xlane = lane >> 4;
      xmax = KB - 1;
      xmul = NB;
      xend = KB * NB - 4 - first;
      psel = (uint32_t)(nb - first) * 0x0101u + (uint32_t)min(nb - first + 1, 3) * 0x01010000u;
    } else if (layout == SSHDP_SCALE_TILE32X4) {
      sbase += (rb >> 5) * (KB >> 2) * 128;
      soff = (rr >> 5) * (KB >> 2) * 128 + (rr & 31) * 4;
      xstep = 128;
      xmax = ((KB >> 2) - 1) * 128;
    } else {
      const int sh = layout == SSHDP_SCALE_ROWMAJOR ? 0 : 5;
      sbase += (rb >> sh) * KB;
      soff = (rr >> sh) * KB;
      xstep = 4;
      xmax = max(KB - 4, 0);
      narrow = KB < 4 ? KB : 0;
      tshift = 8;
      xwords = false;
    }
  }

  // Stages: n side 0, n side 1, m side 0, m side 1 (so a stage is an immediate offset of
  // its LDS reads).  The two sides' loads are issued apart, among matrix instructions: a
  // wave issues in order, and the 8 of one step back to back hold up everything behind
  // them for as long as all waves' loads take to issue.
  __device__ __forceinline__ void load_p(char *smem, int stage, int kt) const {
    kt += kt0;
    const int v = kt < last || (inp && (C::KG == 1 || kt == last)) ? voffp : INT32_MAX - 15;
    char *sp = smem + stage * C::SEGP + wave * 1024;
    const int64_t k0 = (int64_t)kt * kRowB;
    if (NN) {
      constexpr int RPI = 64 / (C::TN / 16);
      int64_t left = (p.k - k0 < kRowB ? p.k - k0 : (int64_t)kRowB) * p.n - n0;
      if (C::KG > 1) left = max(left, (int64_t)0);
#pragma unroll
      for (int i = 0; i < C::NIP; ++i) dma16<NN>(gp + k0 * p.n, left, sp + i * C::NW * 1024, v, i * RPI * C::NW * (int)p.n);
    } else {
      const int64_t rows = p.n - n0 < C::TN ? p.n - n0 : (int64_t)C::TN;
#pragma unroll
      for (int i = 0; i < C::NIP; ++i) dma16<NN>(gp, rows * p.k, sp + i * C::NW * 1024, v, i * 8 * C::NW * (int)p.k + (int)k0);
    }
  }
  __device__ __forceinline__ void load_q(char *smem, int stage, int kt) const {
    kt += kt0;
    const int v = kt < last || (inq && (C::KG == 1 || kt == last)) ? voffq : INT32_MAX - 15;
    char *sq = smem + C::NST * C::SEGP + stage * C::SEGQ + wave * 1024;
    const int64_t rows = p.m - m0 < C::TM ? p.m - m0 : (int64_t)C::TM;
#pragma unroll
    for (int i = 0; i < C::NIQ; ++i) dma16<NN>(gq, rows * p.k, sq + i * C::NW * 1024, v, i * 8 * C::NW * (int)p.k + kt * kRowB);
  }

  // The bytes of this wave's 64 scale rows for steps 4 q .. 4 q + 3 as they lie in memory,
  // lane = row.  Row-contiguous layouts take one 16-byte load (each lane another line, so
  // loads are what counts), from the row's last 16 bytes where fewer are left; SHORT
  // matrices (up to 4 steps, one quad) have too few bytes in a row for that.
  template <bool SHORT>
  __device__ __forceinline__ u32x4_t scales(int q) const {
    u32x4_t w;
    if (SHORT && narrow) {
      w = u32x4_t{0, 0, 0, 0};
      for (int i = 0; i < narrow; ++i) w[0] |= (uint32_t)sbase[soff + i] << (8 * i);
    } else if (SHORT || xwords) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = (kt0 + 4 * q + j) * xstep + xlane;
        uint32_t v;
        __builtin_memcpy(&v, sbase + (uint32_t)(soff + (kEnd ? min(min(x, xmax) * xmul, xend) : min(x, xmax) * xmul)), 4);   // any alignment
        w[j] = v;
      }
    } else {
      __builtin_memcpy(&w, sbase + (uint32_t)(soff + min((kt0 + 4 * q) * 4, xmax - 12)), 16);
    }
    return w;
  }
  // Step 4 q + j's word for the matrix instruction: lane 16 g + r gets block g's bytes of
  // the rows r, 16 + r, 32 + r, 48 + r.
  template <bool SHORT>
  __device__ __forceinline__ void scale_words(const u32x4_t &raw, int q, int lane, uint32_t (&out)[4]) const {
    u32x4_t w = raw;
    // what was read from before its place moves down (no branches here: see pin below);
    // zeros come in beside codes that are all zero
    if (kEnd && wave < C::TN / 64) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] >>= 8 * max(min((kt0 + 4 * q + j) * xstep + xlane, xmax) * xmul - xend, 0);
    } else if (SHORT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] >>= min(max((kt0 + 4 * q + j) * xstep - xmax, 0) * tshift, 24);
    } else {
      const int d = min(max((kt0 + 4 * q) * 4 - (xmax - 12), 0), 15) * tshift;
      const uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
      const uint64_t hs = hi >> (d & 63), ls = (lo >> (d & 63)) | (hi << 1 << (63 - (d & 63)));
      w[0] = (uint32_t)(d < 64 ? ls : hs);
      w[1] = (uint32_t)((d < 64 ? ls : hs) >> 32);
      w[2] = (uint32_t)(d < 64 ? hs : 0);
      w[3] = (uint32_t)((d < 64 ? hs : 0) >> 32);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[j] = NN && wave < C::TN / 64 ? __builtin_amdgcn_perm(w[j], w[j], psel) : lane_transpose(w[j], lane);
  }
};


// The second wave group's sums through LDS to the first, which goes on alone.  The caller
// lets every wave's loads to LDS land and passes a barrier first: the sums take the place of
// stages that other waves' last loads still write and their last fragments are read from.
template <class C>
__device__ __forceinline__ bool join_groups(char *all, int grp, f32x4_t (&acc)[C::FP][C::FQ]) {
  f32x4_t *q = reinterpret_cast<f32x4_t *>(all + C::GROUP) + threadIdx.x % C::NT;
  if (grp == 1) {
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) q[(i * C::FQ + j) * C::NT] = acc[i][j];
  }
  __syncthreads();
  if (grp == 1) return false;
#pragma unroll
  for (int i = 0; i < C::FP; ++i)
#pragma unroll
    for (int j = 0; j < C::FQ; ++j) acc[i][j] += q[(i * C::FQ + j) * C::NT];
  return true;
}

// One K split's sums of a tile, dense M x N4 float32 per split (N4: N to a multiple of 4).
template <class C>
__device__ __forceinline__ void store_part(const GemmMx &p, float *parts, int64_t n0, int64_t m0, int wn, int wm, int lane,
                                           const f32x4_t (&acc)[C::FP][C::FQ]) {
  const int64_t n4 = (p.n + 3) & ~(int64_t)3;
  float *o = parts + (int64_t)blockIdx.y * p.m * n4;
#pragma unroll
  for (int j = 0; j < C::FQ; ++j)
#pragma unroll
    for (int i = 0; i < C::FP; ++i) {
      const int64_t m = m0 + wm * (C::TM / C::WM) + 16 * j + (lane & 15), n = n0 + wn * (C::TN / C::WN) + 16 * i + 4 * (lane >> 4);
      if (m < p.m && n < n4) *reinterpret_cast<f32x4_t *>(o + m * n4 + n) = acc[i][j];
    }
}

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
  const int lane = ld.lane, wave = ld.wave, wn = wave / C::WM, wm = wave % C::WM;
  const int r = lane & 15, g = lane >> 4;
  uint32_t *ring = reinterpret_cast<uint32_t *>(smem + C::NST * C::STAGE);
  constexpr int FP = C::FP, FQ = C::FQ, HP = FP / 2, HQ = FQ / 2;

  // fragment addresses: row 16 i + r of the wave's panel, chunks g and 4 + g
  const int cof = (g ^ swz(r)) * 16;
  const int rowp = (wn * (C::TN / C::WN) + r) * kRowB + cof, rowq = C::NST * C::SEGP + (wm * (C::TM / C::WM) + r) * kRowB + cof;
  // NN: fragment i's 16 columns are one chunk of each k row; a transposing read hands
  // a lane one column's 8 k (rows kb .. kb + 7), read 16 bytes a row by lane pairs
  const int trp = (16 * g + (r >> 1)) * C::TN + ((swz_k<C::TN>(16 * g + (r >> 1)) << 4) ^ (wn * (C::TN / C::WN))) + 8 * (r & 1);

  f32x4_t acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto ldp = [&](int stage, int i) __attribute__((always_inline)) {
    i32x8_t v;
    const char *st = smem + stage * C::SEGP;
    if (NN) {
      typedef int i32x2_t __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
      const char *a = st + (trp ^ (i << 4));
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const i32x2_t w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t *)(a + ((h >> 1) * 64 + (h & 1) * 8) * C::TN));
        v[2 * h] = w[0];
        v[2 * h + 1] = w[1];
      }
    } else {
      const u32x4_t x = *reinterpret_cast<const u32x4_t *>(st + rowp + i * 16 * kRowB);
      const u32x4_t y = *reinterpret_cast<const u32x4_t *>(st + (rowp ^ 64) + i * 16 * kRowB);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = (int)x[k], v[4 + k] = (int)y[k];
    }
    return v;
  };
  auto ldq = [&](int stage, int j) __attribute__((always_inline)) {
    i32x8_t v;
    const char *st = smem + stage * C::SEGQ + j * 16 * kRowB;
    const u32x4_t x = *reinterpret_cast<const u32x4_t *>(st + rowq);
    const u32x4_t y = *reinterpret_cast<const u32x4_t *>(st + (rowq ^ 64));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (int)x[k], v[4 + k] = (int)y[k];
    return v;
  };
  auto lds_scale = [&](int kt, int grp) __attribute__((always_inline)) {
    return (int)ring[((kt & 7) * C::GRPS + grp) * 64 + lane];
  };
  const int gp = wn * (FP / 4), gq = C::TN / 64 + wm;

  // Fragments in registers: P holds half of the n side, its slots reloaded with the other
  // half right after their last use; Q0 and Q1 (by turns) the m side's first pair and second.
  i32x8_t P[HP], Q0[HQ], Q1[HQ];
  int sp[2][FP / 4], sq[2];
  auto put_scales = [&](const u32x4_t &raw, int q) __attribute__((always_inline)) {
    const int lane = lane_again();
    uint32_t w[4];
    ld.template scale_words<SHORT>(raw, q, lane, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) ring[((4 * (q & 1) + j) * C::GRPS + wave) * 64 + lane] = w[j];
  };
  // Control flow lets the compiler move matrix instructions to where their sums are
  // next used, past a barrier: this pins them.
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

  const int nk = ld.nk;
  constexpr int NST = C::NST;
  u32x4_t sw = ld.template scales<SHORT>(0);
  ld.load_p(smem, 0, 0);
  ld.load_q(smem, 0, 0);
  put_scales(sw, 0);
#pragma unroll
  for (int st = 1; st < C::NST; ++st) {
    ld.load_p(smem, st, min(st, nk - 1));
    ld.load_q(smem, st, min(st, nk - 1));
  }
  if (!SHORT) sw = ld.template scales<false>(1);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(0) : "memory");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < HP; ++i) P[i] = ldp(0, i);
#pragma unroll
  for (int j = 0; j < HQ; ++j) Q0[j] = ldq(0, j);
#pragma unroll
  for (int i = 0; i < FP / 4; ++i) sp[0][i] = lds_scale(0, gp + i);
  sq[0] = lds_scale(0, gq);

  constexpr int RP = NN ? 4 : 2;                      // LDS reads of an n-side fragment
  // A quarter of a step: HP x HQ matrix instructions with n-side fragments i0 .. and
  // m-side fragments j0 ...  After a fragment's last use `reload` fills its slot; `nr`
  // other LDS reads and `nv` loads to LDS are spread between the instructions.
  auto mma = [&](int i0, i32x8_t(&Q)[HQ], int j0, const int (&s)[FP / 4], int t, int nr, int nv, bool roll, auto reload)
                 __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HP; ++i) {
#pragma unroll
      for (int j = 0; j < HQ; ++j)
        acc[i0 + i][j0 + j] = mx_mma_pq((i0 + i) & 3, j0 + j, P[i], Q[j], acc[i0 + i][j0 + j], s[(i0 + i) >> 2], t);
      if (roll) P[i] = reload(i);
    }
#pragma unroll
    for (int i = 0; i < HP * HQ; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i % 2 == 0 && i / 2 < nv) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      if (roll && i % HQ == HQ - 1) __builtin_amdgcn_sched_group_barrier(0x100, RP, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto none = [](int) { return i32x8_t{}; };
  // One step: the m side's first pair is in QX, its second goes to QY, then the next
  // step's first.
  auto step = [&](int kt, int q, int phase, i32x8_t(&QX)[HQ], i32x8_t(&QY)[HQ], const int (&s)[FP / 4], int t,
                  int (&sn)[FP / 4], int &tn_) __attribute__((always_inline)) {
    const int stage = phase % NST, next = (phase + 1) % NST;
    // here, where the fewest fragments are held
    if (!SHORT && phase == 3) put_scales(sw, q + 1);
#pragma unroll
    for (int j = 0; j < HQ; ++j) QY[j] = ldq(stage, HQ + j);
    mma(0, QX, 0, s, t, 2 * HQ, 0, false, none);
    mma(0, QY, HQ, s, t, 0, 0, true, [&](int i) __attribute__((always_inline)) { return ldp(stage, HP + i); });
    // every wave has read this step's stage, and the next one has landed: younger is only,
    // in phase 0, the scales' load (or the last of its four)
    stage_barrier<!SHORT>(phase == 0);
    // near the end the reload repeats the last step into a stage nobody reads again
    ld.load_p(smem, stage, min(kt + NST, nk - 1));
#pragma unroll
    for (int i = 0; i < FP / 4; ++i) sn[i] = lds_scale(kt + 1, gp + i);
    tn_ = lds_scale(kt + 1, gq);
    mma(HP, QY, HQ, s, t, FP / 4 + 1, C::NIP, false, none);
    ld.load_q(smem, stage, min(kt + NST, nk - 1));
#pragma unroll
    for (int j = 0; j < HQ; ++j) QY[j] = ldq(next, j);
    mma(HP, QX, 0, s, t, 2 * HQ, C::NIQ, true, [&](int i) __attribute__((always_inline)) { return ldp(next, i); });
    // last of the step's loads, so the next barrier's wait can leave it in flight
    if (!SHORT && phase == 3) {
      pin();
      sw = ld.template scales<false>(q + 2);
    }
  };
  for (int kt = 0, q = 0;; kt += 4, ++q) {
    step(kt, q, 0, Q0, Q1, sp[0], sq[0], sp[1], sq[1]);
    if (kt + 1 >= nk) break;
    step(kt + 1, q, 1, Q1, Q0, sp[1], sq[1], sp[0], sq[0]);
    if (kt + 2 >= nk) break;
    step(kt + 2, q, 2, Q0, Q1, sp[0], sq[0], sp[1], sq[1]);
    if (kt + 3 >= nk) break;
    step(kt + 3, q, 3, Q1, Q0, sp[1], sq[1], sp[0], sq[0]);
    if (kt + 4 >= nk) break;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the trailing reloads
  __syncthreads();

  if (C::KG > 1 && !join_groups<C>(all, grp, acc)) return;
  // the lane again, so that nothing of it is kept in registers over the loop
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  const int r_end = t_end & 15, g_end = t_end >> 4 & 3;
  if (parts) {
    store_part<C>(p, parts, n0, m0, wn, wm, t_end & 63, acc);
    return;
  }
  // bfloat16 tile through LDS (rows m), then whole rows of 16-byte stores
  uint16_t *lt = reinterpret_cast<uint16_t *>(smem);
  constexpr int LP = C::TN + 8;
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const f32x4_t &v = acc[i][j];
      uint2 *d = reinterpret_cast<uint2 *>(lt + (wm * (C::TM / C::WM) + 16 * j + r_end) * LP + wn * (C::TN / C::WN) + 16 * i + 4 * g_end);
      *d = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
    }
  __syncthreads();
  uint16_t *out = static_cast<uint16_t *>(p.out);
  constexpr int CH = C::TN / 8;
  for (int id = t_end; id < C::TM * CH; id += C::NT) {
    const int row = id / CH, c = (id - row * CH) * 8;
    const int64_t m = m0 + row, n = n0 + c;
    if (m >= p.m || n >= p.n) continue;
    const u32x4_t v = *reinterpret_cast<const u32x4_t *>(lt + row * LP + c);
    uint16_t *o = out + m * p.ld + n;
    if (n + 8 <= p.n) {
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4e_t *>(o));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n + k < p.n) o[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
    }
  }
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
  const int lane = ld.lane, wave = ld.wave, wn = wave / C::WM, wm = wave % C::WM;
  const int r = lane & 15, g = lane >> 4;
  uint32_t *ring = reinterpret_cast<uint32_t *>(smem + C::NST * C::STAGE);
  constexpr int FP = C::FP, FQ = C::FQ;
  const int cof = (g ^ swz(r)) * 16;
  const int rowp = (wn * (C::TN / C::WN) + r) * kRowB + cof, rowq = C::NST * C::SEGP + (wm * (C::TM / C::WM) + r) * kRowB + cof;
  const int trp = (16 * g + (r >> 1)) * C::TN + ((swz_k<C::TN>(16 * g + (r >> 1)) << 4) ^ (wn * (C::TN / C::WN))) + 8 * (r & 1);

  f32x4_t acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto ldp = [&](int stage, int h, int i) __attribute__((always_inline)) {
    const char *st = smem + stage * C::SEGP;
    if (NN) {
      typedef int i32x2_t __attribute__((ext_vector_type(2)));
      typedef __attribute__((address_space(3))) i32x2_t lds_i32x2_t;
      const char *a = st + (trp ^ (i << 4)) + h * 64 * C::TN;
      const i32x2_t x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t *)a);
      const i32x2_t y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t *)(a + 8 * C::TN));
      return u32x4_t{(uint32_t)x[0], (uint32_t)x[1], (uint32_t)y[0], (uint32_t)y[1]};
    }
    return *reinterpret_cast<const u32x4_t *>(st + (rowp ^ (h << 6)) + i * 16 * kRowB);
  };
  auto ldq = [&](int stage, int h, int j) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4_t *>(smem + stage * C::SEGQ + (rowq ^ (h << 6)) + j * 16 * kRowB);
  };
  // half h of lane (r, g) lies in block 2 h + g / 2
  const int sl = ((g >> 1) << 4) + r;
  auto lds_scale = [&](int kt, int h, int grp) __attribute__((always_inline)) {
    return ring[((kt & 7) * C::GRPS + grp) * 64 + 32 * h + sl];
  };
  auto convert = [&](const u32x4_t &x, uint32_t word, int byte, u32x4_t(&out)[2]) __attribute__((always_inline)) {
    const uint32_t e = (word >> (8 * byte)) & 0xFFu;
    out[0] = to_bf16((int)x[0], (int)x[1], e);
    out[1] = to_bf16((int)x[2], (int)x[3], e);
  };
  const int gp = wn * (FP / 4), gq = C::TN / 64 + wm;
  auto put_scales = [&](const u32x4_t &raw, int q) __attribute__((always_inline)) {
    const int lane = lane_again();
    uint32_t w[4];
    ld.template scale_words<SHORT>(raw, q, lane, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) ring[((4 * (q & 1) + j) * C::GRPS + wave) * 64 + lane] = w[j];
  };
  // Control flow lets the compiler move matrix instructions to where their sums are
  // next used, past a barrier: this pins them.
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FP; ++i)
#pragma unroll
      for (int j = 0; j < FQ; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

  const int nk = ld.nk;
  constexpr int NST = C::NST;
  u32x4_t sw = ld.template scales<SHORT>(0);
  ld.load_p(smem, 0, 0);
  ld.load_q(smem, 0, 0);
  put_scales(sw, 0);
#pragma unroll
  for (int st = 1; st < C::NST; ++st) {
    ld.load_p(smem, st, min(st, nk - 1));
    ld.load_q(smem, st, min(st, nk - 1));
  }
  if (!SHORT) sw = ld.template scales<false>(1);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();

  u32x4_t P[2], Q[FQ];                                // raw: the next two n-side fragments, the next half's m side
  u32x4_t pc[2][2], qc[FQ][2];                       // converted: this and the next n-side fragment, the m side
  uint32_t sp[2][FP / 4], sq[2];                      // scale words of this half and the next
#pragma unroll
  for (int i = 0; i < FP / 4; ++i) sp[0][i] = lds_scale(0, 0, gp + i);
  sq[0] = lds_scale(0, 0, gq);
#pragma unroll
  for (int j = 0; j < FQ; ++j) Q[j] = ldq(0, 0, j);
  P[0] = ldp(0, 0, 0);
  P[1] = ldp(0, 0, 1);
#pragma unroll
  for (int j = 0; j < FQ; ++j) convert(Q[j], sq[0], j, qc[j]);
  convert(P[0], sp[0][0], 0, pc[0]);

  // Half a step.  Two fragments ahead are read, one ahead is converted; with the last
  // two of the second half, which read the next stage, comes the step's barrier.
  auto half = [&](int kt, int q, int phase, int h) __attribute__((always_inline)) {
    const int stage = phase % NST, ns = h ? (phase + 1) % NST : stage, nh = h ^ 1, nkt = kt + h;
    auto one = [&](int i) __attribute__((always_inline)) {
      // fragment i + 1's conversion, then its slot takes fragment i + 3
      if (i == FP - 2) {
        if (h) {
          // this stage is read, the next has landed
          stage_barrier<!SHORT>(phase == 0);
          ld.load_p(smem, stage, min(kt + NST, nk - 1));
        }
#pragma unroll
        for (int k = 0; k < FP / 4; ++k) sp[nh][k] = lds_scale(nkt, nh, gp + k);
        sq[nh] = lds_scale(nkt, nh, gq);
#pragma unroll
        for (int j = 0; j < FQ; ++j) Q[j] = ldq(ns, nh, j);
      }
      if (i == FP - 1 && h) ld.load_q(smem, stage, min(kt + NST, nk - 1));
      P[i & 1] = i + 2 < FP ? ldp(stage, h, i + 2) : ldp(ns, nh, i + 2 - FP);
      if (i + 1 < FP) convert(P[(i + 1) & 1], sp[h][(i + 1) >> 2], (i + 1) & 3, pc[(i + 1) & 1]);
      else convert(P[0], sp[nh][0], 0, pc[0]);
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        acc[i][j] = mma_bf16(pc[i & 1][0], qc[j][0], acc[i][j]);
        acc[i][j] = mma_bf16(pc[i & 1][1], qc[j][1], acc[i][j]);
        if (i == FP - 1) convert(Q[j], sq[nh], j, qc[j]);
      }
      if (i == FP - 1) {
#pragma unroll
        for (int k = 0; k < 2 * FQ; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
          if (h && k % 2 == 0 && k / 2 < C::NIQ) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      } else {
        __builtin_amdgcn_sched_group_barrier(0x100, NN ? 2 : 1, 0);
#pragma unroll
        for (int k = 0; k < 2 * FQ; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
          if (k & 1) __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
          if (i == FP - 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          if (i == FP - 2 && h && k % 2 == 0 && k / 2 < C::NIP) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    if (!SHORT && phase == 3 && !h) put_scales(sw, q + 1);
#pragma unroll
    for (int i = 0; i < FP; ++i) one(i);
    if (!SHORT && phase == 3 && h) {
      pin();
      sw = ld.template scales<false>(q + 2);
    }
  };
  for (int kt = 0, q = 0;; kt += 4, ++q) {
    half(kt, q, 0, 0);
    half(kt, q, 0, 1);
    if (kt + 1 >= nk) break;
    half(kt + 1, q, 1, 0);
    half(kt + 1, q, 1, 1);
    if (kt + 2 >= nk) break;
    half(kt + 2, q, 2, 0);
    half(kt + 2, q, 2, 1);
    if (kt + 3 >= nk) break;
    half(kt + 3, q, 3, 0);
    half(kt + 3, q, 3, 1);
    if (kt + 4 >= nk) break;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the trailing reloads
  if (C::KG > 1) {
    __syncthreads();
    if (!join_groups<C>(all, grp, acc)) return;
  }
  // the lane again, so that nothing of it is kept in registers over the loop
  int t_end = threadIdx.x;
  asm volatile("" : "+v"(t_end));
  const int r_end = t_end & 15, g_end = t_end >> 4 & 3;
  if (parts) {
    store_part<C>(p, parts, n0, m0, wn, wm, t_end & 63, acc);
    return;
  }
  float *out = static_cast<float *>(p.out);
  const int64_t mw = m0 + wm * (C::TM / C::WM) + r_end, nw = n0 + wn * (C::TN / C::WN) + 4 * g_end;
  if (n0 + C::TN <= p.n) {
    // 16-byte words all inside: one row block's addend words in flight together (rows past
    // the end read the last one)
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const int64_t m = mw + 16 * j, e = m * p.ld + nw;
      if (p.addend) {
        const float *ad = p.addend + min(m, p.m - 1) * p.ld + nw;
        f32x4_t v[FP];
#pragma unroll
        for (int i = 0; i < FP; ++i) v[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4e_t *>(ad + 16 * i));
#pragma unroll
        for (int i = 0; i < FP; ++i) acc[i][j] += v[i];
      }
      if (m < p.m) {
#pragma unroll
        for (int i = 0; i < FP; ++i) *reinterpret_cast<f32x4e_t *>(out + e + 16 * i) = acc[i][j];
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < FQ; ++j)
#pragma unroll
    for (int i = 0; i < FP; ++i) store_f32(p, out, mw + 16 * j, nw + 16 * i, acc[i][j]);
}

using T256 = Tile<256, 256, 2, 4, 1>;
using T128 = Tile<128, 128, 2, 2, 1>;
using T128K = Tile<128, 128, 2, 2, 2>;

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
