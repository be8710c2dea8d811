// gemm_mx.h -- MXFP8 products on gfx950's matrix cores: operands, tiles and their sums, shared by
// the kernels of one product and of products grouped by expert.
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
#pragma once
#include <hip/hip_runtime.h>

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

// What a workgroup's operands are: whole matrices; a gated product, whose n side is two
// matrices of p.n rows, taking turns every 8 * NW rows of a tile's LDS rows; or a range of K
// of wider matrices (rows `pitch` apart, from `start` on, both multiples of 32), whose scales
// are row-major.
enum Form { kWhole, kGated, kRange };
struct GemmPart : GemmMx {
  const uint8_t *b2, *b2s;                           // kGated: the second matrix
  int64_t pitch;                                     // kRange
  int start;
};

// The operand stages' addressing, shared by both matrix forms.
template <class C, bool NN, Form F = kWhole>
struct Loader {
  using Args = std::conditional_t<F == kWhole, GemmMx, GemmPart>;
  const Args &p;
  int64_t n0, m0;
  int kt0, nk, last;                                 // this workgroup's steps: kt0 .. kt0 + nk - 1; the matrix's last
  int wave, lane;
  int voffp, voffq;                                  // lane byte offsets
  bool inp, inq;                                     // whether the lane's chunk lies inside the last step
  const uint8_t *gp, *gq, *gp2;
  const uint8_t *sbase;                              // scales: the wave's 64-row group ...
  int soff, xstep, xlane, xmax, xmul, xend, tshift;  // ... and the lane's address in it
  int narrow;                                        // blocks of a row too short for a 4-byte word, else 0
  static constexpr bool kEnd = NN && C::TN < 256;    // 256-tiles take no NN with N < 128 (and have no register to spare)
  bool xwords;                                       // a step's words lie apart: 4-byte loads
  uint32_t psel;

  __device__ __forceinline__ int64_t pitch() const {
    if constexpr (F == kRange) return p.pitch;
    else return p.k;
  }
  // Bytes of an operand from a tile's first row on.
  __device__ __forceinline__ int64_t span(int64_t rows) const {
    if constexpr (F == kRange) return (rows - 1) * p.pitch + p.k;
    else return rows * p.k;
  }

  // kGated: n0 counts the rows of each of the two matrices.
  __device__ __forceinline__ Loader(const Args &p_, int64_t n0_, int64_t m0_, int kt0_, int nk_)
      : p(p_), n0(n0_), m0(m0_), kt0(kt0_), nk(nk_) {
    const int t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6) % C::NW;
    last = (int)((p.k + kRowB - 1) / kRowB) - 1;
    const int kt = (int)(p.k - (int64_t)last * kRowB);        // k of the last step (a multiple of 32)
    const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz(row);
    voffq = row * (int)pitch() + chunk * 16;
    inq = chunk * 16 < kt;
    gq = p.a + m0 * pitch();
    if constexpr (F == kRange) gq += p.start;
    if (NN) {
      constexpr int CPR = C::TN / 16, RPI = 64 / CPR;
      const int kr = RPI * wave + lane / CPR, c = (lane % CPR) ^ swz_k<C::TN>(kr);
      voffp = n0 + c * 16 < p.n ? kr * (int)p.n + c * 16 : INT32_MAX - 15;
      inp = true;                                     // k rows past K are past the resource
      gp = p.b + n0;
    } else {
      voffp = voffq;
      inp = inq;
      gp = p.b + n0 * pitch();
      if constexpr (F == kRange) gp += p.start;
      if constexpr (F == kGated) gp2 = p.b2 + n0 * p.k;
    }
    // Scales: wave = 64-row group, n side first.  A lane reads one row's 4 bytes of a step
    // at sbase + soff + min(min(step * xstep + xlane, xmax) * xmul, xend).  Rows past the end
    // repeat the last one: their codes are zeros and their results unused.
    const bool ps = wave < C::TN / 64;
    const int layout = ps ? p.lb : p.la, KB = (int)(pitch() >> 5);
    int64_t r0 = ps ? n0 + 64 * wave : m0 + 64 * (wave - C::TN / 64);
    int in = lane;
    bool second = false;                             // kGated: the lane's row is one of the second matrix
    if constexpr (F == kGated) {
      constexpr int H = 8 * C::NW;                   // rows of a turn: 64, or 32 (the wave's halves)
      if (ps) {
        second = H == 64 ? wave & 1 : lane >> 5;
        r0 = n0 + (H == 64 ? 64 * (wave >> 1) : 32 * wave);
        in = lane & (H - 1);
      }
    }
    // the group's first row, or the last row's block of 32 where the group is past the end
    const int64_t rl = (ps ? p.n : p.m) - 1, rb = min(r0, rl & ~(int64_t)31);
    const int rr = (int)min<int64_t>(in, rl - rb);
    sbase = ps ? p.bs : p.as;
    if constexpr (F == kGated) sbase = second ? p.b2s : sbase;
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
    } else if (F == kRange) {
      // words of the range's steps, from the row's last one where that would pass the row's end
      if constexpr (F == kRange) {
        sbase += rb * KB;
        soff = rr * KB;
        xstep = 4;
        xlane = p.start >> 5;
        xmax = KB - 4;
      }
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
      constexpr int TN = F == kGated ? C::TN / 2 : C::TN;
      const int64_t rows = p.n - n0 < TN ? p.n - n0 : (int64_t)TN;
#pragma unroll
      for (int i = 0; i < C::NIP; ++i) {
        const int at = F == kGated ? i >> 1 : i;
        dma16<NN>(F == kGated && (i & 1) ? gp2 : gp, span(rows), sp + i * C::NW * 1024, v, at * 8 * C::NW * (int)pitch() + (int)k0);
      }
    }
  }
  __device__ __forceinline__ void load_q(char *smem, int stage, int kt) const {
    kt += kt0;
    const int v = kt < last || (inq && (C::KG == 1 || kt == last)) ? voffq : INT32_MAX - 15;
    char *sq = smem + C::NST * C::SEGP + stage * C::SEGQ + wave * 1024;
    const int64_t rows = p.m - m0 < C::TM ? p.m - m0 : (int64_t)C::TM;
#pragma unroll
    for (int i = 0; i < C::NIQ; ++i) dma16<NN>(gq, span(rows), sq + i * C::NW * 1024, v, i * 8 * C::NW * (int)pitch() + kt * kRowB);
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
    } else if (F == kRange) {
      // and what lies past the range's end counts as zeros too: it is the next range's
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = (kt0 + 4 * q + j) * 4, in = (int)(p.k >> 5) - x;
        w[j] >>= min(8 * max(x + xlane - xmax, 0), 24);
        w[j] &= in >= 4 ? ~0u : in <= 0 ? 0u : (1u << (8 * in)) - 1;
      }
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

// A tile's sums over a wave group's steps, which must be at least one, by the 8-bit matrix
// instruction.  Every load to LDS has landed when it returns; other waves may still read theirs.
template <class C, bool NN, bool SHORT, class L>
__device__ __forceinline__ void sums8(const L &ld, char *smem, f32x4_t (&acc)[C::FP][C::FQ]) {
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
}

// The same for float32 output: operands converted to bfloat16 on their way from LDS to the
// matrix instructions.  A half step is one 16-byte chunk per lane (64 k): its m-side fragments
// stay converted while the n side's pass by, one converted (8 conversions) beside the previous
// one's 2 x FQ matrix instructions.
// EARLY: the second stage's loads go out before the first scales have come, which saves a trip to
// memory where ranges are short.  `beside` issues BESIDE other loads behind the first two stages';
// the first two steps do not wait for them.
template <class C, bool NN, bool SHORT, bool EARLY, int BESIDE, class L, class B>
__device__ __forceinline__ void sums16(const L &ld, char *smem, f32x4_t (&acc)[C::FP][C::FQ], B beside) {
  const int lane = ld.lane, wave = ld.wave, wn = wave / C::WM, wm = wave % C::WM;
  const int r = lane & 15, g = lane >> 4;
  uint32_t *ring = reinterpret_cast<uint32_t *>(smem + C::NST * C::STAGE);
  constexpr int FP = C::FP, FQ = C::FQ;
  const int cof = (g ^ swz(r)) * 16;
  const int rowp = (wn * (C::TN / C::WN) + r) * kRowB + cof, rowq = C::NST * C::SEGP + (wm * (C::TM / C::WM) + r) * kRowB + cof;
  const int trp = (16 * g + (r >> 1)) * C::TN + ((swz_k<C::TN>(16 * g + (r >> 1)) << 4) ^ (wn * (C::TN / C::WN))) + 8 * (r & 1);

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
  if (!EARLY) put_scales(sw, 0);
#pragma unroll
  for (int st = 1; st < C::NST; ++st) {
    ld.load_p(smem, st, min(st, nk - 1));
    ld.load_q(smem, st, min(st, nk - 1));
  }
  if (EARLY) {
    const u32x4_t first = sw;
    if (!SHORT) sw = ld.template scales<false>(1);
    put_scales(first, 0);
  } else if (!SHORT) {
    sw = ld.template scales<false>(1);
  }
  if constexpr (BESIDE > 0) {
    __builtin_amdgcn_sched_barrier(0);
    beside();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(BESIDE) : "memory");
  } else {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }

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
          if (BESIDE > 0 && kt == 0) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // both stages have landed
          else stage_barrier<!SHORT>(phase == 0);
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
}

template <class C, bool NN, bool SHORT, bool EARLY = false, class L>
__device__ __forceinline__ void sums16(const L &ld, char *smem, f32x4_t (&acc)[C::FP][C::FQ]) {
  sums16<C, NN, SHORT, EARLY, 0>(ld, smem, acc, [] {});
}

// A tile as bfloat16 through LDS (rows m), then whole rows of 16-byte stores.
template <class C>
__device__ __forceinline__ void store_tile_bf16(const GemmMx &p, char *smem, int64_t n0, int64_t m0, int wn, int wm, int t_end,
                                                const f32x4_t (&acc)[C::FP][C::FQ]) {
  constexpr int FP = C::FP, FQ = C::FQ;
  const int r_end = t_end & 15, g_end = t_end >> 4 & 3;
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

// A tile as float32, the addend joined in.
template <class C>
__device__ __forceinline__ void store_tile_f32(const GemmMx &p, int64_t n0, int64_t m0, int wn, int wm, int t_end,
                                               f32x4_t (&acc)[C::FP][C::FQ]) {
  constexpr int FP = C::FP, FQ = C::FQ;
  const int r_end = t_end & 15, g_end = t_end >> 4 & 3;
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

}  // namespace
}  // namespace sshdp
