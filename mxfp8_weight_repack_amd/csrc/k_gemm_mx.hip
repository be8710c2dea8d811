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
          acc = mma_bf16(to_bf16(b[j], b[j + 1], sb), to_bf16(a[j], a[j + 1], sa), acc);
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

constexpr int kBufWord3 = 0x00020000;                // raw gfx9-family buffer resource
constexpr int kRowB = 128;                           // bytes (= k) of a stage row

template <int TN_, int TM_, int WN_, int WM_>
struct Tile {
  static constexpr int TN = TN_, TM = TM_, WN = WN_, WM = WM_, NW = WN * WM, NT = 64 * NW;
  static constexpr int FP = TN / WN / 16, FQ = TM / WM / 16;     // 16-row fragments of a wave: n side, m side
  static constexpr int SEGP = TN * kRowB, SEGQ = TM * kRowB, STAGE = SEGP + SEGQ;
  static constexpr int NIP = SEGP / 1024 / NW, NIQ = SEGQ / 1024 / NW;   // buffer loads per wave and stage
  static constexpr int GRPS = (TN + TM) / 64;                   // 64-row scale groups, n side first
  static constexpr int RING = 2 * 4 * GRPS * 64 * 4;            // scale words: 2 x 4 steps
  static constexpr int EPI = TM * (TN + 8) * 2;                 // bfloat16 output tile
  static constexpr int LDS = 2 * STAGE + RING > EPI ? 2 * STAGE + RING : EPI;
  static_assert(FP % 4 == 0 && FQ == 4 && NT == TN + TM, "a thread per scale row, 64-row groups");
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
// 8 along m, so the 32 workgroups an XCD runs at once share 8 x 4 operand panels.
__device__ __forceinline__ void tile_of(int64_t id, int64_t tiles_m, int64_t tiles_n, int64_t &tm, int64_t &tn) {
  const int64_t total = tiles_m * tiles_n, q = total >> 3, rem = total & 7, x = id & 7;
  const int64_t pos = x * q + min(x, rem) + (id >> 3);
  const int64_t strip = pos / (8 * tiles_n), in = pos - strip * 8 * tiles_n;
  const int64_t h = min<int64_t>(8, tiles_m - strip * 8);
  tn = in / h;
  tm = strip * 8 + in - tn * h;
}

// 16 bytes per lane from memory straight to LDS, lane i at dst + 16 i.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, char *dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}

// The operand stages' addressing, shared by both matrix forms.
template <class C, bool NN>
struct Loader {
  const GemmMx &p;
  int64_t n0, m0;
  int nk;
  int wave, lane;
  int voffp, voffq, tailp, tailq;                    // lane byte offsets; the tail step's
  const uint8_t *gp, *gq;
  const uint8_t *sbase;                              // scales: the wave's 64-row group ...
  int soff, xstep, xlane, xmax, xmul, tshift;        // ... and the lane's address in it
  uint32_t psel;

  __device__ __forceinline__ Loader(const GemmMx &p_, int64_t n0_, int64_t m0_) : p(p_), n0(n0_), m0(m0_) {
    const int t = threadIdx.x;
    lane = t & 63;
    wave = __builtin_amdgcn_readfirstlane(t >> 6);
    nk = (int)((p.k + kRowB - 1) / kRowB);
    const int kt = (int)(p.k - (int64_t)(nk - 1) * kRowB);    // k of the last step (a multiple of 32)
    const int row = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz(row);
    voffq = row * (int)p.k + chunk * 16;
    tailq = chunk * 16 < kt ? voffq : INT32_MAX - 15;
    gq = p.a + m0 * p.k;
    if (NN) {
      // stage rows are k, 256-byte rows of TN columns; chunk c of row k at c ^ (k & 7)
      constexpr int CPR = C::TN / 16, RPI = 64 / CPR;
      const int kr = RPI * wave + lane / CPR, c = (lane % CPR) ^ (kr & 7);
      voffp = n0 + c * 16 < p.n ? kr * (int)p.n + c * 16 : INT32_MAX - 15;
      tailp = voffp;                                  // k rows past K are past the resource
      gp = p.b + n0;
    } else {
      voffp = voffq;
      tailp = tailq;
      gp = p.b + n0 * p.k;
    }
    // Scales: wave = 64-row group, n side first.  A lane reads one row's 4 bytes of a step
    // at sbase + soff + min(step * xstep + xlane, xmax) * xmul.  Rows past the end repeat
    // the last one: their codes are zeros and their results unused.
    const bool ps = wave < C::TN / 64;
    const int layout = ps ? p.lb : p.la, KB = (int)(p.k >> 5);
    const int64_t r0 = ps ? n0 + 64 * wave : m0 + 64 * (wave - C::TN / 64);
    // the group's first row, or the last row's block of 32 where the group is past the end
    const int64_t rl = (ps ? p.n : p.m) - 1, rb = min(r0, rl & ~(int64_t)31);
    const int rr = (int)min<int64_t>(lane, rl - rb);
    sbase = ps ? p.bs : p.as;
    xmul = 1;
    xlane = 0;
    tshift = 0;
    psel = 0;
    if (NN && ps) {
      // the group's 64 columns are two blocks: lane 16 g + r reads 4 neighbouring columns'
      // blocks in block row 4 step + g and keeps its two
      const int NB = (int)(p.n >> 5), nb = min((int)(n0 >> 5) + 2 * wave, NB - 1), first = min(nb, NB - 4);
      sbase += first;
      soff = 0;
      xstep = 4;
      xlane = lane >> 4;
      xmax = KB - 1;
      xmul = NB;
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
      xmax = KB - 4;
      tshift = 8;
    }
  }

  // stages: n side 0, n side 1, m side 0, m side 1 (so a stage is an immediate offset of its LDS reads)
  __device__ __forceinline__ void load(char *smem, int stage, int kt) const {
    const bool last = kt == nk - 1;
    const int vp = last ? tailp : voffp, vq = last ? tailq : voffq;
    char *sp = smem + stage * C::SEGP + wave * 1024, *sq = smem + 2 * C::SEGP + stage * C::SEGQ + wave * 1024;
    const int64_t k0 = (int64_t)kt * kRowB;
    if (NN) {
      constexpr int RPI = 64 / (C::TN / 16);
      const int64_t left = (p.k - k0 < kRowB ? p.k - k0 : (int64_t)kRowB) * p.n - n0;
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(gp + k0 * p.n), 0, (int)left, kBufWord3);
#pragma unroll
      for (int i = 0; i < C::NIP; ++i)
        dma16(r, sp + i * C::NW * 1024,
                                                 vp, i * RPI * C::NW * (int)p.n);
    } else {
      const int64_t rows = p.n - n0 < C::TN ? p.n - n0 : (int64_t)C::TN;
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(gp), 0, (int)(rows * p.k), kBufWord3);
#pragma unroll
      for (int i = 0; i < C::NIP; ++i)
        dma16(r, sp + i * C::NW * 1024,
                                                 vp, i * 8 * C::NW * (int)p.k + (int)k0);
    }
    const int64_t rows = p.m - m0 < C::TM ? p.m - m0 : (int64_t)C::TM;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(gq), 0, (int)(rows * p.k), kBufWord3);
#pragma unroll
    for (int i = 0; i < C::NIQ; ++i)
      dma16(r, sq + i * C::NW * 1024, vq,
                                               i * 8 * C::NW * (int)p.k + (int)k0);
  }

  // The words of this wave's 64 scale rows for steps 4 q .. 4 q + 3, as they lie in
  // memory.  No branches: control flow here would let the compiler move matrix
  // instructions of one phase past the next one's barrier.
  __device__ __forceinline__ u32x4_t scales(int q) const {
    u32x4_t w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = (4 * q + j) * xstep + xlane;
      uint32_t v;
      __builtin_memcpy(&v, sbase + (uint32_t)(soff + min(x, xmax) * xmul), 4);   // any alignment
      w[j] = v;
    }
    return w;
  }
  // One step's word for the matrix instruction: lane 16 g + r gets block g's bytes of the
  // rows r, 16 + r, 32 + r, 48 + r.
  __device__ __forceinline__ uint32_t scale_word(uint32_t x, int step) const {
    // the last word of a row whose blocks are no multiple of 4 was read from its last 4
    // bytes; what the shift brings in scales codes that are all zero
    const uint32_t t = lane_transpose(x >> min(max(step * xstep - xmax, 0) * tshift, 24), lane);
    return NN && wave < C::TN / 64 ? __builtin_amdgcn_perm(x, x, psel) : t;
  }
};

template <class C, bool NN>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_gemm_mx8(GemmMx p, int64_t tiles_m,
                                                                                             int64_t tiles_n) {
  __shared__ __align__(1024) char smem[C::LDS];
  int64_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t n0 = tn * C::TN, m0 = tm * C::TM;
  const Loader<C, NN> ld(p, n0, m0);
  const int lane = ld.lane, wave = ld.wave, wn = wave / C::WM, wm = wave % C::WM;
  const int r = lane & 15, g = lane >> 4;
  uint32_t *ring = reinterpret_cast<uint32_t *>(smem + 2 * C::STAGE);
  constexpr int FP = C::FP, FQ = C::FQ, HP = FP / 2, HQ = FQ / 2;

  // fragment addresses: row 16 i + r of the wave's panel, chunks g and 4 + g
  const int cof = (g ^ swz(r)) * 16;
  const int rowp = (wn * (C::TN / C::WN) + r) * kRowB + cof, rowq = 2 * C::SEGP + (wm * (C::TM / C::WM) + r) * kRowB + cof;
  // NN: fragment i's 16 columns are one chunk of each k row; a transposing read hands
  // a lane one column's 8 k (rows kb .. kb + 7), read 16 bytes a row by lane pairs
  const int trp = (16 * g + (r >> 1)) * C::TN + ((r >> 1) << 4) + 8 * (r & 1) + wn * (C::TN / C::WN);

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
  // half right after their last use; Q0 or Q2 (by turns) and Q1 the m side's two pairs.
  i32x8_t P[HP], Q0[HQ], Q1[HQ], Q2[HQ];
  int sp[2][FP / 4], sq[2];
  auto put_scales = [&](const u32x4_t &w, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ring[((4 * (q & 1) + j) * C::GRPS + wave) * 64 + lane] = ld.scale_word(w[j], 4 * q + j);
  };

  const int nk = ld.nk;
  u32x4_t sw = ld.scales(0);
  ld.load(smem, 0, 0);
  put_scales(sw, 0);
  ld.load(smem, 1, nk > 1 ? 1 : 0);
  sw = ld.scales(1);
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
  // other LDS reads are spread between the instructions.
  auto mma = [&](int i0, i32x8_t(&Q)[HQ], int j0, const int (&s)[FP / 4], int t, int nr, bool roll, auto reload)
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
      if (roll && i % HQ == HQ - 1) __builtin_amdgcn_sched_group_barrier(0x100, RP, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto none = [](int) { return i32x8_t{}; };
  // One step: the m side's first pair is in QX, its second goes to Q1, the next step's
  // first to QZ.
  auto step = [&](int kt, int q, int phase, i32x8_t(&QX)[HQ], i32x8_t(&QZ)[HQ], const int (&s)[FP / 4], int t,
                  int (&sn)[FP / 4], int &tn_) __attribute__((always_inline)) {
    const int stage = phase & 1;
#pragma unroll
    for (int j = 0; j < HQ; ++j) Q1[j] = ldq(stage, HQ + j);
    mma(0, QX, 0, s, t, 2 * HQ, false, none);
    mma(0, Q1, HQ, s, t, 0, true, [&](int i) __attribute__((always_inline)) { return ldp(stage, HP + i); });
    // every wave has read this step's stage, and the next one has landed
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    // near the end the reload repeats the last step into a stage nobody reads again
    ld.load(smem, stage, kt + 2 < nk ? kt + 2 : nk - 1);
    if (phase == 2) put_scales(sw, q + 1);
    if (phase == 3) sw = ld.scales(q + 2);
#pragma unroll
    for (int j = 0; j < HQ; ++j) QZ[j] = ldq(stage ^ 1, j);
#pragma unroll
    for (int i = 0; i < FP / 4; ++i) sn[i] = lds_scale(kt + 1, gp + i);
    tn_ = lds_scale(kt + 1, gq);
    mma(HP, Q1, HQ, s, t, 2 * HQ + FP / 4 + 1, false, none);
    mma(HP, QX, 0, s, t, 0, true, [&](int i) __attribute__((always_inline)) { return ldp(stage ^ 1, i); });
  };
  for (int kt = 0, q = 0;; kt += 4, ++q) {
    step(kt, q, 0, Q0, Q2, sp[0], sq[0], sp[1], sq[1]);
    if (kt + 1 >= nk) break;
    step(kt + 1, q, 1, Q2, Q0, sp[1], sq[1], sp[0], sq[0]);
    if (kt + 2 >= nk) break;
    step(kt + 2, q, 2, Q0, Q2, sp[0], sq[0], sp[1], sq[1]);
    if (kt + 3 >= nk) break;
    step(kt + 3, q, 3, Q2, Q0, sp[1], sq[1], sp[0], sq[0]);
    if (kt + 4 >= nk) break;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the trailing reloads
  __syncthreads();

  // bfloat16 tile through LDS (rows m), then whole rows of 16-byte stores
  uint16_t *lt = reinterpret_cast<uint16_t *>(smem);
  constexpr int LP = C::TN + 8;
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) {
      const f32x4_t &v = acc[i][j];
      uint2 *d = reinterpret_cast<uint2 *>(lt + (wm * (C::TM / C::WM) + 16 * j + r) * LP + wn * (C::TN / C::WN) + 16 * i + 4 * g);
      *d = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
    }
  __syncthreads();
  uint16_t *out = static_cast<uint16_t *>(p.out);
  constexpr int CH = C::TN / 8;
  for (int id = threadIdx.x; id < C::TM * CH; id += C::NT) {
    const int row = id / CH, c = (id - row * CH) * 8;
    const int64_t m = m0 + row, n = n0 + c;
    if (m >= p.m || n >= p.n) continue;
    const u32x4_t v = *reinterpret_cast<const u32x4_t *>(lt + row * LP + c);
    uint16_t *o = out + m * p.ld + n;
    if (n + 8 <= p.n && p.ld % 8 == 0) {
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t *>(o));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n + k < p.n) o[k] = (uint16_t)(v[k >> 1] >> (16 * (k & 1)));
    }
  }
}

// Four consecutive n of one row m: float32 result, the addend joined in.  `vec`: rows
// are 16-byte multiples, so four in range go out together.
__device__ __forceinline__ void store_f32(const GemmMx &p, float *out, int64_t m, int64_t n, f32x4_t v, bool vec) {
  if (m >= p.m || n >= p.n) return;
  const int64_t e = m * p.ld + n;
  if (vec && n + 4 <= p.n) {
    if (p.addend) v += *reinterpret_cast<const f32x4_t *>(p.addend + e);
    *reinterpret_cast<f32x4_t *>(out + e) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < p.n) out[e + k] = p.addend ? v[k] + p.addend[e + k] : v[k];
  }
}

// Float32 output: the same tiles, stages and scale words, with operands converted to
// bfloat16 on their way from LDS to the matrix instructions.  A half step is one 16-byte
// chunk per lane (64 k): its m-side fragments stay converted while the n side's pass by,
// one converted (8 conversions) beside the previous one's 2 x FQ matrix instructions.
template <class C, bool NN>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_gemm_mx16(GemmMx p, int64_t tiles_m,
                                                                                              int64_t tiles_n) {
  __shared__ __align__(1024) char smem[C::LDS];
  int64_t tm, tn;
  tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t n0 = tn * C::TN, m0 = tm * C::TM;
  const Loader<C, NN> ld(p, n0, m0);
  const int lane = ld.lane, wave = ld.wave, wn = wave / C::WM, wm = wave % C::WM;
  const int r = lane & 15, g = lane >> 4;
  uint32_t *ring = reinterpret_cast<uint32_t *>(smem + 2 * C::STAGE);
  constexpr int FP = C::FP, FQ = C::FQ;
  const int cof = (g ^ swz(r)) * 16;
  const int rowp = (wn * (C::TN / C::WN) + r) * kRowB + cof, rowq = 2 * C::SEGP + (wm * (C::TM / C::WM) + r) * kRowB + cof;
  const int trp = (16 * g + (r >> 1)) * C::TN + ((r >> 1) << 4) + 8 * (r & 1) + wn * (C::TN / C::WN);

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
  auto put_scales = [&](const u32x4_t &w, int q) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ring[((4 * (q & 1) + j) * C::GRPS + wave) * 64 + lane] = ld.scale_word(w[j], 4 * q + j);
  };

  const int nk = ld.nk;
  u32x4_t sw = ld.scales(0);
  ld.load(smem, 0, 0);
  put_scales(sw, 0);
  ld.load(smem, 1, nk > 1 ? 1 : 0);
  sw = ld.scales(1);
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
    const int stage = phase & 1, ns = h ? stage ^ 1 : stage, nh = h ^ 1, nkt = kt + h;
    auto one = [&](int i) __attribute__((always_inline)) {
      // fragment i + 1's conversion, then its slot takes fragment i + 3
      if (i == FP - 2) {
        if (h) {
          asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
          __syncthreads();                            // this stage is read, the next has landed
          ld.load(smem, stage, kt + 2 < nk ? kt + 2 : nk - 1);
          if (phase == 2) put_scales(sw, q + 1);
          if (phase == 3) sw = ld.scales(q + 2);
        }
#pragma unroll
        for (int k = 0; k < FP / 4; ++k) sp[nh][k] = lds_scale(nkt, nh, gp + k);
        sq[nh] = lds_scale(nkt, nh, gq);
#pragma unroll
        for (int j = 0; j < FQ; ++j) Q[j] = ldq(ns, nh, j);
      }
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
        }
      } else {
        __builtin_amdgcn_sched_group_barrier(0x100, NN ? 2 : 1, 0);
#pragma unroll
        for (int k = 0; k < 2 * FQ; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
          if (k & 1) __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
          if (i == FP - 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int i = 0; i < FP; ++i) one(i);
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
  float *out = static_cast<float *>(p.out);
  const bool vec = p.ld % 4 == 0;
#pragma unroll
  for (int j = 0; j < FQ; ++j)
#pragma unroll
    for (int i = 0; i < FP; ++i)
      store_f32(p, out, m0 + wm * (C::TM / C::WM) + 16 * j + r, n0 + wn * (C::TN / C::WN) + 16 * i + 4 * g, acc[i][j], vec);
}

using T256 = Tile<256, 256, 2, 4>;

template <class C, bool NN>
hipError_t gemm_tiled(const GemmMx &g, hipStream_t s) {
  const int64_t tm = (g.m + C::TM - 1) / C::TM, tn = (g.n + C::TN - 1) / C::TN;
  if (g.bf16) hipLaunchKernelGGL((k_gemm_mx8<C, NN>), dim3((unsigned)(tm * tn)), dim3(C::NT), 0, s, g, tm, tn);
  else hipLaunchKernelGGL((k_gemm_mx16<C, NN>), dim3((unsigned)(tm * tn)), dim3(C::NT), 0, s, g, tm, tn);
  return hipGetLastError();
}

}  // namespace

int64_t gemm_mx_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_gemm_mx(const GemmMx &g, void *, hipStream_t s) {
  if (g.k >= 128 && g.m >= 128 && g.n >= 128) return g.nn ? gemm_tiled<T256, true>(g, s) : gemm_tiled<T256, false>(g, s);
  const int64_t tm = (g.m + 15) / 16, tn = (g.n + 15) / 16;
  const dim3 grid((unsigned)(tm * tn)), block(64);
  if (g.nn && g.bf16) hipLaunchKernelGGL((k_gemm_mx_16<true, true>), grid, block, 0, s, g, tn);
  else if (g.nn) hipLaunchKernelGGL((k_gemm_mx_16<true, false>), grid, block, 0, s, g, tn);
  else if (g.bf16) hipLaunchKernelGGL((k_gemm_mx_16<false, true>), grid, block, 0, s, g, tn);
  else hipLaunchKernelGGL((k_gemm_mx_16<false, false>), grid, block, 0, s, g, tn);
  return hipGetLastError();
}

}  // namespace sshdp
