// k_moe.hip -- tokens to the experts' rows and back: the slots' order by expert, rows
// gathered into that order with G behind, the weighted sum back to the tokens, and the
// weights' gradient.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "moe.h"
#include "mx_encode.h"

namespace sshdp {
namespace {

// --------------------------------------------------------------------- slots by expert

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortOnce = 2048;                      // slots that one workgroup sorts alone
constexpr int kSortMostChunks = 256;

// Slots a workgroup takes, a power of two from 1024 (one for each lane) on: all of up to 2048,
// else the fewest that leave at most 256 workgroups, each of which reads every other's counts.
// Bound by trips to memory and barriers.  Of 64 experts: 512 slots 4.1 us by one workgroup with
// a slot a lane, 7.0 with four; 2048 slots 5.9 by one, 6.8 in two launches; 4096 8.7 and 6.9; 98286
// 8.1 (2.6 + 6.2 traced), of 1.6 MB, 0.3 us at a copy's rate.
int64_t sort_chunk(int64_t slots) {
  int64_t c = kSortThreads;
  if (slots <= kSortOnce) {
    while (c < slots) c *= 2;
    return c;
  }
  while ((slots + c - 1) / c > kSortMostChunks) c *= 2;
  return c;
}

// The slot's expert, `experts` where it has none or lies past the end.
template <class I>
__device__ __forceinline__ int expert_of(const I *ids, int64_t slot, int64_t slots, int experts) {
  if (slot >= slots) return experts;
  const I id = ids[slot];
  return id >= 0 && id < (I)experts ? (int)id : experts;
}

template <class I>
__global__ __launch_bounds__(kSortThreads) void k_moe_count(const I *ids, int64_t slots, int experts, int64_t chunk,
                                                            int32_t *counts) {
  __shared__ int n[kMoeMaxExperts + 1];
  const int t = threadIdx.x;
  for (int e = t; e <= experts; e += kSortThreads) n[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk;
  for (int64_t i = t; i < chunk; i += kSortThreads) {
    const int e = expert_of(ids, first + i, slots, experts);
    if (e < experts) atomicAdd(&n[e], 1);             // whole numbers: any order gives the same
  }
  __syncthreads();
  for (int e = t; e < experts; e += kSortThreads) counts[(int64_t)blockIdx.x * experts + e] = n[e];
}

// The lanes whose key is the caller's; every lane of the wave must call it.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = key >> b & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Between LDS accesses of lanes of one wave to what other lanes of it read or wrote: the compiler
// keeps their order.  No instruction comes of it, a wave's LDS accesses are done in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A workgroup places its chunk's slots: a wave takes consecutive ones, counts its slots of
// each expert 64 at a time (a lane's rank among the 64 is the number of lower lanes with its
// expert), the waves' counts become first rows, and the same passes over the slots hand the
// rows out.  Slots of one expert so keep their order, with no atomics.
template <class I>
__global__ __launch_bounds__(kSortThreads) void k_moe_place(const I *ids, int64_t slots, int experts, int align,
                                                            int64_t rows, int64_t chunk, const int32_t *counts,
                                                            int32_t *offsets, int32_t *place, int32_t *source) {
  __shared__ int next[kSortWaves][kMoeMaxExperts];    // counts, then each wave's next row of each expert
  __shared__ int total[kMoeMaxExperts], before[kMoeMaxExperts], first_row[kMoeMaxExperts + 1], sums[kSortWaves];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int bits = 32 - __builtin_clz(experts);       // of the keys 0 .. experts
  for (int e = lane; e < experts; e += 64) next[wave][e] = 0;
  for (int e = t; e < experts; e += kSortThreads) total[e] = before[e] = 0;
  __syncthreads();
  const int64_t per = chunk / kSortWaves, s0 = blockIdx.x * chunk + wave * per;
  const uint64_t lower = (1ull << lane) - 1;
  for (int64_t i = 0; i < per; i += 64) {
    if (s0 + i >= slots) break;
    const int e = expert_of(ids, s0 + i + lane, slots, experts);
    const uint64_t m = same_key(e, bits);
    if (e < experts && !(m & lower)) next[wave][e] += __popcll(m);
    wave_order();
  }
  if (counts) {
    // all chunks' counts, and those of the chunks before this one
    const int pitch = experts <= 64 ? 64 : experts <= 256 ? 256 : 1024;
    const int e = t % pitch, parts = kSortThreads / pitch;
    if (e < experts) {
      int all = 0, mine = 0;
      for (int c0 = t / pitch; c0 < (int)gridDim.x; c0 += 8 * parts) {
        int v[8];                                     // in flight together
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i * parts < (int)gridDim.x ? counts[(int64_t)(c0 + i * parts) * experts + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          all += v[i];
          mine += c0 + i * parts < (int)blockIdx.x ? v[i] : 0;
        }
      }
      atomicAdd(&total[e], all);
      atomicAdd(&before[e], mine);
    }
  }
  __syncthreads();
  // experts' first rows: an exclusive sum of their rows, one expert a thread
  int n = 0;
  if (t < experts) {
    if (counts) {
      n = total[t];
    } else {
      for (int w = 0; w < kSortWaves; ++w) n += next[w][t];
      total[t] = n;
    }
  }
  const int size = (n + align - 1) / align * align;
  int x = size;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) sums[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += sums[w];
  if (t < experts) {
    first_row[t] = x - size;
    if (t == experts - 1) first_row[experts] = x;
    int at = x - size + before[t];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = next[w][t];
      next[w][t] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t i = 0; i < per; i += 64) {
    const int64_t s = s0 + i + lane;
    if (s0 + i >= slots) break;
    const int e = expert_of(ids, s, slots, experts);
    const uint64_t m = same_key(e, bits);
    int at = -1;
    if (e < experts) {
      at = next[wave][e] + __popcll(m & lower);
      source[at] = (int)s;
    }
    // the lanes of one expert have read its next row before their first one moves it
    wave_order();
    if (e < experts && !(m & lower)) next[wave][e] = at + __popcll(m);
    wave_order();
    if (s < slots) place[s] = at;
  }
  if (blockIdx.x == 0)
    for (int e = t; e <= experts; e += kSortThreads) offsets[e] = first_row[e];
  // padding behind each expert's slots, and what is behind the last expert
  const int lanes = (int)gridDim.x * kSortThreads, id = blockIdx.x * kSortThreads + t;
  if (align > 1)
    for (int e = blockIdx.x * kSortWaves + wave; e < experts; e += (int)gridDim.x * kSortWaves)
      for (int r = first_row[e] + total[e] + lane; r < first_row[e + 1]; r += 64) source[r] = -1;
  for (int64_t r = first_row[experts] + (int64_t)id; r < rows; r += lanes) source[r] = -1;
}

// ---------------------------------------------------------------------- rows gathered

// The token of slot `slot`, -1 for padding.
__device__ __forceinline__ int token_of(const sshdp_moe_gather &a, int slot) {
  return slot >= 0 && slot < a.tokens * a.top_k ? (int)((uint32_t)slot / (uint32_t)a.top_k) : -1;
}

// Rows in use, whatever the offsets hold.
__device__ __forceinline__ int64_t rows_in_use(const sshdp_moe_gather &a) {
  return min((int64_t)max(a.offsets[a.experts], 0), a.rows);
}

constexpr int kMrRuns = 4;                           // runs of 8 elements a lane has in flight

// y, and the codes along the rows if wanted: 8 elements a lane and 4 lanes a block, 1024
// consecutive runs of all rows a workgroup.  A run waits for its row's source and then for the
// token: four of them together.
template <bool BF16, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_moe_rows(sshdp_moe_gather a, uint32_t runs_per_row) {
  const int64_t used = rows_in_use(a), first = blockIdx.x * (int64_t)(256 * kMrRuns), row0 = first / runs_per_row;
  const uint32_t rem = (uint32_t)(first - row0 * runs_per_row);
  int64_t row[kMrRuns];
  uint32_t run[kMrRuns];
  int slot[kMrRuns];
#pragma unroll
  for (int u = 0; u < kMrRuns; ++u) {
    const uint32_t x = rem + u * 256 + threadIdx.x, q = x / runs_per_row;
    row[u] = row0 + q;
    run[u] = x - q * runs_per_row;
    slot[u] = row[u] < a.rows ? a.source[row[u]] : -1;
  }
  Raw8<BF16> raw[kMrRuns];
  float w[kMrRuns];
#pragma unroll
  for (int u = 0; u < kMrRuns; ++u) {
    const int token = token_of(a, slot[u]);
    raw[u] = Raw8<BF16>{};
    w[u] = 0.f;
    if (token >= 0) {
      if (WEIGHTED) w[u] = a.weights[slot[u]];
      raw[u] = load8<BF16>(a.x, token * a.ld_x + run[u] * 8);
    }
  }
#pragma unroll
  for (int u = 0; u < kMrRuns; ++u) {
    const int64_t e = row[u] * runs_per_row + run[u];   // blocks are whole in or out: 4 runs each
    const bool in = row[u] < used;
    float v[8];
    if (WEIGHTED) {
      unpack8<BF16>(raw[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= w[u];
      if (in) store8<BF16>(a.y, e * 8, pack8<BF16>(v));
    } else if (in) {
      store8<BF16>(a.y, e * 8, raw[u]);
    }
    if (!a.out.codes) continue;
    uint32_t sb;
    const u32x2_t c = WEIGHTED ? mx_codes4(v, sb) : mx_codes4_raw<BF16>(raw[u], sb);
    if (!in) continue;
    *reinterpret_cast<u32x2_t *>(a.out.codes + e * 8) = c;
    if ((threadIdx.x & 3) == 0) a.out.scales[e >> 2] = (uint8_t)sb;
  }
}

constexpr int kMtRows = 128, kMtCols = 128;          // tile of one workgroup
// Runs only with y wanted, whose stores weigh more than a tile's few of the codes, and only where
// tiles are few: 960 x 8192 (512 tiles) 7.0 us by runs and 6.9 by tiles, float32 13.3 and 17.6;
// 960 x 2048 (128) 4.6 and 5.1, 6.2 and 8.2; 7680 x 2048 (960) 11.5 and 11.9, 30.6 and 31.1; 24558 x
// 2048 36.9 and 34.2, 86 and 81.  Codes alone 960 x 8192 6.3 and 4.7, 96 x 2048 4.0 and 3.7.
constexpr int64_t kMtLeast = 768;

// Column tiles side by side that an XCD takes row by row: two, where there are results along the
// rows, whose runs of memory are then twice as long, and where half the L2 holds that much of x.
// 24558 rows of 4093 bfloat16 tokens x 2048, both ways, 26 us, a column tile at a time 29; of 8192
// tokens 52 and 51, 16384 129 and 124.
uint32_t moe_band(const sshdp_moe_gather &a) {
  const int64_t x = a.tokens * 2 * kMtCols * (a.dtype == SSHDP_DTYPE_BF16 ? 2 : 4);
  return (a.y || a.out.codes) && x <= 2 << 20 ? 2 : 1;
}

// Tiles, wherever runs do not serve better: the tile of k_quant_tiles (LDS
// columns rotated by the row group, a lane two columns' 32 rows), its rows fetched by `source`,
// their weights beside them.  A token is read once for each of its choices, by rows far apart:
// XCD i % 8 takes a contiguous eighth of the tiles, one or two columns of them at a time, so that
// what it reads of x meanwhile, 128 or 256 columns of all tokens, stays in its L2 (24558 x 2048
// bfloat16 of 4093 tokens, both ways 26 us, 119 MB at 4.6 TB/s, nearly all of it writes; with rows
// tile by tile, before stores were as wide, 46 against 31).
// Along the rows a lane takes 16 elements, 16 codes a store, and keeps the scales of its rows'
// four blocks until one store has them all: a store instruction's cost does not go by its bytes.
template <bool BF16, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_moe_tiles(sshdp_moe_gather a, uint32_t tiles_r, uint32_t tiles,
                                                   uint32_t band) {
  constexpr int ES = BF16 ? 2 : 4, ROT = BF16 ? 32 : 16, NP = kMtRows / 32;
  __shared__ __align__(16) char sm[kMtRows * kMtCols * ES];
  __shared__ float sw[WEIGHTED ? kMtRows : 1];
  const int t = threadIdx.x;
  const uint32_t xcd = blockIdx.x & 7, pos = xcd * (tiles >> 3) + min(xcd, tiles & 7) + (blockIdx.x >> 3);
  const uint32_t b = pos / (tiles_r * band), in_b = pos - b * tiles_r * band, wide = min(band, tiles / tiles_r - b * band);
  const int64_t r0 = in_b / wide * (int64_t)kMtRows, c0 = (b * band + in_b % wide) * (int64_t)kMtCols;
  const int lc = (t & 7) * 16, lr = t >> 3;
  const bool in_c = c0 + lc < a.cols;
  int slot[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int64_t r = r0 + lr + 32 * p;
    slot[p] = r < a.rows ? a.source[r] : -1;
  }
  const int64_t used = rows_in_use(a);
  if (r0 >= used) return;
  Raw8<BF16> raw[NP][2];
  float w[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int token = r0 + lr + 32 * p < used ? token_of(a, slot[p]) : -1;
    raw[p][0] = raw[p][1] = Raw8<BF16>{};
    w[p] = 0.f;
    if (token >= 0) {
      if (WEIGHTED) w[p] = a.weights[slot[p]];
      if (in_c) {
        raw[p][0] = load8<BF16>(a.x, token * a.ld_x + c0 + lc);
        raw[p][1] = load8<BF16>(a.x, token * a.ld_x + c0 + lc + 8);
      }
    }
  }
  uint32_t sbs = 0;                                  // lane p of 8: the scales of its row of pass p
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int rr = lr + 32 * p;
    if (a.out.codes_t) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<Raw8<BF16> *>(sm + (rr * kMtCols + ((lc + 8 * h) ^ (p * ROT))) * ES) = raw[p][h];
      if (WEIGHTED && lc == 0) sw[rr] = w[p];
    }
    const bool in = in_c && r0 + rr < used;
    const int64_t e = (r0 + rr) * a.cols + c0 + lc;
    float v[16];
    if (WEIGHTED) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[8];
        unpack8<BF16>(raw[p][h], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * h + j] = x[j] *= w[p];
        if (a.y) raw[p][h] = pack8<BF16>(x);
      }
    }
    if (a.y) {
      if constexpr (BF16) {
        u32x4r_t x[2];
        mx_in_runs(raw[p][0].w, raw[p][1].w, t, x);
        u32x4r_t *d = reinterpret_cast<u32x4r_t *>(static_cast<uint16_t *>(a.y) + e - (t & 3) * 16) + (t & 3);
        const int64_t c = c0 + (lc & ~63);             // the four lanes' first column: a store is a block of 32
        // ordinary stores: nontemporal ones made y alone 32 us instead of 24
        if (r0 + rr < used && c < a.cols) *d = x[0];
        if (r0 + rr < used && c + 32 < a.cols) d[4] = x[1];
      } else if (in) {                               // ordinary stores: the L2 puts the lines together
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<u32x4r_t *>(static_cast<float *>(a.y) + e)[k] = raw[p][k >> 1].w[k & 1];
      }
    }
    if (!a.out.codes) continue;
    uint32_t sb;
    const u32x4r_t x = WEIGHTED ? mx_codes2(v, sb) : mx_codes2_raw<BF16>(raw[p], sb);
    if (in) __builtin_nontemporal_store(x, reinterpret_cast<u32x4r_t *>(a.out.codes + e));
    // the row's four scale bytes in a word, in all of its 8 lanes
    uint32_t q = sb << (8 * ((t & 7) >> 1));
    q |= (uint32_t)__builtin_amdgcn_mov_dpp((int)q, 0x4E, 0xF, 0xF, true);        // quad_perm [2, 3, 0, 1]
    q |= (uint32_t)__builtin_amdgcn_mov_dpp((int)q, 0x141, 0xF, 0xF, true);       // row_half_mirror
    if ((t & 7) == p) sbs = q;
  }
  if (a.out.codes && (t & 7) < NP) {
    typedef uint32_t u32u_t __attribute__((aligned(1)));
    const int64_t r = r0 + lr + 32 * (t & 7);
    uint8_t *d = a.out.scales + r * (a.cols >> 5) + (c0 >> 5);
    const int n = (int)min<int64_t>(4, (a.cols - c0) >> 5);
    if (r < used) {
      if (n == 4) *reinterpret_cast<u32u_t *>(d) = sbs;
      else for (int k = 0; k < n; ++k) d[k] = (uint8_t)(sbs >> (8 * k));
    }
  }
  if (!a.out.codes_t) return;
  __syncthreads();
  const int grp = t & 3, c = (t >> 2) * 2;
  if (c0 + c >= a.cols) return;
  const int blocks = (int)min<int64_t>(4, (used - r0 + 31) / 32);
  const char *q = sm + (32 * grp * kMtCols + (c ^ (grp * ROT))) * ES;
  MxColumn o[2];
  if constexpr (BF16 && !WEIGHTED) {
    uint32_t x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = *reinterpret_cast<const uint32_t *>(q + j * kMtCols * ES);
    mx_columns_bf16(x, o);
  } else {
    float v[2][32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (BF16) {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(q + j * kMtCols * ES);
        v[0][j] = __uint_as_float(x << 16);
        v[1][j] = __uint_as_float(x & 0xFFFF0000u);
      } else {
        const float2 x = *reinterpret_cast<const float2 *>(q + j * kMtCols * ES);
        v[0][j] = x.x;
        v[1][j] = x.y;
      }
      if (WEIGHTED) {
        const float wj = sw[32 * grp + j];
        v[0][j] *= wj;
        v[1][j] *= wj;
      }
    }
    o[0] = mx_column(v[0]);
    o[1] = mx_column(v[1]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e = (c0 + c + h) * a.rows + r0;
    mx_store_column(o[h], a.out.codes_t + e, blocks, t);
    if (grp < blocks) a.out.scales_t[(e >> 5) + grp] = (uint8_t)o[h].scale;
  }
}

// --------------------------------------------------------------------- back to the tokens

constexpr int kCombineAt = 8;                        // choices whose rows are in flight together

// 8 elements of a token a lane: its choices' rows are read together and added in order.  Bound by
// HBM: 8191 tokens of 6 choices, 2048 bfloat16 and a residual 48 us, 5.5 TB/s.
template <bool BF16>
__global__ __launch_bounds__(256) void k_moe_combine(sshdp_moe_combine_args a, int runs_per_row) {
  const int64_t runs = a.tokens * runs_per_row;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < runs; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / runs_per_row, c = (i - t * runs_per_row) * 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.top_k; j0 += kCombineAt) {
      Raw8<BF16> raw[kCombineAt];
      float w[kCombineAt];
      bool have[kCombineAt];
#pragma unroll
      for (int j = 0; j < kCombineAt; ++j) {
        have[j] = false;
        if (j0 + j < a.top_k) {
          const int64_t s = t * a.top_k + j0 + j;
          const int p = a.place[s];
          have[j] = p >= 0 && p < a.rows;
          if (have[j]) {
            w[j] = a.weights ? a.weights[s] : 1.f;
            raw[j] = load8<BF16>(a.y, p * a.cols + c);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kCombineAt; ++j)
        if (have[j]) {
          float v[8];
          unpack8<BF16>(raw[j], v);
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[j], v[k], acc[k]);
        }
    }
    if (a.residual) {
      float v[8];
      unpack8<BF16>(load8<BF16>(a.residual, i * 8), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] += v[k];
    }
    store8<BF16>(a.out, i * 8, pack8<BF16>(acc));
  }
}

// The weights' gradient: a wave per token, 512 columns at a time, its choices' rows in flight
// together (4093 tokens of 6 choices, 2048 bfloat16: 20 us, 5.9 TB/s; a row after the other 35).
template <bool BF16>
__global__ __launch_bounds__(256) void k_moe_dweights(sshdp_moe_combine_grad a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * (int64_t)4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.tokens) return;
  for (int j0 = 0; j0 < a.top_k; j0 += kCombineAt) {
    int p[kCombineAt];
    float sum[kCombineAt] = {};
#pragma unroll
    for (int j = 0; j < kCombineAt; ++j) {
      p[j] = j0 + j < a.top_k ? __builtin_amdgcn_readfirstlane(a.place[t * a.top_k + j0 + j]) : -1;
      if (p[j] >= a.rows) p[j] = -1;
    }
    for (int64_t c = lane * 8; c < a.cols; c += 512) {
      const Raw8<BF16> rd = load8<BF16>(a.dout, t * a.ld_dout + c);
      Raw8<BF16> ry[kCombineAt];
#pragma unroll
      for (int j = 0; j < kCombineAt; ++j) {
        ry[j] = Raw8<BF16>{};
        if (p[j] >= 0) ry[j] = load8<BF16>(a.y, p[j] * a.cols + c);
      }
      float d[8];
      unpack8<BF16>(rd, d);
#pragma unroll
      for (int j = 0; j < kCombineAt; ++j) {
        float v[8];
        unpack8<BF16>(ry[j], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[j] = p[j] >= 0 ? fmaf(d[k], v[k], sum[j]) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < kCombineAt; ++j) {
      if (j0 + j >= a.top_k) break;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) sum[j] += __shfl_xor(sum[j], d);
      if (lane == 0) a.dweights[t * a.top_k + j0 + j] = sum[j];
    }
  }
}

template <class I>
hipError_t moe_sort(const MoeSort &a, int32_t *counts, hipStream_t s) {
  const int64_t chunk = sort_chunk(a.slots);
  const unsigned chunks = (unsigned)std::max<int64_t>(1, (a.slots + chunk - 1) / chunk);
  const I *ids = static_cast<const I *>(a.ids);
  if (chunks > 1) {
    hipLaunchKernelGGL((k_moe_count<I>), dim3(chunks), dim3(kSortThreads), 0, s, ids, a.slots, a.experts, chunk, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((k_moe_place<I>), dim3(chunks), dim3(kSortThreads), 0, s, ids, a.slots, a.experts, a.align, a.rows,
                     chunk, chunks > 1 ? counts : nullptr, a.offsets, a.place, a.source);
  return hipGetLastError();
}

dim3 run_grid(int64_t runs) { return dim3((unsigned)std::min<int64_t>((runs + 255) / 256, 1 << 20)); }

}  // namespace

int64_t moe_sort_counts(int64_t slots, int experts) {
  const int64_t chunk = sort_chunk(slots), chunks = (slots + chunk - 1) / chunk;
  return chunks > 1 ? chunks * experts : 0;
}

hipError_t launch_moe_sort(const MoeSort &a, int32_t *counts, hipStream_t s) {
  return a.i64 ? moe_sort<int64_t>(a, counts, s) : moe_sort<int32_t>(a, counts, s);
}

hipError_t launch_moe_gather(const sshdp_moe_gather &a, hipStream_t s) {
  auto run = [&](auto bf16, auto weighted) {
    constexpr bool B = decltype(bf16)::value, W = decltype(weighted)::value;
    const int64_t tr = (a.rows + kMtRows - 1) / kMtRows, tiles = tr * ((a.cols + kMtCols - 1) / kMtCols);
    if (a.out.codes_t || !a.y || tiles >= kMtLeast) {
      hipLaunchKernelGGL((k_moe_tiles<B, W>), dim3((unsigned)tiles), dim3(256), 0, s, a, (uint32_t)tr, (uint32_t)tiles,
                         moe_band(a));
    } else {
      const int64_t runs = a.rows * (a.cols / 8), each = 256 * kMrRuns;
      hipLaunchKernelGGL((k_moe_rows<B, W>), dim3((unsigned)((runs + each - 1) / each)), dim3(256), 0, s, a,
                         (uint32_t)(a.cols / 8));
    }
  };
  const bool bf16 = a.dtype == SSHDP_DTYPE_BF16;
  if (bf16 && a.weights) run(std::true_type{}, std::true_type{});
  else if (bf16) run(std::true_type{}, std::false_type{});
  else if (a.weights) run(std::false_type{}, std::true_type{});
  else run(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_moe_combine(const sshdp_moe_combine_args &a, hipStream_t s) {
  const int runs = (int)(a.cols / 8);
  if (a.dtype == SSHDP_DTYPE_BF16)
    hipLaunchKernelGGL((k_moe_combine<true>), run_grid(a.tokens * runs), dim3(256), 0, s, a, runs);
  else
    hipLaunchKernelGGL((k_moe_combine<false>), run_grid(a.tokens * runs), dim3(256), 0, s, a, runs);
  return hipGetLastError();
}

hipError_t launch_moe_dweights(const sshdp_moe_combine_grad &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 3) / 4));
  if (a.dtype == SSHDP_DTYPE_BF16) hipLaunchKernelGGL((k_moe_dweights<true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_moe_dweights<false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace sshdp
