// gemm_shape.h -- how an MXFP8 product runs: which kernel, tile and split of K, chosen on the
// host from its sizes, operand form and output type.  Plain C++, so the choice can be looked
// at without a GPU.
#pragma once
#include <stdint.h>

#include <algorithm>

namespace sshdp {

constexpr int kGemmStep = 128;                       // k of one step of a tile

// Up to 4 steps: a row's scale bytes are fewer than the 16 of one load.
inline bool gemm_short(int64_t k) { return k <= 4 * kGemmStep; }

// Waves of the kernel of up to 16 rows with A in registers, 8 steps each.
inline int gemm_few_waves(int64_t k) { return k <= 2048 ? 2 : k <= 4096 ? 4 : 8; }

// Rows of m that the few-row kernel takes at a time.
inline int gemm_rows_block(int64_t m) { return m <= 16 ? 16 : m <= 32 ? 32 : 64; }

// How a product runs: the kernel of up to 16 rows with A in registers (tile 16), the few-row
// kernel (tile 0), or tiles of 256 or 128 by `groups` wave groups, with K in `splits` parts,
// each of `groups` runs of `steps` 128-k steps (a multiple of 4: scale words come 4 steps at a
// time).
struct GemmShape {
  int tile, groups, splits, steps;
};

// The candidate with the least modelled time, in microseconds on an idle MI355X.  The
// constants were fitted to 300 timed choices from m 1 .. 4096, n and k 128 .. 28672, both
// operand forms and output types.  Of 220 others timed with operands from HBM (110 sizes of
// those ranges) what it picks takes 5.0% more than the best candidate on average; at worst
// 1.34 times up to 16 rows, 1.83 from 17 to 256 (the few-row kernel in float32) and 1.22
// above.  Always unsplit 128-tiles: 52% and 5.5 times; always unsplit 256-tiles: 175%.
//   few rows:  the operands' bytes as the kernel gets them, or its waves' steps in turn;
//   128-tiles: two workgroups a CU, 0.95 us for a step of both, 0.61 for one alone;
//   128-tiles by two wave groups: one workgroup a CU, 1.1 us for a step of both;
//   256-tiles: one workgroup a CU, 1.21 us a step (1.87 float32, its matrix rate is half);
//   a K split: the join's launch, and its partial sums' bytes.
inline GemmShape gemm_shape_of(int64_t m, int64_t n, int64_t k, bool nn, bool bf16) {
  // from 84 MB of B on ahead of the others (1 x 10240 x 8192: 20.0 us against 22.4, float32 27.7;
  // 16 x 23606 x 7744: 41.1 against 50.9), around 20 MB level with them; under 10 MB, where a
  // call takes 5 to 7 us, up to 1.8 us behind the few-row kernel or unsplit tiles
  if (!nn && m <= 16 && k <= 8192) return {16, 1, 1, 0};
  const int nk = (int)((k + kGemmStep - 1) / kGemmStep);
  GemmShape best{0, 1, 1, 0};
  double least = 1e30;
  auto consider = [&](const GemmShape &s, double us) {
    if (us < least) least = us, best = s;
  };
  const bool tiles = nn ? (k >> 5) * (n >> 5) >= 4 : k > 0;   // NN reads scales 4 at a time
  if (!tiles || (!nn && m <= 256)) {
    const int rows = gemm_rows_block(m);
    const double rate = rows == 16 ? 5.8e6 : rows == 32 ? 3.4e6 : 5.0e6;
    const double us = std::max(rows == 64 ? 1.34 * ((nk + 7) / 8) : 0.0, (double)n * k * ((m + rows - 1) / rows) / rate);
    consider({0, 1, 1, 0}, 6.7 + us * (bf16 ? 1.0 : 1.2));
  }
  if (!tiles) return best;
  const int64_t t128 = (m + 127) / 128 * ((n + 127) / 128), t256 = (m + 255) / 256 * ((n + 255) / 256);
  for (int groups : {1, 2})
    for (int want : {1, 2, 3, 4, 6, 8, 16}) {
      const int parts = groups * want, steps = ((nk + parts - 1) / parts + 3) / 4 * 4;
      const int splits = (nk + groups * steps - 1) / (groups * steps);
      if (splits != want || (groups == 2 && nk <= steps)) continue;
      const double join = splits > 1 ? 3.0 + (double)splits * m * n * 4 / 2.66e6 : 0.0;
      if (groups == 2) {
        consider({128, 2, splits, steps}, 2.8 + (t128 * splits + 255) / 256 * (1.2 + steps * (bf16 ? 1.1 : 1.94)) + join);
        continue;
      }
      const int run = std::min(steps, nk);
      const double one = bf16 ? 0.61 : 0.9, two = bf16 ? 0.95 : 1.13;
      const int64_t pairs = t128 * splits / 512, rest = t128 * splits % 512;
      double us = 3.2 + pairs * (1.4 + run * two) + join;
      if (rest) us += 1.4 + run * (rest <= 256 ? one : one + (two - one) * (rest - 256) / 256);
      consider({128, 1, splits, steps}, us);
      if (nn && n < 128) continue;
      consider({256, 1, splits, steps}, 4.5 + (t256 * splits + 255) / 256 * (2.3 + run * (bf16 ? 1.21 : 1.87)) + join);
    }
  return best;
}

}  // namespace sshdp
