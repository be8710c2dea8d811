// grouped_shape.h -- how a product grouped by expert runs: which kernel, chosen on the host from
// its sizes.  The experts' shares of the rows are not known there.  Plain C++, so the choice can
// be looked at without a GPU.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace sshdp {

enum GroupForm { kRowsNT, kRowsNN, kRowsGated, kColumns };

// Pieces of `piece` rows that `rows` rows of `groups` experts come to: half a piece an expert
// more than the rows fill, and one at least for each expert that rows dealt at random reach.
inline double grouped_pieces(int64_t groups, int64_t rows, int piece) {
  const double used = (double)groups * (1.0 - std::exp(-(double)rows / (double)groups));
  return std::max(used, (double)rows / piece + used / 2);
}

// Columns of B (gated: of each of the two) that a tile takes.
inline int grouped_cols(GroupForm form, int tile) {
  const int c = tile == 16 ? 64 : tile;
  return form == kRowsGated ? c / 2 : c;
}

// 16: the kernel of a few rows an expert; else the tile's edge.  The candidate with the least
// modelled time in microseconds.  The tiles' constants were fitted to 216 sizes of 1, 8 and 64
// experts, 512 .. 24576 rows dealt evenly, 704 x 512 .. 2048 x 4096, operands from HBM: there what it
// picks takes 1.2% more than the better of the two on average and 1.26 times at worst (always 128:
// 6.4% and 1.36 times).  Few rows against 128-tiles at 216 sizes of 4 .. 1024 rows, 320 x 1024 ..
// 2048 x 4096: 1.7% and 1.36 times (products of 9 us).  At 90 other sizes (2 to 128 experts, 33 ..
// 24576 rows, n and k 320 .. 4096), rows dealt evenly, as a router with favourites deals them, and
// with most of them at a few experts: between the tiles 1.1, 0.4 and 0.6% on average and 1.29 times at
// worst (always 128: 4% and 1.39 times); where few rows come into question (17 sizes) 8% and 1.7
// times, with K under 512, of which one wave of the few rows' four has all the work.
//   few rows:  each piece reads its expert's B, at 5.5 TB/s, in no less than 3 us a round (64
//              experts, gated 1408 x 2048: 96 rows 51 us, 128-tiles 54; 768 rows 91 and 83; one
//              expert of 16 rows 9.4 and 14.3);
//   128-tiles: two workgroups a CU, 1.36 us for a step of both, 0.64 for one alone, and no
//              faster than they read B, at 5.2 TB/s;
//   256-tiles: one workgroup a CU, 1.6 us a step, which is half as much for the same work, but
//              experts of uneven hundreds of rows fill them worse.
// Float32 output takes 128-tiles: 256-tiles gain 5% at the largest sizes and lose up to twice at
// the small ones.
inline int grouped_tile(GroupForm form, int64_t groups, int64_t rows, int64_t n, int64_t k, bool bf16) {
  if (form == kColumns) return 128;
  const double steps = (double)((k + 127) / 128);
  auto tiles = [&](int tile) {
    const int c = grouped_cols(form, tile);
    return (int64_t)(grouped_pieces(groups, rows, tile) * (double)((n + c - 1) / c));
  };
  const int64_t t = tiles(128), pairs = t / 512, rest = t % 512;
  double us128 = 3.5 + (double)pairs * (2.2 + 1.36 * steps);
  if (rest) us128 += 2.2 + steps * (rest <= 256 ? 0.64 : 0.64 + 0.72 * (double)(rest - 256) / 256);
  if (form != kRowsNN) {
    const double b = (double)n * (double)k * (form == kRowsGated ? 2 : 1);
    const double read = grouped_pieces(groups, rows, 16) * b / 5.5e6, walk = (double)tiles(16) / 512 * 3.0;
    // (a launch has under 2^32 threads)
    const double tiles_read = 7.0 + grouped_pieces(groups, rows, 128) * b / 5.2e6;
    if (6.0 + std::max(read, walk) <= std::max(us128, tiles_read) && tiles(16) <= 1 << 21) return 16;
  }
  if (!bf16 || (form == kRowsNN && n < 128)) return 128;
  return (double)((tiles(256) + 255) / 256) * (7.0 + 1.6 * steps) < us128 ? 256 : 128;
}

// Workgroups of a launch at most.
inline int64_t grouped_tiles(GroupForm form, int64_t groups, int64_t m, int64_t n, int tile) {
  const int cols = grouped_cols(form, tile);
  const int64_t tn = (n + cols - 1) / cols;
  if (form == kColumns) return groups * ((m + tile - 1) / tile) * tn;
  return (m / tile + std::min(groups, m)) * tn;        // no more experts than rows have any
}

}  // namespace sshdp
