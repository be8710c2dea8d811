// Prints, for each line "form groups rows n k bf16" of its input, the kernel that a grouped
// product of those sizes runs (grouped_shape.h), built with g++ by tests/test_moe_host.py.
#include <cstdio>
#include <cstring>

#include "gemm_shape.h"
#include "grouped_shape.h"

int main() {
  char form[16];
  long long groups, rows, n, k;
  int bf16;
  while (std::scanf("%15s %lld %lld %lld %lld %d", form, &groups, &rows, &n, &k, &bf16) == 6) {
    const sshdp::GroupForm f = !std::strcmp(form, "nt") ? sshdp::kRowsNT
                               : !std::strcmp(form, "nn") ? sshdp::kRowsNN
                                                          : sshdp::kRowsGated;
    const int tile = sshdp::grouped_tile(f, groups, rows, n, k, bf16);
    const long long tiles = sshdp::grouped_tiles(f, groups, rows, n, tile);
    if (tile == 16) std::printf("few %s %s %d %lld\n", form, bf16 ? "bf16" : "fp32", k <= 2048 ? 4 : 8, tiles);
    else std::printf("tile%d %s %s %s %lld\n", tile, form, bf16 ? "bf16" : "fp32", sshdp::gemm_short(k) ? "short" : "long", tiles);
  }
  return 0;
}
