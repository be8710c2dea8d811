// Host-only check of the gradient norm's work items: reads data trees in the
// format of host_planner_check.cpp, plans each host-only and marks every element
// of every chunk and of every unit.  Prints, per tree, the unit elements and the
// number of chunks; fails if a unit element is not in exactly one chunk, a chunk
// holds anything else, or a chunk is empty or too long.
#include <cstdio>
#include <cstdint>
#include <vector>

#include "internal.h"

int main(int argc, char **argv) {
  if (argc != 2) return 2;
  FILE *f = std::fopen(argv[1], "rb");
  if (!f) return 2;
  for (;;) {
    int32_t n = 0, layout = 0;
    int64_t root = 0;
    uint32_t flags = 0;
    if (std::fread(&n, sizeof n, 1, f) != 1) break;
    if (std::fread(&root, sizeof root, 1, f) != 1 || std::fread(&layout, sizeof layout, 1, f) != 1 ||
        std::fread(&flags, sizeof flags, 1, f) != 1)
      return 3;
    std::vector<sshdp_node> nodes(n);
    if (std::fread(nodes.data(), sizeof(sshdp_node), n, f) != (size_t)n) return 3;
    sshdp_plan_opts o;
    sshdp_default_opts(&o);
    o.scale_layout = layout;
    o.flags = flags | SSHDP_PLAN_HOST_ONLY;
    sshdp_plan *p = nullptr;
    if (sshdp_plan_views(nodes.data(), n, root, &o, &p) != SSHDP_OK) return 4;
    std::vector<uint8_t> seen(root, 0);
    for (const sshdp::GChunk &c : p->gchunks) {
      if (c.n < 1 || c.n > sshdp::kChunk || c.base < 0 || c.base + c.n > root) return 5;
      for (int64_t e = c.base; e < c.base + c.n; ++e)
        if (seen[e]++) return 6;
    }
    int64_t units = 0;
    for (int32_t i = 0; i < n; ++i) {
      if (!nodes[i].is_unit) continue;
      for (int64_t r = 0; r < nodes[i].rows; ++r)
        for (int64_t c = 0; c < nodes[i].cols; ++c) {
          uint8_t &s = seen[p->node_abs[i] + r * nodes[i].row_stride + c];
          if (s != 1) return 7;
          s = 2;
          ++units;
        }
    }
    for (uint8_t s : seen)
      if (s == 1) return 8;
    std::printf("%lld %zu\n", (long long)units, p->gchunks.size());
    sshdp_plan_destroy(p);
  }
  std::fclose(f);
  return 0;
}
