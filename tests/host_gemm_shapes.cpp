// host_gemm_shapes.cpp -- which of the compiled MXFP8 product kernels a size runs, with K
// whole or split, on the host.  Reads lines "nn m n k bf16" and prints each one's instance; or, called with a
// count, prints every instance that as many drawn sizes reach, with its smallest size (least
// m n k; of rows and columns in 32s and k in 128s if a second argument is given).
#include <stdio.h>
#include <stdlib.h>

#include <cmath>
#include <map>
#include <random>
#include <string>
#include <tuple>

#include "gemm_shape.h"

using namespace sshdp;

static std::string instance(bool nn, int64_t m, int64_t n, int64_t k, bool bf16) {
  const GemmShape s = gemm_shape_of(m, n, k, nn, bf16);
  const std::string type = bf16 ? " bf16" : " fp32", op = nn ? " nn" : " nt";
  if (s.tile == 16) return "few" + type + " " + std::to_string(gemm_few_waves(k));
  if (s.tile == 0) return "rows" + op + type + (nn ? "" : " " + std::to_string(gemm_rows_block(m)));
  // what every tile relies on: whole quads of steps, no split without work, all of K
  const int64_t nk = (k + kGemmStep - 1) / kGemmStep;
  if (s.steps % 4 || (int64_t)s.steps * s.groups * s.splits < nk || (int64_t)s.steps * s.groups * (s.splits - 1) >= nk ||
      (s.groups == 2 && gemm_short(k)) || (s.splits > 1 && gemm_short(k)) || (s.tile == 256 && nn && n < 128))
    return "bad shape";
  return "tile" + std::to_string(s.tile) + "x" + std::to_string(s.groups) + op + type + (gemm_short(k) ? " short" : " long") +
         (s.splits > 1 ? " split" : " whole");
}

int main(int argc, char **argv) {
  if (argc < 2) {
    long long nn, m, n, k, b;
    while (scanf("%lld %lld %lld %lld %lld", &nn, &m, &n, &k, &b) == 5) puts(instance(nn, m, n, k, b).c_str());
    return 0;
  }
  std::mt19937_64 rng(7);
  auto log_draw = [&](double lo, double hi) {
    return (int64_t)std::llround(lo * std::pow(hi / lo, (double)(rng() >> 11) * 0x1p-53));
  };
  std::map<std::string, std::tuple<double, long long, long long, long long>> seen;
  for (long i = 0; i < atol(argv[1]); ++i) {
    const bool nn = rng() & 1, b = rng() & 1;
    int64_t m = log_draw(1, 30000), n = log_draw(1, 30000), k = 32 * log_draw(1, 1000);
    if (nn) n = std::max<int64_t>(32, n / 32 * 32);
    if (argc > 2) m = (m + 31) / 32 * 32, n = (n + 31) / 32 * 32, k = (k + 127) / 128 * 128;
    const std::string name = instance(nn, m, n, k, b);
    const double size = (double)m * n * k;
    auto it = seen.find(name);
    if (it == seen.end() || size < std::get<0>(it->second)) seen[name] = {size, m, n, k};
  }
  for (auto &kv : seen)
    printf("%s,%lld,%lld,%lld\n", kv.first.c_str(), std::get<1>(kv.second), std::get<2>(kv.second), std::get<3>(kv.second));
  return 0;
}
