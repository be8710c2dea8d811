"""Sizes for every way a product grouped by expert may run (as tests/host_grouped_shapes.cpp names it): rows of each
expert, n and k."""

SIZES = {
    "few nt bf16 4": ([3, 0, 17, 1], 71, 544),
    "few nt bf16 8": ([5, 20], 45, 4256),
    "few nt fp32 4": ([16, 1, 0, 33], 67, 1056),
    "few nt fp32 8": ([1, 0, 2], 64, 2080),
    "few gated bf16 4": ([1, 18, 0], 96, 1184),
    "few gated bf16 8": ([2, 7], 64, 8224),
    "tile128 nt bf16 short": ([700, 0, 333], 131, 96),
    "tile128 nt bf16 long": ([700, 800, 1, 0], 455, 672),
    "tile128 nt fp32 short": ([2900, 1, 801], 131, 288),
    "tile128 nt fp32 long": ([900, 0, 300], 387, 1056),
    "tile128 nn bf16 short": ([3, 0, 200], 96, 160),
    "tile128 nn bf16 long": ([1, 130], 160, 1056),
    "tile128 nn fp32 short": ([33, 5, 0], 96, 128),
    "tile128 nn fp32 long": ([256, 0, 70], 288, 544),
    "tile128 gated bf16 short": ([640, 3, 0, 421], 160, 288),
    "tile128 gated bf16 long": ([640, 3, 0, 421], 288, 1120),
    "tile256 nt bf16 short": ([9000, 0, 7301], 700, 512),
    "tile256 nt bf16 long": ([5000, 0, 3113], 1411, 1056),
    "tile256 nn bf16 short": ([8999, 0, 7300], 704, 512),
    "tile256 nn bf16 long": ([5000, 0, 3113], 1408, 1056),
    "tile256 gated bf16 short": ([2500, 0, 5601], 704, 512),
    "tile256 gated bf16 long": ([1200, 0, 2889], 1408, 1056),
}
