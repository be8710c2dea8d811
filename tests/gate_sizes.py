"""Sizes of gated products of 768 columns with a short K, one for each kernel (as tests/host_grouped_shapes.cpp names
it): rows of each expert and k."""

GATE_COLUMNS = 768
GATE_SIZES = {
    "few gated bf16 4": ([3, 18], 64),
    "few gated bf16 8": ([1, 2], 2080),
    "tile128 gated bf16 short": ([700, 300], 64),
    "tile256 gated bf16 short": ([4000, 2001], 64),
}
