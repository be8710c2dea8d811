"""Each size of tests/gate_sizes.py runs the kernel it is named after (no GPU)."""

from gate_sizes import GATE_COLUMNS, GATE_SIZES
from test_moe_host import _choices


def test_gate_sizes_run_the_kernels_they_name(tmp_path):
    lines = [f"gated {len(c)} {sum(c)} {GATE_COLUMNS} {k} 1" for c, k in GATE_SIZES.values()]
    assert [g[0] for g in _choices(tmp_path, lines)] == list(GATE_SIZES)
