"""GPU parity of the gated activation's gradient against float64, at sizes, ends and gates where it can go wrong."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
from gpu_util import say
from test_gpu_moe_products import check_codes, decode, stream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = 2.0 ** -118                                     # float32 ends its normal range near gates of -87


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def near(g):
    """The sigmoid's error relative to itself, and silu's and h's: the exponent x log2(e) is off by half a step of its
    rounding and log2(e) by 2^-26.1 of itself, together 1.23 |x| 2^-24 of the exponential; then exp2 and the reciprocal
    (a step, 2, each), the sum and two products (half a step, 1, each): 7."""
    return (1.25 * g.abs() + 8) * 2.0 ** -24


def formula(dh, gate, up):
    """{name: (value, bound)} in float64.  dgate's factor s (1 + gate (1 - s)) has each s off by near, 1 - s by that and a
    rounding, in terms no larger than s (1 + |gate|); then five more roundings."""
    d, g, u = (t.double() for t in (dh, gate, up))
    s = torch.special.expit(g)
    dg, du, h = d * u * s * (1 + g * (1 - s)), d * g * s, g * s * u
    edge = TINY * (1 + g.abs()) * (1 + d.abs()) * (1 + u.abs())
    return {"dgate": (dg, (2 * near(g) + 2.0 ** -22) * (d * u * s).abs() * (1 + g.abs()) + edge),
            "dup": (du, near(g) * du.abs() + edge), "h": (h, near(g) * h.abs() + edge)}


def call(dh, gate, up, wanted, offsets=None, groups=1):
    """The pairs named in wanted ({output: "rows", "columns" or "both"}), in buffers of 0xA5."""
    rows, cols = gate.shape
    out = {}
    for name, way in wanted.items():
        t = {}
        if way != "columns":
            t["codes"], t["scales"] = torch.empty(rows, cols), torch.empty(rows, cols // 32)
        if way != "rows":
            t["codes_t"], t["scales_t"] = torch.empty(cols, rows), torch.empty(cols, rows // 32)
        out[name] = {k: torch.full(v.shape, 0xA5, dtype=torch.uint8, device="cuda") for k, v in t.items()}
    sh.swiglu_backward_mxfp8(dh, gate, up, rows, cols, offsets=offsets, groups=groups,
                             **{n: sh.mx_pair(**t) for n, t in out.items()}, stream=stream())
    return out


def check(out, ref, used, rows):
    for name, t in out.items():
        v, e = ref[name]
        if "codes" in t:
            check_codes(t["codes"][:used], t["scales"][:used], v[:used], e[:used])
            assert bool((t["codes"][used:] == 0xA5).all()) and bool((t["scales"][used:] == 0xA5).all())
        if "codes_t" in t:
            full = -(-used // 32) * 32
            v, e = v.clone(), e.clone()
            v[used:], e[used:] = 0, 0
            check_codes(t["codes_t"][:, :full], t["scales_t"][:, :full // 32], v[:full].t().contiguous(),
                        e[:full].t().contiguous())
            assert bool((t["codes_t"][:, full:] == 0xA5).all()) and bool((t["scales_t"][:, full // 32:] == 0xA5).all())


def inputs(rows, cols, seed=0):
    g = torch.Generator(device="cuda").manual_seed(rows + cols + seed)
    r = lambda s: (torch.randn(rows, cols, generator=g, device="cuda") * s).bfloat16()   # noqa: E731
    return r(1e-3), r(3.0), r(1.0)


@pytest.mark.parametrize("rows,cols,used", [(32, 32, 32), (32, 64, 1), (64, 96, 0), (128, 64, 128), (160, 32, 33),
                                            (384, 1408, 300), (288, 160, 287), (4096, 96, 4095)])
def test_every_output(rows, cols, used):
    say(f"swiglu gradient {rows} x {cols}, {used} in use")
    dh, gate, up = inputs(rows, cols)
    dh[used:], gate[used:], up[used:] = float("nan"), float("nan"), float("nan")
    off = torch.tensor([0, 0, used], dtype=torch.int32, device="cuda")
    ref = formula(dh, gate, up)
    both = call(dh, gate, up, dict(dgate="both", dup="both", h="both"), off, 2)
    check(both, ref, used, rows)
    for wanted in (dict(dgate="rows", dup="rows"), dict(dgate="both", dup="both", h="columns"), dict(dup="columns"),
                   dict(h="rows"), dict(dgate="rows"), dict(h="both")):
        out = call(None if set(wanted) == {"h"} else dh, gate, up, wanted, off, 2)
        for name, t in out.items():
            for k, v in t.items():
                assert torch.equal(v, both[name][k]), (wanted, name, k)
    if used == rows:
        out = call(dh, gate, up, dict(dgate="both", dup="both", h="both"))
        assert all(torch.equal(v, both[n][k]) for n, t in out.items() for k, v in t.items())


def test_rows_alone_of_any_count():
    say("swiglu gradient, 37 rows")
    dh, gate, up = inputs(37, 64)
    check(call(dh, gate, up, dict(dgate="rows", dup="rows", h="rows")), formula(dh, gate, up), 37, 37)


def test_every_gate():
    """Every finite bfloat16 gate, with dh and up one: no value is far from the formula's, whatever its size."""
    say("swiglu gradient, every gate")
    b = torch.arange(65536, dtype=torch.int32, device="cuda").short().view(torch.bfloat16)
    gate = torch.sort(b[torch.isfinite(b)].float()).values.bfloat16().view(-1, 32)   # blocks of like sizes
    one = torch.ones_like(gate)
    ref = formula(one, gate, one)
    out = call(one, gate, one, dict(dgate="rows", dup="rows", h="rows"))
    for name, t in out.items():
        assert bool((t["scales"] < 255).all())
        check_codes(t["codes"], t["scales"], *ref[name])


@pytest.mark.parametrize("columns", [False, True])
def test_non_finite_values(columns):
    """A NaN makes its blocks NaN and no other; so do infinities where the formula has none."""
    say("swiglu gradient, non-finite")
    dh, gate, up = inputs(64, 128)
    want = dict.fromkeys(("dgate", "dup", "h"), "both" if columns else "rows")
    ref = call(dh, gate, up, want)
    gate[3, 5], dh[20, 40], up[40, 100] = float("nan"), float("inf"), float("-inf")
    out = call(dh, gate, up, want)
    hit = {"dgate": [(3, 5), (20, 40), (40, 100)], "dup": [(3, 5), (20, 40)], "h": [(3, 5), (40, 100)]}
    for name, t in out.items():
        bad = torch.zeros(64, 4, dtype=torch.bool, device="cuda")
        bad_t = torch.zeros(128, 2, dtype=torch.bool, device="cuda")
        for r, c in hit[name]:
            bad[r, c // 32], bad_t[c, r // 32] = True, True
        for k, b in (("", bad), ("_t", bad_t))[:1 + columns]:
            assert bool((t["scales" + k][b] == 255).all())
            assert torch.equal(t["scales" + k][~b], ref[name]["scales" + k][~b])
            wide = b.repeat_interleave(32, 1)
            assert bool((t["codes" + k][wide] == 0x7F).all())
            assert torch.equal(t["codes" + k][~wide], ref[name]["codes" + k][~wide])


def test_wild_ends():
    say("swiglu gradient, wild ends")
    dh, gate, up = inputs(96, 32)
    full = call(dh, gate, up, dict(dup="both"))
    for end, used in ((1 << 30, 96), (-(1 << 31), 0), (97, 96)):
        off = torch.tensor([5, end], dtype=torch.int32, device="cuda")
        out = call(dh, gate, up, dict(dup="both"), off)
        assert torch.equal(out["dup"]["codes"][:used], full["dup"]["codes"][:used])
        assert bool((out["dup"]["codes"][used:] == 0xA5).all())


def test_it_is_the_gradient_of_the_forward_product():
    """h recomputed from the kept products has the forward's codes but for the products' rounding to bfloat16."""
    say("swiglu, forward and recomputed")
    g = torch.Generator(device="cuda").manual_seed(4)
    p, n, k = 96, 160, 256

    def mx(rows, scale):
        x = torch.randn(rows, k, generator=g, device="cuda") * scale
        c, s = torch.empty(rows, k, dtype=torch.uint8, device="cuda"), torch.empty(rows, k // 32, dtype=torch.uint8, device="cuda")
        sh.quant_mxfp8(x, "fp32", rows, k, c, s, stream=stream())
        return sh.mx_matrix(c, s, rows, k)
    codes, scales = torch.zeros(p, n, dtype=torch.uint8, device="cuda"), torch.zeros(p, n // 32, dtype=torch.uint8, device="cuda")
    gate, up = (torch.zeros(p, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sh.gemm_mxfp8_swiglu(mx(p, 1.0), mx(n, 0.1), mx(n, 0.1), codes, scales, gate=gate, up=up, stream=stream())
    again = call(None, gate, up, dict(h="rows"))["h"]
    a, step = decode(codes, scales)
    b, step_b = decode(again["codes"], again["scales"])
    gd, ud = gate.double(), up.double()
    s = torch.special.expit(gd)
    moved = 2.0 ** -8 * (gd * ud).abs() * (s * (1 + gd.abs()) + s) + 2.0 ** -15 * (1 + gd.abs()) * (1 + ud.abs())
    assert bool(((a - b).abs() <= moved + (step + step_b) * 1.001).all())
