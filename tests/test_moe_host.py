"""The expert layer's operators on the host (no GPU): their refusals (every argument error comes before anything
touches the device), the sizes they ask for, and their gradients' formulas against differences."""

import itertools
import os
import subprocess

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import moe_ref as M
from grouped_sizes import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20                                            # an aligned address that no refused call follows


def refused(name, call, *a, **k):
    with pytest.raises(sh.SshdpError) as e:
        call(*a, **k)
    assert e.value.name == name, (e.value.name, name)


@pytest.mark.parametrize("align", [1, 2, 16, 32, 64, 256])
def test_rows_hold_the_worst_ids(align):
    """Every way to spread the slots over the experts fits, and some way needs each expert's whole padding."""
    for t, k, e in [(0, 1, 3), (1, 1, 1), (3, 2, 2), (5, 1, 4), (2, 2, 64)]:
        n = sh.moe_rows(t, k, e, align)
        assert n == M.rows_for(t, k, e, align)
        worst = 0
        for ids in itertools.product(range(min(e, 4)), repeat=t * k):
            worst = max(worst, int(M.sort(ids, e, align, n)[0][-1]))
        spread = M.sort([i % e for i in range(t * k)], e, align, n)[0][-1]
        assert max(worst, spread) <= n
        assert align < 32 or n % 128 == 0


def test_rows_and_workspace_refusals():
    for f in (lambda *a: sh.moe_rows(*a, 1), sh.moe_sort_workspace):
        refused("ARG", f, -1, 1, 1)
        refused("ARG", f, 1, 0, 1)
        refused("ARG", f, 1, 1, 0)
        refused("SCHEMA", f, 1, 65, 1)
        refused("SCHEMA", f, 1, 1, 1025)
        refused("SCHEMA", f, (1 << 24) // 3 + 1, 3, 8)
    refused("ARG", sh.moe_rows, 1, 1, 1, 0)
    refused("ARG", sh.moe_rows, 1, 1, 1, 48)
    refused("SCHEMA", sh.moe_rows, 1, 1, 1, 512)
    assert sh.moe_sort_workspace(1, 6, 64) == 0
    assert sh.moe_sort_workspace(16381, 6, 64) % 4 == 0 < sh.moe_sort_workspace(16381, 6, 64)


def test_sort_refusals():
    def q(ids=P, tokens=9, top_k=2, experts=4, offsets=P, place=P, source=P, rows=18, **k):
        return lambda: sh.moe_sort(ids, tokens, top_k, experts, offsets, place, source, rows, **k)
    refused("ARG", q(ids_dtype="int8"))
    for k in ("ids", "offsets", "place", "source"):
        refused("ARG", q(**{k: None}))
        refused("ALIGN", q(**{k: P + 2}))
    refused("ALIGN", q(ids=P + 4, ids_dtype="int64"))
    refused("ARG", q(align=3))
    refused("SCHEMA", q(rows=17))
    refused("SCHEMA", q(rows=18, align=2))
    refused("SCHEMA", q(rows=(1 << 30) + 1))
    refused("SCHEMA", q(experts=1025))
    n = sh.moe_sort_workspace(4096, 2, 4)
    refused("WORKSPACE", q(tokens=4096, rows=8192))
    refused("WORKSPACE", q(tokens=4096, rows=8192, workspace=P, workspace_bytes=n - 1))
    refused("ALIGN", q(tokens=4096, rows=8192, workspace=P + 4, workspace_bytes=n))


def test_gather_refusals():
    def q(x=P, source=P, offsets=P, tokens=4, top_k=2, experts=4, rows=32, cols=64, **k):
        return lambda: sh.moe_gather_mxfp8(x, source, offsets, tokens, top_k, experts, rows, cols,
                                           **{**dict(codes=P, scales=P), **k})
    refused("ARG", q(dtype="fp16"))
    refused("ARG", q(rows=-1))
    refused("ARG", q(cols=-32))
    refused("ARG", q(codes=None, scales=None))         # no output
    refused("ARG", q(scales=None))
    refused("ARG", q(codes_t=P))
    for k in ("x", "source", "offsets"):
        refused("ARG", q(**{k: None}))
    refused("SCHEMA", q(cols=48))
    refused("SCHEMA", q(ld_x=32))
    refused("SCHEMA", q(ld_x=68))
    refused("SCHEMA", q(rows=33, codes_t=P, scales_t=P))
    refused("SCHEMA", q(rows=(1 << 30) + 32))
    refused("SCHEMA", q(top_k=65))
    refused("SCHEMA", q(experts=1025))
    refused("ALIGN", q(x=P + 8))
    refused("ALIGN", q(y=P + 8))
    refused("ALIGN", q(codes=P + 8))
    refused("ALIGN", q(codes_t=P + 8, scales_t=P))
    for k in ("source", "offsets", "weights"):
        refused("ALIGN", q(**{k: P + 2}))
    q(rows=0)()                                        # nothing to do
    q(cols=0)()


def test_combine_refusals():
    def q(y=P, place=P, out=P, tokens=4, top_k=2, rows=8, cols=64, **k):
        return lambda: sh.moe_combine(y, place, out, tokens, top_k, rows, cols, **k)
    refused("ARG", q(dtype="x"))
    refused("ARG", q(rows=-1))
    refused("ARG", q(tokens=-1))
    refused("ARG", q(top_k=0))
    for k in ("y", "place", "out"):
        refused("ARG", q(**{k: None}))
    refused("SCHEMA", q(cols=40))
    refused("SCHEMA", q(top_k=65))
    refused("SCHEMA", q(rows=(1 << 30) + 1))
    for k in ("y", "out", "residual"):
        refused("ALIGN", q(**{k: P + 8}))
    for k in ("place", "weights"):
        refused("ALIGN", q(**{k: P + 2}))
    q(tokens=0, y=None, place=None, out=None)()
    q(cols=0, y=None, place=None, out=None)()


def test_combine_backward_refusals():
    def q(dout=P, y=P, weights=P, place=P, source=P, offsets=P, tokens=4, top_k=2, experts=4, rows=32, cols=64, **k):
        return lambda: sh.moe_combine_backward(dout, y, weights, place, source, offsets, tokens, top_k, experts, rows,
                                               cols, **{**dict(codes=P, scales=P, dweights=P), **k})
    none = dict(codes=None, scales=None)
    refused("ARG", q(dtype="x"))
    refused("ARG", q(**none, dweights=None))           # no output
    refused("ARG", q(scales=None))
    for k in ("dout", "source", "offsets"):
        refused("ARG", q(**{k: None}))
    for k in ("dout", "y", "place"):
        refused("ARG", q(**none, **{k: None}))
    refused("SCHEMA", q(cols=40))
    refused("SCHEMA", q(ld_dout=32))
    refused("SCHEMA", q(rows=33, codes_t=P, scales_t=P))
    for k in ("dout", "dy", "codes"):
        refused("ALIGN", q(**{k: P + 8}))
    for k in ("y", "place", "dweights"):
        refused("ALIGN", q(**none, **{k: P + 2}))
    q(rows=0, tokens=0, dout=None, y=None, place=None)()


def test_combine_gradient_formulas_against_differences():
    """The loss sum(dout * combine(y, weights)) moves with y and weights as their gradients say."""
    rng = np.random.default_rng(3)
    tokens, top_k, experts, cols = 7, 3, 5, 32
    ids = rng.integers(-1, experts, (tokens, top_k))
    rows = M.rows_for(tokens, top_k, experts, 2)
    offsets, place, source = M.sort(ids, experts, 2, rows)
    y, w = rng.standard_normal((rows, cols)), rng.random((tokens, top_k))
    dout = rng.standard_normal((tokens, cols)).astype(np.float32)
    w = w.astype(np.float32)
    loss = lambda y_, w_: float(np.sum(dout * M.combine(y_, place, w_, None, top_k, "fp32")[0]))   # noqa: E731
    dy = M.gather(dout, w, source, offsets, top_k)
    dw, _ = M.dweights(dout, y, place, top_k)
    vy, vw, h = rng.standard_normal(y.shape), rng.standard_normal(w.shape), 2.0 ** -10
    # the loss is linear in each: differences are exact but for float64's (and dy's float32) rounding
    got = (loss(y + h * vy, w) - loss(y - h * vy, w)) / (2 * h)
    assert abs(got - np.sum(dy * vy)) <= 1e-5 * np.sum(np.abs(dy * vy))
    got = (loss(y, w + h * vw) - loss(y, w - h * vw)) / (2 * h)
    assert abs(got - np.sum(dw * vw)) <= 1e-9 * np.sum(np.abs(dw * vw))
    # x's gradient through the gather is the combine of the rows' gradients
    x, g = rng.standard_normal((tokens, cols)).astype(np.float32), rng.standard_normal((rows, cols))
    lx = np.sum(M.gather(x, w, source, offsets, top_k).astype(np.float64) * g)
    assert abs(lx - np.sum(x * M.combine(g, place, w, None, top_k, "fp32")[0])) <= 1e-5 * np.sum(np.abs(x)) * 4


def _m(rows, cols, layout="rowmajor", codes=P):
    return sh.mx_matrix(codes, P, rows, cols, layout)


def test_grouped_product_refusals():
    def q(a=None, b=None, out=P, offsets=P, groups=4, op="nt", **k):
        a = a or _m(8, 64)
        b = b or _m(4 * 64, 64, "block32x32")
        return lambda: sh.gemm_mxfp8_grouped(a, b, out, offsets, groups, op=op, **{**dict(out_dtype="fp32"), **k})
    refused("ARG", q(op="tt"))
    refused("ARG", q(out_dtype="fp16"))
    refused("ARG", q(out=None))
    refused("ARG", q(offsets=None))
    refused("ARG", q(groups=0))
    refused("ARG", q(a=_m(8, 64, codes=None)))
    refused("ARG", q(a=_m(8, 64, "other")))
    refused("SCHEMA", q(groups=1025, b=_m(1025 * 32, 64)))
    refused("SCHEMA", q(groups=3))                     # no equal parts
    refused("SCHEMA", q(groups=8, b=_m(8 * 16, 64, "block32x32")))
    refused("SCHEMA", q(a=_m(32, 64, "block32x32")))
    refused("SCHEMA", q(a=_m(8, 96)))
    refused("SCHEMA", q(a=_m(8, 0), b=_m(256, 0)))
    refused("SCHEMA", q(a=_m(8, (1 << 22) + 32), b=_m(4, (1 << 22) + 32)))
    refused("SCHEMA", q(ld_out=63))
    refused("SCHEMA", q(op="nn", b=_m(256, 64)))
    refused("SCHEMA", q(op="nn", a=_m(8, 32), b=_m(128, 96, "block32x32")))    # experts of three blocks
    refused("SCHEMA", q(a=_m(1 << 30, 64), b=_m(4 * 4096, 64)))                # too many tiles
    t = dict(op="tn", a=_m(40, 128), b=_m(64, 128))
    refused("ARG", q(**{**t, "out_dtype": "bf16"}))
    refused("SCHEMA", q(**{**t, "a": _m(40, 160), "b": _m(64, 160)}))
    refused("SCHEMA", q(**{**t, "a": _m(40, 256)}))
    refused("SCHEMA", q(**{**t, "b": _m(64, 128, "block32x32")}))
    refused("ALIGN", q(out=P + 4))
    refused("ALIGN", q(addend=P + 4))
    refused("ALIGN", q(offsets=P + 2))
    refused("ALIGN", q(a=_m(8, 64, codes=P + 8)))
    q(a=_m(0, 64), out=None)()                         # nothing to do


def test_gated_product_refusals():
    def q(a=None, g=None, u=None, codes=P, scales=P, offsets=P, groups=4, **k):
        g = g or _m(4 * 64, 64, "block32x32")
        u = u or _m(4 * 64, 64, "block32x32")
        return lambda: sh.gemm_mxfp8_swiglu(a or _m(8, 64), g, u, codes, scales, offsets=offsets, groups=groups, **k)
    refused("ARG", q(codes=None))
    refused("ARG", q(codes=None, scales=None))         # no output
    refused("ARG", q(gate=P))
    refused("ARG", q(offsets=None))
    refused("ARG", q(u=_m(4 * 64, 64, "other")))
    refused("SCHEMA", q(u=_m(4 * 32, 64, "block32x32")))
    refused("SCHEMA", q(u=_m(4 * 64, 64)))
    refused("SCHEMA", q(u=_m(4 * 64, 96, "block32x32")))
    refused("SCHEMA", q(g=_m(4 * 40, 64), u=_m(4 * 40, 64)))
    refused("SCHEMA", q(a=_m(8, 96)))
    for k in ("codes", "gate", "up"):
        refused("ALIGN", q(**{**dict(gate=P, up=P), k: P + 8}))
    refused("ALIGN", q(u=_m(4 * 64, 64, "block32x32", codes=P + 8)))
    q(a=_m(0, 64), codes=None, scales=None)()


def test_activation_gradient_refusals():
    r, c = sh.mx_pair(P, P), sh.mx_pair(P, P, P, P)

    def q(dh=P, gate=P, up=P, rows=32, cols=64, **k):
        return lambda: sh.swiglu_backward_mxfp8(dh, gate, up, rows, cols, **{**dict(dgate=r, dup=r), **k})
    refused("ARG", q(rows=-1))
    refused("ARG", q(dgate=None, dup=None))            # no output
    for k in ("dh", "gate", "up"):
        refused("ARG", q(**{k: None}))
        refused("ALIGN", q(**{k: P + 8}))
    refused("ARG", q(h=sh.mx_pair(P)))
    refused("ARG", q(h=sh.mx_pair(None, None, None, P)))
    refused("ARG", q(offsets=P, groups=0))
    refused("SCHEMA", q(offsets=P, groups=1025))
    refused("SCHEMA", q(cols=40))
    refused("SCHEMA", q(rows=33, dup=c))
    refused("SCHEMA", q(rows=(1 << 30) + 32))
    refused("ALIGN", q(offsets=P + 2))
    refused("ALIGN", q(dup=sh.mx_pair(P + 8, P)))
    refused("ALIGN", q(h=sh.mx_pair(None, None, P + 8, P)))
    q(rows=0, dh=None, gate=None, up=None)()
    q(cols=0)()


def test_activation_gradient_formula_against_differences():
    rng = np.random.default_rng(1)
    g, u, d = rng.standard_normal(400) * 4, rng.standard_normal(400), rng.standard_normal(400)
    f = lambda g_, u_: d * g_ / (1 + np.exp(-g_)) * u_   # noqa: E731
    s, h = 1 / (1 + np.exp(-g)), 1e-5
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    # central differences of a function whose third derivative is under 1: off by h^2, and 1e-16 / h of rounding
    assert np.all(np.abs((f(g + h, u) - f(g - h, u)) / (2 * h) - dg) <= 1e-9 * (1 + np.abs(d * u)) * (1 + np.abs(g)))
    assert np.all(np.abs((f(g, u + h) - f(g, u - h)) / (2 * h) - du) <= 1e-9 * (1 + np.abs(d * g)) * (1 + np.abs(u)))


# ------------------------------------------------------------------------------------------- the choice of the kernel

def _choices(tmp_path, lines):
    exe = str(tmp_path / "shapes")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "mxfp8_weight_repack_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host_grouped_shapes.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True).stdout
    return [r.rsplit(" ", 1) for r in out.splitlines()]


def test_every_grouped_kernel_has_its_size(tmp_path):
    """Each size of tests/grouped_sizes.py runs the kernel it is named after, and no drawn size runs another."""
    def line(name, counts, n, k):
        words = name.split()
        return f"{words[1]} {len(counts)} {sum(counts)} {n} {k} {int(words[2] == 'bf16')}"
    got = _choices(tmp_path, [line(n, *s) for n, s in SIZES.items()])
    assert [g[0] for g in got] == list(SIZES)
    rng = np.random.default_rng(0)
    lines = []
    for _ in range(4000):
        form = str(rng.choice(["nt", "nn", "gated"]))
        p, n, k = (int(2 ** rng.uniform(0, top)) for top in (20, 13, 14))
        n, k = (-(-n // 32) * 32 if form != "nt" else n), -(-k // 32) * 32
        lines.append(f"{form} {int(2 ** rng.uniform(0, 10))} {p} {n} {k} {int(form == 'gated' or rng.random() < 0.5)}")
    names, tiles = zip(*_choices(tmp_path, lines))
    assert set(names) <= set(SIZES)
    # a launch has under 2^32 threads, of 512 at most
    assert max(int(t) for t in tiles) < 1 << 23
