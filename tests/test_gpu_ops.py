"""GPU parity of the operators around the update -- gradient norm and clip, MXFP8
quantisation, residual RMS norm and its gradient, MXFP8 products -- against
float64 references (tests/ops_ref.py) and the oracle's codes, at sizes and
values where they can go wrong."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import ops_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def stream():
    return torch.cuda.current_stream().cuda_stream


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def buf(*shape, dtype=torch.uint8, fill=0xA5):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


def work(n):
    """Workspace of exactly n bytes with stale contents (0xFF: NaN as floats)."""
    return buf(max(n, 16), fill=0xFF)


# ------------------------------------------------------------------ norm and clip

def unit(offset, rows, cols, stride=None, opt="adamw", parent=-1):
    return dict(parent=parent, offset=offset, rows=rows, cols=cols, row_stride=stride or cols, is_unit=True,
                optimizer=opt, quantize=None)


def _unit_mask(nodes, n):
    m = np.zeros(n, bool)
    for d in nodes:
        for i in range(d["rows"]):
            m[d["offset"] + i * d["row_stride"]:d["offset"] + i * d["row_stride"] + d["cols"]] = True
    return m


TREES = {
    "one element": ([unit(5, 1, 1)], 8),
    "whole root": ([unit(0, 1, 4096)], 4096),
    "odd runs": ([unit(1, 1, 3), unit(7, 1, 4097), unit(4105, 1, 2), unit(4200, 1, 8191)], 13000),
    "touching heads": ([unit(64 * h, 96, 64, 256, opt="muon") for h in range(4)], 96 * 256),
    "strided, gaps": ([unit(3, 50, 33, 41), unit(2100, 7, 5, 9), unit(2304, 64, 64, opt="muon")], 8192),
    "many": ([unit(40 * i, 1, 1 + (7 * i) % 40) for i in range(500)], 20000),
    "large": ([unit(0, 1, 9_000_001), unit(9_000_004, 3000, 1000)], 12_000_016),
}


def _clip(nodes, n, g, max_norm, in_place=False, split=False):
    plan = sh.Plan(nodes, n)
    gd = dev(g)
    out = gd if in_place else torch.full_like(gd, 7.0)
    stats = buf(2, dtype=torch.float32, fill=-1.0)
    nb = sh.grad_workspace(plan)
    ws = work(nb)
    if split:
        s = buf(2, dtype=torch.float64, fill=-1.0)
        sh.grad_sumsq(plan, gd, s, ws, nb, stream())
        sh.grad_clip(plan, gd, out, s, max_norm, stats, stream())
    else:
        sh.grad_clip_norm(plan, gd, out, max_norm, stats, ws, nb, stream())
    return host(out), host(stats)


@pytest.mark.parametrize("max_norm", [0.37, 1e6])
@pytest.mark.parametrize("tree", sorted(TREES))
def test_clip_against_float64(tree, max_norm):
    say(f"clip {tree} max {max_norm}")
    nodes, n = TREES[tree]
    rng = np.random.default_rng(len(tree))
    g = rng.standard_normal(n).astype(np.float32)
    mask = _unit_mask(nodes, n)
    g[~mask] = np.nan                                  # gaps are neither read ...
    norm = np.sqrt(np.sum(g[mask].astype(np.float64) ** 2))
    coef = float(np.float32(max_norm)) / norm if norm > np.float32(max_norm) else 1.0
    for kw in (dict(), dict(in_place=True), dict(split=True)):
        out, stats = _clip(nodes, n, g, max_norm, **kw)
        # one rounding to float32 each; float64 sums add less than 1% of one
        assert abs(stats[0] - norm) <= 1.01 * R.U * norm
        assert abs(stats[1] - coef) <= 1.01 * R.U * coef
        ref = g[mask].astype(np.float64) * coef
        assert np.all(np.abs(out[mask] - ref) <= 2.02 * R.U * np.abs(ref) + 2.0 ** -149)
        rest = out[~mask]                              # ... nor written
        assert np.all(np.isnan(rest)) if kw.get("in_place") else np.all(rest == 7.0)


@pytest.mark.parametrize("scale", [1e-30, 1e30, 3e38])
def test_clip_of_extreme_gradients(scale):
    """Squares far outside float32's range: the norm is exact, the clip finite."""
    say(f"clip scale {scale}")
    n = 5000
    g = (np.random.default_rng(1).uniform(-1, 1, n) * scale).astype(np.float32)
    norm = np.sqrt(np.sum(g.astype(np.float64) ** 2))
    out, stats = _clip([unit(0, 1, n)], n, g, 1.0)
    want = np.float32(norm) if norm <= np.finfo(np.float32).max else np.inf
    assert stats[0] == want or abs(stats[0] - norm) <= 1.01 * R.U * norm
    coef = 1.0 / norm if norm > 1 else 1.0
    # a coefficient below float32's normal range is off by half its smallest step
    bound = 2.02 * R.U * np.abs(g * coef) + np.abs(g.astype(np.float64)) * 2.0 ** -150 + 2.0 ** -149
    assert np.all(np.abs(out - g.astype(np.float64) * coef) <= bound)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_clip_of_non_finite_gradients(bad):
    say(f"clip with {bad}")
    g = np.random.default_rng(2).standard_normal(6000).astype(np.float32)
    g[4321] = bad
    out, stats = _clip([unit(0, 1, 6000)], 6000, g, 1.0)
    ok = np.arange(6000) != 4321
    if np.isnan(bad):
        assert np.isnan(stats[0]) and stats[1] == 1.0 and np.array_equal(out[ok], g[ok])
    else:
        assert np.isinf(stats[0]) and stats[1] == 0.0 and np.all(out[ok] == 0)
    assert np.isnan(out[4321])


def test_clip_is_reproducible():
    nodes, n = TREES["large"]
    g = np.random.default_rng(3).standard_normal(n).astype(np.float32)
    a, sa = _clip(nodes, n, g, 1.0)
    b, sb = _clip(nodes, n, g, 1.0)
    c, sc = _clip(nodes, n, g, 1.0, split=True)
    assert np.array_equal(a, b, equal_nan=True) and np.array_equal(sa, sb)
    assert np.array_equal(a, c, equal_nan=True) and np.array_equal(sa, sc)


# ---------------------------------------------------------------------- quantising

def _matrix(rng, r, c, dtype, special=True):
    x = (rng.standard_normal((r, c)) * np.exp(rng.standard_normal((r, 1)))).astype(np.float32)
    x = R.as_dtype(x, dtype)
    if special and r * c >= 32 * 8:
        f = x.reshape(-1)
        f[rng.integers(0, f.size, 12)] = [np.nan, np.inf, -np.inf, -0.0, 0.0, 448.0, 449.0, 1e-40, -1e-45, 3e38,
                                          2.0 ** -126, -448.0 * 2.0 ** -20]
        x[:, :32] = np.where(rng.random((r, 1)) < 0.3, 0, x[:, :32])
        x = R.as_dtype(x, dtype)
    return x


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols,ld", [(1, 32, 32), (1, 4096, 4096), (31, 96, 104), (32, 128, 128), (33, 160, 160),
                                          (127, 1056, 1064), (129, 256, 512), (300, 64, 64), (1000, 2048, 2048)])
def test_quant_bit_exact(rows, cols, ld, dtype):
    say(f"quant {rows}x{cols} ld {ld} {dtype}")
    rng = np.random.default_rng(rows * 7 + cols)
    x = _matrix(rng, rows, cols, dtype)
    full = np.full((rows, ld), np.nan, np.float32)
    full[:, :cols] = x
    src = dev(full, dtype)
    qc, qs = R.quant_rows(x)
    tc, ts = R.quant_cols(x)
    for along in ("rows", "cols", "both"):
        c = s = ct = st = None
        if along != "cols":
            c, s = buf(rows * cols + 64), buf(rows * cols // 32 + 64)
        if along != "rows":
            ct, st = buf(tc.size + 64), buf(ts.size + 64)
        sh.quant_mxfp8(src, dtype, rows, cols, c, s, ct, st, ld=ld, stream=stream())
        for got, ref in ((c, qc), (s, qs), (ct, tc), (st, ts)):
            if got is None:
                continue
            got = host(got)
            assert np.array_equal(got[:ref.size], ref.reshape(-1)), along
            assert np.all(got[ref.size:] == 0xA5)      # nothing behind the last row


# ------------------------------------------------------------------------ RMS norm

NORM_SIZES = [(1, 32), (1, 8192), (3, 512), (5, 544), (7, 1056), (130, 2048), (33, 2080), (2, 4128), (9, 8224),
              (3, 16416), (2, 32768), (2500, 64)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_rmsnorm_codes_bit_exact(rows, cols, dtype, wdtype):
    say(f"rmsnorm {rows}x{cols} {dtype}/{wdtype}")
    rng = np.random.default_rng(rows + cols)
    ldx, ldr = cols + 8, cols + 16
    x = np.full((rows, ldx), np.nan, np.float32)
    r = np.full((rows, ldr), np.nan, np.float32)
    x[:, :cols] = _matrix(rng, rows, cols, dtype, special=False)
    r[:, :cols] = _matrix(rng, rows, cols, dtype, special=False)
    if rows > 2:
        x[1, :cols] = 0
        r[1, :cols] = 0                                # a row of zeros: eps alone
    w = R.as_dtype(1 + 0.2 * rng.standard_normal(cols), wdtype)
    for residual in (True, False):
        eps = 1e-5
        h, rstd, y = R.rmsnorm(x[:, :cols], r[:, :cols] if residual else None, w, eps, dtype)
        qc, qs = R.quant_rows(y)
        td = torch.bfloat16 if dtype == "bf16" else torch.float32
        hd, yd = buf(rows + 1, cols, dtype=td, fill=3.0), buf(rows + 1, cols, dtype=td, fill=3.0)
        c, s, rs = buf(rows + 1, cols), buf(rows + 1, cols // 32), buf(rows + 1, dtype=torch.float32, fill=3.0)
        sh.rmsnorm_mxfp8(dev(x, dtype), dev(w, wdtype), rows, cols, dtype=dtype, weight_dtype=wdtype,
                         residual=dev(r, dtype) if residual else None, h=hd if residual else None, y=yd, codes=c,
                         scales=s, rstd=rs, eps=eps, ld_x=ldx, ld_residual=ldr, stream=stream())
        if residual:
            assert np.array_equal(host(hd)[:rows], h) and np.all(host(hd)[rows] == 3.0)
        assert np.array_equal(host(c)[:rows], qc) and np.all(host(c)[rows] == 0xA5)
        assert np.array_equal(host(s)[:rows], qs) and np.all(host(s)[rows] == 0xA5)
        assert np.all(np.abs(host(rs)[:rows] - rstd) <= 1.01 * R.U * rstd) and host(rs)[rows] == 3.0
        # y in float32 may differ where the float64 product sits within its own error of a rounding border
        yr = R.as_dtype(y, dtype)
        assert np.all(np.abs(host(yd)[:rows] - yr) <= 2 * R.HALF[dtype] * np.abs(yr)) and np.all(host(yd)[rows] == 3.0)
        assert np.mean(host(yd)[:rows] != yr) <= 1e-4


def test_rmsnorm_in_place_and_alone():
    """h may be the residual itself; each output may be asked for alone."""
    rng = np.random.default_rng(5)
    rows, cols = 37, 1056
    x, r = (_matrix(rng, rows, cols, "bf16", special=False) for _ in range(2))
    w = np.ones(cols, np.float32)
    h, rstd, y = R.rmsnorm(x, r, w, 1e-6, "bf16")
    rd = dev(r, "bf16")
    sh.rmsnorm_mxfp8(dev(x, "bf16"), dev(w), rows, cols, residual=rd, h=rd, stream=stream())
    assert np.array_equal(host(rd), h)
    rs = buf(rows, dtype=torch.float32, fill=0)
    sh.rmsnorm_mxfp8(rd, dev(w), rows, cols, rstd=rs, stream=stream())
    assert np.all(np.abs(host(rs) - rstd) <= 1.01 * R.U * rstd)
    yd = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    sh.rmsnorm_mxfp8(rd, dev(w), rows, cols, y=yd, stream=stream())
    assert np.array_equal(host(yd), R.as_dtype(y, "bf16"))


def test_rmsnorm_of_non_finite_rows():
    rng = np.random.default_rng(6)
    rows, cols = 6, 256
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x[1, 40], x[2, 70], x[3, :] = np.nan, np.inf, 0.0
    x[4] *= 1e30                                       # squares beyond float32
    x[5] *= 1e-30
    w = np.ones(cols, np.float32)
    for eps in (1e-6, 0.0):
        h, rstd, y = R.rmsnorm(x, None, w, eps, "fp32")
        qc, qs = R.quant_rows(y)
        c, s = buf(rows, cols), buf(rows, cols // 32)
        sh.rmsnorm_mxfp8(dev(x), dev(w), rows, cols, dtype="fp32", codes=c, scales=s, eps=eps, stream=stream())
        assert np.array_equal(host(c), qc) and np.array_equal(host(s), qs), eps


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(4100, 96)])
def test_rmsnorm_backward_against_float64(rows, cols, dtype, wdtype):
    say(f"rmsnorm backward {rows}x{cols} {dtype}/{wdtype}")
    rng = np.random.default_rng(rows * 3 + cols)
    dy, h, dh = (_matrix(rng, rows, cols, dtype, special=False) for _ in range(3))
    w = R.as_dtype(1 + 0.2 * rng.standard_normal(cols), wdtype)
    rstd = R.rmsnorm(h, None, w, 1e-6, dtype)[1].astype(np.float32)
    nb = sh.rmsnorm_backward_workspace(rows, cols)
    base = rng.standard_normal(cols).astype(np.float32)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    for through, first in ((True, True), (False, False)):
        dx, bdx, dw, bdw = R.rmsnorm_grad(dy, h, w, rstd, dh if through else None, dtype)
        dxd, dwd = buf(rows + 1, cols, dtype=td, fill=3.0), dev(np.concatenate([base, [9.0]]).astype(np.float32))
        sh.rmsnorm_backward(dev(dy, dtype), dev(h, dtype), dev(w, wdtype), dev(rstd), dxd, dwd, rows, cols,
                            dtype=dtype, weight_dtype=wdtype, dh=dev(dh, dtype) if through else None, first=first,
                            workspace=work(nb), workspace_bytes=nb, stream=stream())
        got = host(dxd)
        assert np.all(np.abs(got[:rows] - dx) <= bdx) and np.all(got[rows] == 3.0)
        if not first:
            dw, bdw = dw + base, bdw + R.U * (np.abs(dw + base) + np.abs(base))
        got = host(dwd)
        assert np.all(np.abs(got[:cols] - dw) <= bdw) and got[cols] == 9.0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(64, 2048), (65, 96), (1000, 544), (1024, 8192), (1025, 8192), (1024, 32), (300, 16416)])
def test_rmsnorm_backward_of_few_rows_and_more(rows, cols, dtype):
    """On both sides of where one launch does it all; twice into the same weight gradient, reproducibly."""
    say(f"rmsnorm backward rows {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + 5 * cols)
    dy, h, dh = (_matrix(rng, rows, cols, dtype, special=False) for _ in range(3))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    rstd = R.rmsnorm(h, None, w, 1e-6, dtype)[1].astype(np.float32)
    dx, bdx, dw, bdw = R.rmsnorm_grad(dy, h, w, rstd, dh, dtype)
    nb, td = sh.rmsnorm_backward_workspace(rows, cols), torch.bfloat16 if dtype == "bf16" else torch.float32
    runs = []
    for _ in range(2):
        dxd, dwd = buf(rows, cols, dtype=td, fill=3.0), buf(cols, dtype=torch.float32, fill=3.0)
        for first in (True, False):
            sh.rmsnorm_backward(dev(dy, dtype), dev(h, dtype), dev(w), dev(rstd), dxd, dwd, rows, cols, dtype=dtype,
                                dh=dev(dh, dtype), first=first, workspace=work(nb), workspace_bytes=nb, stream=stream())
        assert np.all(np.abs(host(dxd) - dx) <= bdx)
        assert np.all(np.abs(host(dwd) - 2 * dw) <= 2 * bdw + R.U * np.abs(2 * dw))
        runs.append((dxd, dwd))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


@pytest.mark.parametrize("over", ["dy", "dh"])
@pytest.mark.parametrize("rows,cols", [(33, 2048), (700, 8192), (1024, 512), (1500, 1056)])
def test_rmsnorm_backward_over_its_inputs(rows, cols, over):
    """dx may be dy or dh, at any number of rows."""
    say(f"rmsnorm backward over {over} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols)
    dy, h, dh = (_matrix(rng, rows, cols, "bf16", special=False) for _ in range(3))
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    rstd = R.rmsnorm(h, None, w, 1e-6, "bf16")[1].astype(np.float32)
    dx, bdx, dw, bdw = R.rmsnorm_grad(dy, h, w, rstd, dh, "bf16")
    nb = sh.rmsnorm_backward_workspace(rows, cols)
    args = [dev(h, "bf16"), dev(w), dev(rstd)]
    for _ in range(5):
        dyd, dhd, dwd = dev(dy, "bf16"), dev(dh, "bf16"), buf(cols, dtype=torch.float32, fill=3.0)
        out = dyd if over == "dy" else dhd
        sh.rmsnorm_backward(dyd, *args, out, dwd, rows, cols, dh=dhd, workspace=work(nb), workspace_bytes=nb,
                            stream=stream())
        assert np.all(np.abs(host(out) - dx) <= bdx) and np.all(np.abs(host(dwd) - dw) <= bdw)


def test_rmsnorm_backward_in_place_and_empty():
    rng = np.random.default_rng(8)
    rows, cols = 20, 96
    dy, h, dh = (_matrix(rng, rows, cols, "fp32", special=False) for _ in range(3))
    w = np.ones(cols, np.float32)
    rstd = R.rmsnorm(h, None, w, 1e-6, "fp32")[1].astype(np.float32)
    dx, bdx, _, _ = R.rmsnorm_grad(dy, h, w, rstd, dh, "fp32")
    nb = sh.rmsnorm_backward_workspace(rows, cols)
    dwd = torch.zeros(cols, device="cuda")
    d = dev(dy)
    sh.rmsnorm_backward(d, dev(h), dev(w), dev(rstd), d, dwd, rows, cols, dtype="fp32", dh=dev(dh), workspace=work(nb),
                        workspace_bytes=nb, stream=stream())
    assert np.all(np.abs(host(d) - dx) <= bdx)
    before = host(dwd).copy()
    sh.rmsnorm_backward(None, None, None, None, None, dwd, 0, cols, first=False, stream=stream())
    assert np.array_equal(host(dwd), before)
    sh.rmsnorm_backward(None, None, None, None, None, dwd, 0, cols, first=True, stream=stream())
    assert np.all(host(dwd) == 0)


# ------------------------------------------------------------------------ products

def _operand(rng, rows, cols, layout, exact):
    """codes, flat scales and float64 values; `exact`: small whole numbers under
    scales 1 and 2, so that every partial sum is a whole number below 2^24 and
    the float32 result must be the exact one."""
    if exact:
        v = rng.choice(np.array([0x00, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0x48], np.uint8), (rows, cols))   # 0 1 2 3 -1 -2 4
        n = {"block32x32": (rows // 32) * (cols // 32)}.get(layout, rows * cols // 32)
        s = rng.choice(np.array([127, 128], np.uint8), max(n, 1))
        return v, s, R.decode(v, s, layout)
    w = (rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32)
    c, s = R.quant_weight(w, layout)
    return c, s, R.decode(c, s, layout)


def _gemm(a, b, m, n, out_dtype, op="nt", addend=None, pad=0, layouts=("rowmajor", "rowmajor"), in_place=False):
    (ac, as_), (bc, bs) = a, b
    A = sh.mx_matrix(dev(ac), dev(as_), ac.shape[0], ac.shape[1], layouts[0])
    B = sh.mx_matrix(dev(bc), dev(bs), bc.shape[0], bc.shape[1], layouts[1])
    td = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    out = buf(m + 1, n + pad, dtype=td, fill=3.0)
    ad = None
    if addend is not None:
        full = np.full((m + 1, n + pad), 3.0, np.float32)
        full[:m, :n] = addend
        ad = dev(full)
        if in_place:
            out = ad
    nb = sh.gemm_mxfp8_workspace(A, B, op=op)
    sh.gemm_mxfp8(A, B, out, out_dtype, op=op, addend=ad, ld_out=n + pad, workspace=work(nb) if nb else None,
                  workspace_bytes=nb, stream=stream())
    o = host(out)
    assert np.all(o[m] == 3.0) and np.all(o[:, n:] == 3.0)      # nothing behind the last row or column
    return o[:m, :n]


SHAPES = [(1, 1, 32), (1, 64, 64), (1, 2048, 2048), (3, 33, 160), (16, 128, 4096), (17, 100, 96), (31, 257, 1056),
          (64, 96, 512), (65, 300, 288), (100, 1000, 1000 // 32 * 32), (127, 129, 128), (256, 256, 256),
          (300, 520, 640), (513, 384, 2048), (1030, 777, 224)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_nt_exact_sums(m, n, k):
    """Whole-number operands: the float32 output must equal the exact sum."""
    say(f"gemm nt exact {m}x{n}x{k}")
    rng = np.random.default_rng(m + n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, n, k, "rowmajor", True)
    add = rng.integers(-50, 50, (m, n)).astype(np.float32)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32"), a @ b.T)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", addend=add, pad=4), a @ b.T + add)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", addend=add, pad=7, in_place=True), a @ b.T + add)


@pytest.mark.parametrize("m,n,k", [(1, 32, 32), (2, 64, 128), (33, 96, 256), (130, 544, 96), (257, 256, 1024),
                                   (64, 2048, 512), (600, 320, 288)])
def test_gemm_nn_exact_sums(m, n, k):
    say(f"gemm nn exact {m}x{n}x{k}")
    rng = np.random.default_rng(m + n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, k, n, "block32x32", True)
    lay = ("rowmajor", "block32x32")
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", "nn", layouts=lay), a @ b)
    add = rng.integers(-50, 50, (m, n)).astype(np.float32)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", "nn", addend=add, pad=3, layouts=lay), a @ b + add)


@pytest.mark.parametrize("la,lb", [("rowmajor", "tile32x4"), ("rowmajor", "block32x32"), ("tile32x4", "rowmajor"),
                                   ("block32x32", "tile32x4"), ("tile32x4", "block32x32")])
@pytest.mark.parametrize("m,n,k", [(32, 64, 128), (96, 160, 512), (288, 544, 640), (32, 2048, 1152)])
def test_gemm_scale_layouts_exact(m, n, k, la, lb):
    say(f"gemm layouts {la} {lb} {m}x{n}x{k}")
    rng = np.random.default_rng(m + n + k)
    ac, as_, a = _operand(rng, m, k, la, True)
    bc, bs, b = _operand(rng, n, k, lb, True)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", layouts=(la, lb)), a @ b.T)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_nt_against_float64(m, n, k, out):
    say(f"gemm nt {m}x{n}x{k} {out}")
    rng = np.random.default_rng(m * 5 + n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", False)
    bc, bs, b = _operand(rng, n, k, "rowmajor", False)
    ref, bound = R.product(a, b, None, out)
    got = _gemm((ac, as_), (bc, bs), m, n, out, pad=5)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("m,n,k", [(1, 64, 256), (130, 544, 96), (300, 320, 1024)])
def test_gemm_nn_against_float64(m, n, k):
    say(f"gemm nn {m}x{n}x{k}")
    rng = np.random.default_rng(m * 5 + n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", False)
    bc, bs, b = _operand(rng, k, n, "block32x32", False)
    for out in ("fp32", "bf16"):
        ref, bound = R.product(a, b.T, None, out)
        got = _gemm((ac, as_), (bc, bs), m, n, out, "nn", layouts=("rowmajor", "block32x32"))
        assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("m", [2, 40, 300])
def test_gemm_nan_blocks_and_extreme_scales(m):
    """A NaN block spoils its row (and column) alone; scales at both ends of E8M0."""
    say(f"gemm NaN blocks m {m}")
    rng = np.random.default_rng(m)
    n, k = 96, 384
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, n, k, "rowmajor", True)
    sa, sb = as_.reshape(m, k // 32), bs.reshape(n, k // 32)
    sa[1, :], sb[:, :] = 250, 10                       # 2^123 * 2^-117: finite products
    ac[1, 5 * 32:6 * 32], sa[1, 5] = 0, 0
    a, b = R.decode(ac, sa, "rowmajor"), R.decode(bc, sb, "rowmajor")
    got = _gemm((ac, sa), (bc, sb), m, n, "fp32")
    ref, bound = R.product(a, b, None, "fp32")
    assert np.all(np.abs(got - ref) <= bound)
    sa[0, 3], sb[7, 2] = 255, 255
    got = _gemm((ac, sa), (bc, sb), m, n, "fp32")
    bad = np.zeros((m, n), bool)
    bad[0, :], bad[:, 7] = True, True
    assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], _gemm((ac, sa), (bc, np.where(sb == 255, 10, sb)),
                                                                          m, n, "fp32")[~bad])


def test_gemm_empty_sizes():
    rng = np.random.default_rng(0)
    z = np.zeros((0, 64), np.uint8)
    ac, as_, a = _operand(rng, 5, 64, "rowmajor", True)
    assert _gemm((z, z.reshape(-1)), (ac, as_), 0, 5, "bf16").shape == (0, 5)
    k0 = np.zeros((5, 0), np.uint8), np.zeros(0, np.uint8)
    add = rng.standard_normal((5, 5)).astype(np.float32)
    assert np.all(_gemm(k0, k0, 5, 5, "bf16", pad=3) == 0)
    assert np.array_equal(_gemm(k0, k0, 5, 5, "fp32", addend=add, in_place=True), add)


# Of what the shape choice may pick (all of it: gemm_sizes.py): few rows, 128-tiles by one wave
# group or two, 256-tiles, each with up to 4 steps or more of 128 k, K splits where tiles are few.
PICKS = [("nt", 1, 64, 544), ("nt", 33, 64, 544), ("nt", 257, 64, 544), ("nt", 1, 64, 128), ("nt", 33, 64, 8224),
         ("nt", 257, 64, 2080), ("nt", 3000, 160, 2048), ("nt", 2050, 4128, 544), ("nt", 3001, 4127, 544),
         ("nt", 8001, 3101, 128), ("nt", 2050, 6017, 224), ("nt", 130, 8224, 1056), ("nn", 1, 64, 544),
         ("nn", 1, 160, 544), ("nn", 1, 160, 128), ("nn", 3, 160, 1056), ("nn", 5, 160, 2080), ("nn", 3000, 160, 2048),
         ("nn", 2050, 4128, 544), ("nn", 3001, 4128, 544), ("nn", 8001, 3104, 128), ("nn", 2050, 6016, 224)]


@pytest.mark.parametrize("op,m,n,k", PICKS)
def test_gemm_every_shape_exact(op, m, n, k):
    """Whole-number operands, both output types, scales at an odd address: exact sums
    (bfloat16: rounded once; its products differ by less than 2^14, so none is cut off)."""
    say(f"gemm shapes {op} {m}x{n}x{k}")
    rng = np.random.default_rng(m + 3 * n + k)
    nn = op == "nn"
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, k if nn else n, n if nn else k, "block32x32" if nn else "rowmajor", True)
    ad, bd = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    ref = (ad @ (bd if nn else bd.t())).float()
    A = sh.mx_matrix(dev(ac), dev(np.concatenate([[0], as_]).astype(np.uint8))[1:], m, k)
    B = sh.mx_matrix(dev(bc), dev(np.concatenate([[0, 0, 0], bs]).astype(np.uint8))[3:], bc.shape[0], bc.shape[1],
                     "block32x32" if nn else "rowmajor")
    nb = sh.gemm_mxfp8_workspace(A, B, op=op)
    ws = work(nb)
    add = torch.randint(-50, 50, (m, n), device="cuda").float()
    for dtype, td in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        out = buf(m, n, dtype=td, fill=3.0)
        sh.gemm_mxfp8(A, B, out, dtype, op=op, workspace=ws, workspace_bytes=nb, stream=stream())
        assert torch.equal(out, ref.to(td)), dtype
    out = add.clone()
    sh.gemm_mxfp8(A, B, out, "fp32", op=op, addend=out, workspace=ws, workspace_bytes=nb, stream=stream())
    assert torch.equal(out, ref + add)


# Up to 16 rows: 2, 4 or 8 waves by K, its end inside a wave's part, more groups of
# 16 columns than run at once, the last one short.
FEW = [(1, 1, 32), (16, 17, 2048), (5, 16421, 2016), (2, 300, 2080), (16, 8225, 4096), (7, 8200, 3552), (1, 100, 4128),
       (16, 4130, 8192), (3, 9001, 8160), (13, 4097, 7680), (1, 4112, 6176)]


@pytest.mark.parametrize("m,n,k", FEW)
def test_gemm_few_rows_exact(m, n, k):
    """Whole-number operands, scales at an odd address: the exact sums rounded once (no product is cut off)."""
    say(f"gemm few rows {m}x{n}x{k}")
    rng = np.random.default_rng(m + 3 * n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, n, k, "rowmajor", True)
    A = sh.mx_matrix(dev(ac), dev(np.concatenate([[0], as_]).astype(np.uint8))[1:], m, k)
    B = sh.mx_matrix(dev(bc), dev(np.concatenate([[0, 0, 0], bs]).astype(np.uint8))[3:], n, k)
    for ld in (n, n + 3, (n + 7) // 4 * 4):
        out = buf(m + 1, ld, dtype=torch.bfloat16, fill=3.0)
        nb = sh.gemm_mxfp8_workspace(A, B)
        sh.gemm_mxfp8(A, B, out, "bf16", ld_out=ld, workspace=work(nb), workspace_bytes=nb, stream=stream())
        assert np.array_equal(host(out)[:m, :n], R.as_dtype((a @ b.T).astype(np.float32), "bf16"))
        assert bool((out[m] == 3.0).all()) and bool((out[:, n:] == 3.0).all())


@pytest.mark.parametrize("m,n,k", FEW + [(9, 300, 1056), (16, 2100, 992), (4, 4500, 3104)])
def test_gemm_few_rows_float32(m, n, k):
    """The same in float32, with an addend and over it, against exact sums; random codes against float64."""
    say(f"gemm few rows fp32 {m}x{n}x{k}")
    rng = np.random.default_rng(m + 5 * n + k)
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, n, k, "rowmajor", True)
    add = rng.integers(-50, 50, (m, n)).astype(np.float32)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", pad=1), a @ b.T)
    for over in (False, True):
        assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", addend=add, pad=5, in_place=over), a @ b.T + add)
    sa, sb = as_.reshape(m, k // 32).copy(), bs.reshape(n, k // 32).copy()
    sa[m // 2, -1], sb[n // 2, 0], sb[n - 1, -1] = 255, 255, 255
    got = _gemm((ac, sa), (bc, sb), m, n, "fp32")
    bad = np.zeros((m, n), bool)
    bad[m // 2, :], bad[:, [n // 2, n - 1]] = True, True
    assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], (a @ b.T)[~bad])
    ac, as_, a = _operand(rng, m, k, "rowmajor", False)
    bc, bs, b = _operand(rng, n, k, "rowmajor", False)
    ref, bound = R.product(a, b, None, "fp32")
    assert np.all(np.abs(_gemm((ac, as_), (bc, bs), m, n, "fp32") - ref) <= bound)


@pytest.mark.parametrize("layout", ["tile32x4", "block32x32"])
@pytest.mark.parametrize("n,k", [(64, 640), (4128, 1920), (5024, 3968), (4160, 8064), (4320, 5376)])
def test_gemm_few_rows_in_every_layout(n, k, layout):
    say(f"gemm few rows {layout} {n}x{k}")
    rng = np.random.default_rng(n + k)
    for m in (1, 9):
        ac, as_, a = _operand(rng, m, k, "rowmajor", True)
        bc, bs, b = _operand(rng, n, k, layout, True)
        assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "bf16", layouts=("rowmajor", layout)),
                              R.as_dtype((a @ b.T).astype(np.float32), "bf16"))


@pytest.mark.parametrize("n,k", [(48, 384), (4400, 4064), (4200, 8000)])
def test_gemm_few_rows_nan_blocks_stay_in_their_row(n, k):
    """NaN scales at a row's ends, next to rows and K ends that are read around."""
    say(f"gemm few rows NaN {n}x{k}")
    rng = np.random.default_rng(n + k)
    m = 6
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, n, k, "rowmajor", True)
    clean = _gemm((ac, as_), (bc, bs), m, n, "bf16")
    assert np.array_equal(clean, R.as_dtype((a @ b.T).astype(np.float32), "bf16"))
    sa, sb = as_.reshape(m, k // 32).copy(), bs.reshape(n, k // 32).copy()
    sa[2, 0], sa[4, -1], sb[16, 0], sb[n - 2, -1], sb[31, k // 64] = 255, 255, 255, 255, 255
    got = _gemm((ac, sa), (bc, sb), m, n, "bf16")
    bad = np.zeros((m, n), bool)
    bad[[2, 4], :], bad[:, [16, n - 2, 31]] = True, True
    assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], clean[~bad])


# Rows of fewer scale bytes than a word: K under 128, and of an NN operand N under 128.
THIN = [("nt", 300, 520, 32, "rowmajor"), ("nt", 1030, 300, 96, "rowmajor"), ("nt", 257, 260, 64, "rowmajor"),
        ("nt", 3000, 2050, 32, "rowmajor"), ("nt", 300, 544, 96, "block32x32"), ("nt", 513, 1024, 32, "block32x32"),
        ("nn", 300, 32, 128, None), ("nn", 129, 64, 1056, None), ("nn", 2229, 96, 4480, None), ("nn", 40, 96, 64, None),
        ("nn", 5, 96, 2080, None), ("nn", 700, 160, 32, None), ("nn", 1, 320, 96, None), ("nn", 2500, 2048, 64, None),
        ("nn", 3, 64, 64, None), ("nn", 300, 64, 32, None)]


@pytest.mark.parametrize("op,m,n,k,layout", THIN)
def test_gemm_thin_operands(op, m, n, k, layout):
    """Exact sums, and NaN scales that spoil their own block's row or columns alone."""
    say(f"gemm thin {op} {m}x{n}x{k} {layout}")
    rng = np.random.default_rng(m + 3 * n + k)
    nn = op == "nn"
    lay = "block32x32" if nn else layout
    ac, as_, a = _operand(rng, m, k, "rowmajor", True)
    bc, bs, b = _operand(rng, k if nn else n, n if nn else k, lay, True)
    ref = (a @ (b if nn else b.T)).astype(np.float32)
    sa, sb = as_.reshape(m, k // 32).copy(), bs.copy()
    sa[m // 2, 0], sa[m - 1, -1] = 255, 255
    sb[sb.size // 2], sb[-1] = 255, 255
    bad = np.zeros((m, n), bool)
    bad[[m // 2, m - 1], :] = True
    for i in (sb.size // 2, sb.size - 1):
        if nn:
            bad[:, i % (n // 32) * 32:i % (n // 32) * 32 + 32] = True
        elif lay == "block32x32":
            bad[:, i // (k // 32) * 32:i // (k // 32) * 32 + 32] = True
        else:
            bad[:, i // (k // 32)] = True
    lays = ("rowmajor", lay)
    for out in ("fp32", "bf16"):
        assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, out, op, layouts=lays, pad=3), R.as_dtype(ref, out)), out
        got = _gemm((ac, sa), (bc, sb), m, n, out, op, layouts=lays)
        assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], R.as_dtype(ref, out)[~bad]), out
    add = rng.integers(-50, 50, (m, n)).astype(np.float32)
    assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", op, addend=add, layouts=lays, in_place=True), ref + add)


@pytest.mark.parametrize("n,k", [(64, 640), (2080, 1152), (160, 4224)])
@pytest.mark.parametrize("layout", ["tile32x4", "block32x32"])
def test_gemm_long_rows_in_every_layout(n, k, layout):
    """The weight's layouts where rows take several quads of steps, the last one short."""
    say(f"gemm long rows {layout} {n}x{k}")
    rng = np.random.default_rng(n + k)
    for m in (1, 40, 384):
        ac, as_, a = _operand(rng, m, k, "rowmajor", True)
        bc, bs, b = _operand(rng, n, k, layout, True)
        assert np.array_equal(_gemm((ac, as_), (bc, bs), m, n, "fp32", layouts=("rowmajor", layout)), a @ b.T)


# ----------------------------------------------------------------- together, and shared

class Layer:
    """Norm, up and down projection of a small block on a plan: weights in 32 x 32 blocks,
    two microbatches of a ragged token count, then clip and update."""
    M, D, F = 77, 128, 256

    def __init__(self, seed=0):
        D, F = self.D, self.F
        q = dict(parent=-1, is_unit=True, optimizer="muon", quantize=True)
        nodes = [dict(q, offset=0, rows=F, cols=D, row_stride=D), dict(q, offset=F * D, rows=D, cols=F, row_stride=F),
                 dict(parent=-1, offset=2 * F * D, rows=1, cols=D, row_stride=D, is_unit=True, optimizer="adamw",
                      quantize=None)]
        self.n = 2 * F * D + D
        self.plan = sh.Plan(nodes, self.n, layout="block32x32")
        st = self.plan.stats()
        rng = np.random.default_rng(seed)
        w = rng.standard_normal(self.n).astype(np.float32) * 0.05
        w[2 * F * D:] = 1 + 0.1 * rng.standard_normal(D)
        self.w, self.g, self.gc = dev(w), torch.zeros(self.n, device="cuda"), torch.zeros(self.n, device="cuda")
        self.m, self.v = torch.zeros(self.n, device="cuda"), torch.zeros(self.n, device="cuda")
        self.codes, self.scales = buf(self.n, fill=0), buf(st["scale_bytes"], fill=0)
        self.x = [dev(rng.standard_normal((self.M, D)).astype(np.float32), "bf16") for _ in range(2)]
        self.res = [dev(rng.standard_normal((self.M, D)).astype(np.float32), "bf16") for _ in range(2)]
        self.dy = [dev(rng.standard_normal((self.M, D)).astype(np.float32) * 0.01, "bf16") for _ in range(2)]
        self.ws_bytes = max(st["workspace_bytes"], sh.grad_workspace(self.plan), 1 << 20)
        self.ws, self.stats = buf(self.ws_bytes), buf(2, dtype=torch.float32, fill=0)
        self.W1, self.W2 = (self.plan.mx_matrix(i, self.codes, self.scales) for i in (0, 1))
        sh.requant_mxfp8(self.plan, self.w, self.codes, self.scales, stream())
        M, P = self.M, (self.M + 31) // 32 * 32
        b16 = dict(dtype=torch.bfloat16)
        self.t = {"h": buf(M, D, **b16), "y": buf(M, D, **b16), "rstd": buf(M, dtype=torch.float32), "a": buf(M, F, **b16),
                  "out": buf(M, D, dtype=torch.float32), "da": buf(M, F, **b16), "dn": buf(M, D, **b16), "dx": buf(M, D, **b16)}
        for name, r, c in (("yq", M, D), ("aq", M, F), ("dyq", M, D), ("daq", M, F)):
            self.t[name], self.t[name + "_s"] = buf(r, c), buf(r, c // 32)
        for name, r in (("yt", D), ("at", F), ("dyt", D), ("dat", F)):
            self.t[name], self.t[name + "_s"] = buf(r, P), buf(r, P // 32)

    def mat(self, name):
        return sh.mx_matrix(self.t[name], self.t[name + "_s"], *self.t[name].shape)

    def gemm(self, a, b, out, dtype, op="nt", addend=None):
        assert sh.gemm_mxfp8_workspace(a, b, op=op) <= self.ws_bytes
        sh.gemm_mxfp8(a, b, out, dtype, op=op, addend=addend, workspace=self.ws, workspace_bytes=self.ws_bytes,
                      stream=stream())

    def quant(self, src, rows, cols, name=None, name_t=None):
        q = [self.t[n] if n else None for n in (name, name and name + "_s", name_t, name_t and name_t + "_s")]
        sh.quant_mxfp8(src, "bf16", rows, cols, *q, stream=stream())

    def microbatch(self, i):
        t, M, D, F, s = self.t, self.M, self.D, self.F, stream()
        gamma = self.w[2 * F * D:]
        sh.rmsnorm_mxfp8(self.x[i], gamma, M, D, residual=self.res[i], h=t["h"], y=t["y"], codes=t["yq"],
                         scales=t["yq_s"], rstd=t["rstd"], stream=s)
        self.gemm(self.mat("yq"), self.W1, t["a"], "bf16")
        self.quant(t["a"], M, F, "aq", "at")
        self.gemm(self.mat("aq"), self.W2, t["out"], "fp32")
        self.quant(self.dy[i], M, D, "dyq", "dyt")
        self.gemm(self.mat("dyq"), self.W2, t["da"], "bf16", "nn")
        g1, g2, g3 = self.g[:F * D], self.g[F * D:2 * F * D], self.g[2 * F * D:]
        self.gemm(self.mat("dyt"), self.mat("at"), g2, "fp32", addend=g2 if i else None)
        self.quant(t["da"], M, F, "daq", "dat")
        self.quant(t["y"], M, D, None, "yt")
        self.gemm(self.mat("daq"), self.W1, t["dn"], "bf16", "nn")
        self.gemm(self.mat("dat"), self.mat("yt"), g1, "fp32", addend=g1 if i else None)
        sh.rmsnorm_backward(t["dn"], t["h"], gamma, t["rstd"], t["dx"], g3, M, D, dh=self.dy[i], first=i == 0,
                            workspace=self.ws, workspace_bytes=self.ws_bytes, stream=s)

    def step(self):
        for i in range(2):
            self.microbatch(i)
        sh.grad_clip_norm(self.plan, self.g, self.gc, 0.5, self.stats, self.ws, self.ws_bytes, stream())
        sh.update_step(self.plan, sh.buffers(self.w, self.gc, self.m, self.v, self.codes, self.scales), sh.muon_hp(),
                       sh.adamw_hp(), 1, self.ws, self.ws_bytes, stream())

    def state(self):
        torch.cuda.synchronize()
        return {k: getattr(self, k).clone() for k in ("w", "g", "gc", "m", "v", "codes", "scales", "stats")} | \
            {k: v.clone() for k, v in self.t.items()}


def test_a_layer_forwards_backwards_and_updates():
    """Every operator's result inside the run, each against its reference on the run's own inputs."""
    say("layer")
    L = Layer()
    t, M, D, F = L.t, L.M, L.D, L.F
    w0 = host(L.w).copy()
    wq = [R.decode(host(L.codes)[i * F * D:(i + 1) * F * D].reshape(s), host(L.scales)[i * F * D // 1024:], "block32x32")
          for i, s in ((0, (F, D)), (1, (D, F)))]
    grads = np.zeros(L.n)
    bounds = np.zeros(L.n)
    for i in range(2):
        L.microbatch(i)
        T = {k: host(v) for k, v in t.items()}
        dec = lambda n: R.decode(T[n], T[n + "_s"], "rowmajor")   # noqa: E731
        h, rstd, y = R.rmsnorm(host(L.x[i]), host(L.res[i]), w0[2 * F * D:], 1e-6, "bf16")
        assert np.array_equal(T["h"], h) and np.array_equal(T["yq"], R.quant_rows(y)[0])
        for got, (a, b), dtype in ((T["a"], (dec("yq"), wq[0]), "bf16"), (T["out"], (dec("aq"), wq[1]), "fp32"),
                                   (T["da"], (dec("dyq"), wq[1].T), "bf16"), (T["dn"], (dec("daq"), wq[0].T), "bf16")):
            ref, bound = R.product(a, b, None, dtype)
            assert np.all(np.abs(got - ref) <= bound)
        assert np.array_equal(T["at"], R.quant_cols(T["a"])[0]) and np.array_equal(T["dat_s"], R.quant_cols(T["da"])[1])
        for off, (a, b) in ((0, ("dat", "yt")), (F * D, ("dyt", "at"))):
            ref, bound = R.product(dec(a), dec(b), None, "fp32")
            grads[off:off + F * D] += ref.reshape(-1)
            bounds[off:off + F * D] += bound.reshape(-1)
        dx, bdx, dw, bdw = R.rmsnorm_grad(T["dn"], T["h"], w0[2 * F * D:], T["rstd"], host(L.dy[i]), "bf16")
        assert np.all(np.abs(T["dx"] - dx) <= bdx)
        grads[2 * F * D:] += dw
        bounds[2 * F * D:] += bdw
    # the second microbatch's addition rounds once more
    g = host(L.g)
    assert np.all(np.abs(g - grads) <= bounds + 2 * R.U * np.abs(grads))
    M2 = Layer()
    M2.step()
    assert torch.equal(M2.g, L.g)                      # the same run again, to the bit
    norm = np.sqrt(np.sum(g.astype(np.float64) ** 2))
    assert norm > 0.5 and abs(host(M2.stats)[0] - norm) <= 1.01 * R.U * norm
    assert np.all(np.abs(host(M2.gc) - g * (0.5 / norm)) <= 2.02 * R.U * np.abs(g))
    # the update's codes are G of its new weights, and the next forward reads them
    assert not np.array_equal(host(M2.w), w0)
    for i, s in ((0, (F, D)), (1, (D, F))):
        c, _ = R.quant_weight(host(M2.w)[i * F * D:(i + 1) * F * D].reshape(s), "block32x32")
        assert np.array_equal(host(M2.codes)[i * F * D:(i + 1) * F * D].reshape(s), c)


def test_a_step_captured_in_a_hip_graph():
    """Forward, backward, clip and update captured once and replayed three times on new
    inputs, with eager work between, each replay against an eager step from the same state."""
    say("layer graph")
    G, E = Layer(1), Layer(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.step()                                       # warm up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    E.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        G.step()
    for rep in range(3):
        rng = np.random.default_rng(10 + rep)
        for L in (G, E):
            r = np.random.default_rng(10 + rep)
            for k in range(2):
                L.x[k].copy_(dev(r.standard_normal((L.M, L.D)).astype(np.float32), "bf16"))
                L.dy[k].copy_(dev(r.standard_normal((L.M, L.D)).astype(np.float32) * 0.01, "bf16"))
        graph.replay()
        E.step()
        torch.cuda.synchronize()
        a, b = G.state(), E.state()
        for k in a:
            assert torch.equal(a[k], b[k]) or (a[k].is_floating_point() and torch.equal(a[k].nan_to_num(), b[k].nan_to_num())), (rep, k)
        del rng


def test_two_streams_at_once():
    """Two layers' steps on two streams, issued in turn, give what each gives alone."""
    say("two streams")
    alone = []
    for seed in (2, 3):
        L = Layer(seed)
        L.step()
        alone.append(L.state())
    layers, streams = [Layer(2), Layer(3)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for L, s in zip(layers, streams):
        with torch.cuda.stream(s):
            L.step()
    torch.cuda.synchronize()
    for L, a in zip(layers, alone):
        b = L.state()
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_foreign_pointers_are_refused():
    """Host memory that the runtime does not know is an argument error, not a GPU fault."""
    h = torch.zeros(64, 64)
    d = torch.zeros(64, 64, device="cuda")
    u = torch.zeros(64 * 64, dtype=torch.uint8, device="cuda")
    p = h.data_ptr() + (-h.data_ptr() % 16)
    node = unit(0, 1, 64)
    plan = sh.Plan([node], 64)
    m = sh.mx_matrix(u, u, 32, 64)
    for call in (lambda: sh.quant_mxfp8(p, "fp32", 4, 64, u, u, stream=stream()),
                 lambda: sh.rmsnorm_mxfp8(d, p, 4, 64, dtype="fp32", y=d, stream=stream()),
                 lambda: sh.gemm_mxfp8(m, m, p, "fp32", stream=stream()),
                 lambda: sh.gemm_mxfp8(sh.mx_matrix(u, p, 32, 64), m, d, "fp32", stream=stream()),
                 lambda: sh.grad_clip_norm(plan, d, d, 1.0, d, p, 1 << 20, stream()),
                 lambda: sh.grad_clip_norm(plan, p, d, 1.0, d, u, 4096, stream())):
        with pytest.raises(sh.SshdpError) as e:
            call()
        assert e.value.name == "ARG"
    torch.cuda.synchronize()


# ------------------------------------------------------------------ past 32-bit offsets

def _codes(rows, cols, seed=0):
    """Codes of 1, 2 and 4 and scales of 1 and 2, made on the GPU: exact sums."""
    torch.manual_seed(seed)
    c = torch.randint(0, 3, (rows, cols), dtype=torch.uint8, device="cuda").mul_(8).add_(0x38)
    return c, torch.randint(127, 129, (rows, cols // 32), dtype=torch.uint8, device="cuda")


def _mm(a, b, m, n, dtype="fp32", op="nt"):
    out = torch.full((m, n), 3.0, dtype=torch.float32 if dtype == "fp32" else torch.bfloat16, device="cuda")
    nb = sh.gemm_mxfp8_workspace(a, b, op=op)
    sh.gemm_mxfp8(a, b, out, dtype, op=op, workspace=work(nb), workspace_bytes=nb, stream=stream())
    return out


def test_rows_past_32_bit_offsets():
    """The last rows of matrices of more than 2^32 elements are what they are alone."""
    rows, cols, cut = 140001, 32768, 139872             # cut: a multiple of 32
    n = rows - cut
    say("quant past 2^32")
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    c, s = buf(rows, cols), buf(rows, cols // 32)
    ct, st = buf(cols, (rows + 31) // 32 * 32), buf(cols, (rows + 31) // 32)
    sh.quant_mxfp8(x, "bf16", rows, cols, c, s, ct, st, stream=stream())
    c1, s1, ct1, st1 = buf(n, cols), buf(n, cols // 32), buf(cols, (n + 31) // 32 * 32), buf(cols, (n + 31) // 32)
    sh.quant_mxfp8(x[cut:], "bf16", n, cols, c1, s1, ct1, st1, stream=stream())
    assert torch.equal(c[cut:], c1) and torch.equal(s[cut:], s1)
    assert torch.equal(ct[:, cut:], ct1) and torch.equal(st[:, cut // 32:], st1)
    c.fill_(0xA5)
    sh.quant_mxfp8(x, "bf16", rows, cols, c, s, stream=stream())
    assert torch.equal(c[cut:], c1)
    del ct, st
    say("rmsnorm past 2^32")
    w = torch.ones(cols, device="cuda")
    h, rs = torch.empty_like(x), torch.empty(rows, device="cuda")
    sh.rmsnorm_mxfp8(x, w, rows, cols, residual=x, h=h, codes=c, scales=s, rstd=rs, stream=stream())
    h1, rs1 = torch.empty_like(x[cut:]), torch.empty(n, device="cuda")
    sh.rmsnorm_mxfp8(x[cut:], w, n, cols, residual=x[cut:], h=h1, codes=c1, scales=s1, rstd=rs1, stream=stream())
    assert torch.equal(h[cut:], h1) and torch.equal(rs[cut:], rs1)
    assert torch.equal(c[cut:], c1) and torch.equal(s[cut:], s1)
    say("rmsnorm backward past 2^32")
    x[:-1] = 0                                          # dy: the last row alone, so its weight gradient is exact
    dw, dw1 = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    nb = sh.rmsnorm_backward_workspace(rows, cols)
    dx = torch.empty_like(x)
    sh.rmsnorm_backward(x, h, w, rs, dx, dw, rows, cols, workspace=work(nb), workspace_bytes=nb, stream=stream())
    dx1 = torch.empty_like(x[cut:])
    sh.rmsnorm_backward(x[cut:], h1, w, rs1, dx1, dw1, n, cols, workspace=work(nb), workspace_bytes=nb, stream=stream())
    assert torch.equal(dx[cut:], dx1) and torch.equal(dw, dw1) and bool((dw != 0).any())


def test_products_past_32_bit_offsets():
    rows, k, cut = 140001, 32768, 139700
    n = rows - cut
    c, s = _codes(rows, k)
    big, tail = sh.mx_matrix(c, s, rows, k), sh.mx_matrix(c[cut:], s[cut:], n, k)
    for m in (5, 100, 300):                             # few rows, and tiles
        say(f"operand past 2^32, m {m}")
        a = sh.mx_matrix(*_codes(m, k, 1), m, k)
        for dtype in ("fp32", "bf16"):
            assert torch.equal(_mm(a, big, m, rows, dtype)[:, cut:], _mm(a, tail, m, n, dtype))
            assert torch.equal(_mm(big, a, rows, m, dtype)[cut:], _mm(tail, a, n, m, dtype))
    del c, s, big, tail
    say("nn operand past 2^32")
    rows, cut = 140032, 139712
    n = rows - cut
    c = _codes(k, rows)[0]
    s = torch.randint(127, 129, (k // 32, rows // 32), dtype=torch.uint8, device="cuda")
    big = sh.mx_matrix(c, s, k, rows, "block32x32")
    tail = sh.mx_matrix(c[:, cut:].t().contiguous(), s[:, cut // 32:].t().contiguous(), n, k, "block32x32")
    a = sh.mx_matrix(*_codes(300, k, 1), 300, k)
    for dtype in ("fp32", "bf16"):
        assert torch.equal(_mm(a, big, 300, rows, dtype, "nn")[:, cut:], _mm(a, tail, 300, n, dtype))
    del c, s, big, tail
    say("output past 2^32")
    m, n, k, cut = 70001, 65536, 256, 69800
    c, s = _codes(m, k)
    b = sh.mx_matrix(*_codes(n, k, 1), n, k)
    for dtype in ("fp32", "bf16"):
        assert torch.equal(_mm(sh.mx_matrix(c, s, m, k), b, m, n, dtype)[cut:],
                           _mm(sh.mx_matrix(c[cut:], s[cut:], m - cut, k), b, m - cut, n, dtype))


def test_narrow_outputs_of_very_many_rows():
    """More workgroups than one launch may have threads for."""
    say("2^27 + 5 rows")
    m, n, k = (1 << 27) + 5, 32, 32
    c, s = _codes(m, k)
    for op in ("nt", "nn"):
        b = sh.mx_matrix(_codes(32, 32, 1)[0], torch.full((32,), 127, dtype=torch.uint8, device="cuda"), 32, 32,
                         "rowmajor" if op == "nt" else "block32x32")
        out = _mm(sh.mx_matrix(c, s, m, k), b, m, n, "bf16", op)
        for at in [i << 22 for i in range(0, 32)] + [m - 40]:
            lo, hi = max(at - 40, 0), min(at + 40, m)
            assert torch.equal(out[lo:hi], _mm(sh.mx_matrix(c[lo:hi], s[lo:hi], hi - lo, k), b, hi - lo, n, "bf16", op))


def test_clip_past_32_bit_offsets():
    say("clip past 2^32")
    n, at = (1 << 32) + 3_000_000, (1 << 32) - 1_000_003
    plan = sh.Plan([unit(1, 1, 1000), unit(at, 1, 3_000_001)], n)
    g = torch.full((n,), float("nan"), device="cuda")
    for lo, ln in ((1, 1000), (at, 3_000_001)):
        g[lo:lo + ln].normal_()
    own = torch.cat([g[1:1001], g[at:at + 3_000_001]])
    out, stats, nb = torch.full_like(g, 7.0), buf(2, dtype=torch.float32, fill=0), sh.grad_workspace(plan)
    sh.grad_clip_norm(plan, g, out, 0.5, stats, work(nb), nb, stream())
    norm = float(own.double().norm())
    st = host(stats)
    assert abs(st[0] - norm) <= 2 * R.U * norm and abs(st[1] - 0.5 / norm) <= 4 * R.U * st[1]
    assert torch.equal(torch.cat([out[1:1001], out[at:at + 3_000_001]]), own * float(st[1]))
    assert bool((out[1001:at] == 7.0).all()) and bool((out[at + 3_000_001:] == 7.0).all())
