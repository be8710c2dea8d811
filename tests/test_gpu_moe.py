"""GPU parity of the expert layer's operators -- slots sorted by expert, rows gathered with G behind, the weighted sum
back and its gradient -- against plain references (tests/moe_ref.py) and the oracle's codes, at sizes, choices and
values where they can go wrong."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import moe_ref as M
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


def choices(rng, tokens, top_k, experts, how):
    if how == "spread":
        return rng.integers(0, experts, (tokens, top_k))
    if how == "dropped":                               # a third of them name no expert of ours
        return rng.integers(-experts // 4 - 1, experts + experts // 4 + 1, (tokens, top_k))
    if how == "none":
        return np.full((tokens, top_k), -1)
    if how == "one":
        return np.full((tokens, top_k), experts - 1)
    return np.minimum(rng.geometric(0.2, (tokens, top_k)) - 1, experts - 1)   # skewed


def sort(ids, tokens, top_k, experts, align, rows=None, i64=False):
    rows = sh.moe_rows(tokens, top_k, experts, align) if rows is None else rows
    i32 = dict(dtype=torch.int32, fill=-7)
    offsets, place, source = buf(experts + 1, **i32), buf(max(tokens * top_k, 1), **i32), buf(max(rows, 1), **i32)
    n = sh.moe_sort_workspace(tokens, top_k, experts)
    ws = buf(max(n, 16), fill=0xFF)
    sh.moe_sort(dev(np.asarray(ids, np.int64 if i64 else np.int32)), tokens, top_k, experts, offsets, place, source, rows,
                align=align, ids_dtype="int64" if i64 else "int32", workspace=ws, workspace_bytes=n, stream=stream())
    return offsets, place, source, rows


# ---------------------------------------------------------------------------------------------------------------- sort

@pytest.mark.parametrize("how", ["spread", "dropped", "none", "one", "skewed"])
@pytest.mark.parametrize("tokens,top_k,experts,align", [
    (1, 1, 1, 1), (1, 6, 64, 1), (1, 1, 1024, 256), (21, 3, 2, 2), (16, 6, 64, 32), (64, 1, 63, 1), (65, 1, 65, 32),
    (683, 6, 64, 32), (4096, 1, 256, 16), (4097, 1, 257, 32), (5000, 8, 8, 1), (1000, 64, 1000, 4),
    (16381, 6, 64, 32), (44001, 6, 17, 128)])
def test_sort(tokens, top_k, experts, align, how):
    say(f"sort {tokens} x {top_k} to {experts}, align {align}, {how}")
    rng = np.random.default_rng(tokens + top_k)
    ids = choices(rng, tokens, top_k, experts, how)
    for i64 in (False, True):
        got = sort(ids, tokens, top_k, experts, align, i64=i64)
        want = M.sort(ids, experts, align, got[3])
        for g, w, name in zip(got, want, ("offsets", "place", "source")):
            np.testing.assert_array_equal(host(g)[:w.size], w, err_msg=name)


@pytest.mark.parametrize("slots", [1, 63, 64, 65, 1023, 1024, 1025, 2047, 2048, 2049])
def test_sort_where_the_split_changes(slots):
    ids = np.random.default_rng(slots).integers(-1, 40, (slots, 1))
    got = sort(ids, slots, 1, 39, 32)
    for g, w in zip(got, M.sort(ids, 39, 32, got[3])):
        np.testing.assert_array_equal(host(g)[:len(w)], w)


def test_sort_of_wide_ids_and_roomy_buffers():
    """64-bit ids whose low halves name experts are dropped; more rows than needed are filled with -1."""
    say("sort, wide ids")
    ids = np.array([[3, (1 << 32) + 3], [-(1 << 63), (1 << 63) - 1], [-(1 << 32), 0], [1 << 31, 3]], np.int64)
    got = sort(ids, 4, 2, 4, 32, rows=1000, i64=True)
    want = M.sort(ids, 4, 32, 1000)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(host(g), w)
    i32 = np.array([[-(1 << 31), (1 << 31) - 1, 2]], np.int32)
    got = sort(i32, 1, 3, 3, 1)
    for g, w in zip(got, M.sort(i32, 3, 1, 3)):
        np.testing.assert_array_equal(host(g), w)


def test_sort_of_no_tokens():
    say("sort of nothing")
    offsets, _, source, _ = sort(np.zeros((0, 2)), 0, 2, 5, 1, rows=37)
    assert not host(offsets).any() and (host(source) == -1).all()


def test_sort_of_many_slots():
    """Past 2^18 slots a workgroup takes more than 1024; the order is a stable sort's."""
    say("sort of 2^24 slots")
    tokens, top_k, experts = (1 << 24) // 8, 8, 129
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(-3, experts, (tokens * top_k,), generator=g, device="cuda", dtype=torch.int32)
    n = sh.moe_sort_workspace(tokens, top_k, experts)
    rows = sh.moe_rows(tokens, top_k, experts, 32)
    i32 = dict(dtype=torch.int32, fill=-7)
    offsets, place, source = buf(experts + 1, **i32), buf(tokens * top_k, **i32), buf(rows, **i32)
    sh.moe_sort(ids, tokens, top_k, experts, offsets, place, source, rows, align=32, workspace=buf(n),
                workspace_bytes=n, stream=stream())
    key = torch.where(ids < 0, experts, ids).long()
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    ends = torch.cumsum((counts + 31) // 32 * 32, 0)
    assert torch.equal(offsets[1:].long(), ends) and int(offsets[0]) == 0
    order = torch.sort(key, stable=True).indices
    live = order[:int(counts.sum())]
    assert torch.equal(source[source >= 0].long(), live)
    assert torch.equal(place[live].long(), torch.nonzero(source >= 0).view(-1))
    assert bool((place[order[live.numel():]] == -1).all())


# -------------------------------------------------------------------------------------------------------------- gather

def _x(rng, tokens, cols, dtype):
    return R.as_dtype(rng.standard_normal((tokens, cols)) * np.exp(rng.standard_normal((tokens, 1))), dtype)


SIZES = [(1, 1, 1, 32, 1), (1, 6, 64, 2048, 1), (3, 2, 4, 96, 32), (37, 5, 7, 160, 1), (37, 5, 7, 160, 32),
         (130, 2, 3, 544, 32), (129, 8, 16, 256, 64), (515, 3, 9, 1408, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,top_k,experts,cols,align", SIZES)
def test_gather(tokens, top_k, experts, cols, align, dtype):
    say(f"gather {tokens} x {top_k} of {cols} to {experts}, align {align}, {dtype}")
    rng = np.random.default_rng(cols + tokens)
    ids = choices(rng, tokens, top_k, experts, "dropped")
    ld = cols + 32
    x = _x(rng, tokens, ld, dtype)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    offsets, _, source, rows = sort(ids, tokens, top_k, experts, align)
    rows_t = rows % 32 == 0
    xd, end = dev(x, dtype), int(host(offsets)[-1])
    for weights in (None, w):
        y = M.gather(x[:, :cols], weights, host(source), host(offsets), top_k)
        wd = None if weights is None else dev(weights)
        codes, scales = R.quant_rows(y)
        full = np.arange(rows) < end
        c, s, yd = buf(rows, cols), buf(rows, cols // 32), buf(rows, cols, dtype=xd.dtype, fill=3.0)
        ct, st = buf(cols, max(rows, 1)), buf(cols, max(rows // 32, 1))
        common = dict(dtype=dtype, weights=wd, ld_x=ld, stream=stream())
        sh.moe_gather_mxfp8(xd, source, offsets, tokens, top_k, experts, rows, cols, codes=c, scales=s, y=yd, **common)
        np.testing.assert_array_equal(host(c), np.where(full[:, None], codes, 0xA5))
        np.testing.assert_array_equal(host(s), np.where(full[:, None], scales, 0xA5))
        np.testing.assert_array_equal(host(yd), np.where(full[:, None], R.as_dtype(y, dtype), 3.0))
        if not rows_t or not rows:
            continue
        codes_t, scales_t = R.quant_cols(y)
        blocks = np.arange(rows // 32) * 32 < end
        for both in (False, True):
            c2, s2, y2 = buf(rows, cols), buf(rows, cols // 32), buf(rows, cols, dtype=xd.dtype, fill=3.0)
            ct.fill_(0xA5), st.fill_(0xA5)
            kw = dict(codes=c2, scales=s2, y=y2) if both else {}
            sh.moe_gather_mxfp8(xd, source, offsets, tokens, top_k, experts, rows, cols, codes_t=ct, scales_t=st, **kw,
                                **common)
            np.testing.assert_array_equal(host(ct), np.where(np.repeat(blocks, 32)[None], codes_t, 0xA5))
            np.testing.assert_array_equal(host(st), np.where(blocks[None], scales_t, 0xA5))
            if both:
                assert torch.equal(c2, c) and torch.equal(s2, s) and torch.equal(y2, yd)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,cols", [(1, 32), (16, 96), (333, 2080), (2100, 2048)])
def test_gather_of_any_set_of_outputs(tokens, cols, weighted, dtype):
    """Each output alone, and with the others: one set of bits, whichever kernel makes it."""
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, 8, (tokens, 3))
    offsets, _, source, rows = sort(ids, tokens, 3, 8, 32)
    x = dev(rng.standard_normal((tokens, cols)).astype(np.float32), dtype)
    w = dev(rng.standard_normal((tokens, 3)).astype(np.float32)) if weighted else None
    made = {}
    for names in (("y",), ("codes", "scales"), ("y", "codes", "scales"), ("codes_t", "scales_t"),
                  ("y", "codes", "scales", "codes_t", "scales_t")):
        out = dict(y=torch.full((rows, cols), 7.0, dtype=x.dtype, device="cuda"), codes=buf(rows, cols),
                   scales=buf(rows, cols // 32), codes_t=buf(cols, rows), scales_t=buf(cols, rows // 32))
        sh.moe_gather_mxfp8(x, source, offsets, tokens, 3, 8, rows, cols, dtype=dtype, weights=w, stream=stream(),
                            **{n: out[n] for n in names})
        for n in names:
            got = host(out[n]).view(np.uint32 if n == "y" else np.uint8)
            np.testing.assert_array_equal(got, made.setdefault(n, got))


@pytest.mark.parametrize("both", [False, True])
def test_gather_of_non_finite_tokens(both):
    """NaN and infinity stay in their own rows' (and columns') blocks; dropped tokens' are never read."""
    say("gather, non-finite")
    rng = np.random.default_rng(1)
    tokens, top_k, experts, cols, align = 40, 2, 3, 64, 32
    ids = choices(rng, tokens, top_k, experts, "spread")
    ids[::5] = -1
    x = _x(rng, tokens, cols, "bf16")
    x[::5] = np.nan
    x[1, 3], x[2, 40], x[3, 7] = np.nan, np.inf, -np.inf
    offsets, _, source, rows = sort(ids, tokens, top_k, experts, align)
    y = M.gather(x, None, host(source), host(offsets), top_k)
    end = int(host(offsets)[-1])
    c, s, ct, st = buf(rows, cols), buf(rows, cols // 32), buf(cols, rows), buf(cols, rows // 32)
    kw = dict(codes_t=ct, scales_t=st) if both else {}
    sh.moe_gather_mxfp8(dev(x, "bf16"), source, offsets, tokens, top_k, experts, rows, cols, codes=c, scales=s, **kw,
                        stream=stream())
    codes, scales = R.quant_rows(y)
    np.testing.assert_array_equal(host(c)[:end], codes[:end])
    np.testing.assert_array_equal(host(s)[:end], scales[:end])
    if both:
        codes, scales = R.quant_rows(y.T)
        np.testing.assert_array_equal(host(ct)[:, :end], codes[:, :end])
        np.testing.assert_array_equal(host(st)[:, :end // 32], scales[:, :end // 32])


def test_gather_reads_no_slot_that_is_not_there():
    """A source that names no slot of these tokens gives zeros, offsets past the buffers count as their end."""
    say("gather, foreign source")
    x = torch.ones(4, 32, device="cuda")
    source = torch.tensor([0, 7, 8, 1 << 30, -1, -(1 << 31), 3, 2] + [5] * 24, dtype=torch.int32, device="cuda")
    want = (source >= 0) & (source < 8)
    for end, upto in ((32, 32), (1 << 30, 32), (-5, 0), (6, 6)):
        offsets = torch.tensor([0, end], dtype=torch.int32, device="cuda")
        for t in (False, True):
            y = buf(32, 32, dtype=torch.float32, fill=9.0)
            kw = dict(codes_t=buf(32, 32), scales_t=buf(32, 1)) if t else {}
            sh.moe_gather_mxfp8(x, source, offsets, 4, 2, 1, 32, 32, dtype="fp32", y=y, **kw, stream=stream())
            got = host(y)
            assert (got[upto:] == 9.0).all()
            np.testing.assert_array_equal(got[:upto, 0], host(want)[:upto].astype(np.float32))


# ------------------------------------------------------------------------------------------------------------- combine

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,top_k,experts,cols,align", SIZES + [(9, 17, 33, 64, 1), (2, 64, 5, 32, 2)])
def test_combine_and_its_gradient(tokens, top_k, experts, cols, align, dtype):
    say(f"combine {tokens} x {top_k} of {cols} from {experts}, {dtype}")
    rng = np.random.default_rng(cols + top_k)
    ids = choices(rng, tokens, top_k, experts, "dropped")
    offsets, place, source, rows = sort(ids, tokens, top_k, experts, align)
    y = _x(rng, rows, cols, dtype)
    y[host(source) < 0] = np.nan                       # rows that no slot has are not read
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    res = _x(rng, tokens, cols, dtype)
    yd = dev(y, dtype)
    for weights, residual in ((None, None), (w, None), (None, res), (w, res)):
        out = buf(tokens, cols, dtype=yd.dtype, fill=5.0)
        wd = None if weights is None else dev(weights)
        rd = None if residual is None else dev(residual, dtype)
        sh.moe_combine(yd, place, out, tokens, top_k, rows, cols, dtype=dtype, weights=wd, residual=rd, stream=stream())
        ref, bound = M.combine(y, host(place), weights, residual, top_k, dtype)
        assert np.all(np.abs(host(out) - ref) <= bound)
        if rd is not None:                             # over the residual itself
            sh.moe_combine(yd, place, rd, tokens, top_k, rows, cols, dtype=dtype, weights=wd, residual=rd, stream=stream())
            assert torch.equal(rd, out)
    dout = _x(rng, tokens, cols + 32, dtype)
    dd, wd = dev(dout, dtype), dev(w)
    dw, dy = buf(tokens, top_k, dtype=torch.float32, fill=5.0), buf(rows, cols, dtype=yd.dtype, fill=3.0)
    c, s = buf(rows, cols), buf(rows, cols // 32)
    common = dict(dtype=dtype, ld_dout=cols + 32, stream=stream())
    sh.moe_combine_backward(dd, yd, wd, place, source, offsets, tokens, top_k, experts, rows, cols, dy=dy, codes=c,
                            scales=s, dweights=dw, **common)
    ref, bound = M.dweights(dout[:, :cols], y, host(place), top_k)
    assert np.all(np.abs(host(dw) - ref) <= bound)
    end = int(host(offsets)[-1])
    g = M.gather(dout[:, :cols], w, host(source), host(offsets), top_k)
    codes, scales = R.quant_rows(g)
    np.testing.assert_array_equal(host(c)[:end], codes[:end])
    np.testing.assert_array_equal(host(s)[:end], scales[:end])
    np.testing.assert_array_equal(host(dy)[:end], R.as_dtype(g, dtype)[:end])
    assert (host(dy)[end:] == 3.0).all() and (host(c)[end:] == 0xA5).all()
    dw2 = buf(tokens, top_k, dtype=torch.float32, fill=5.0)      # each part alone
    sh.moe_combine_backward(dd, yd, None, place, None, None, tokens, top_k, experts, rows, cols, dweights=dw2, **common)
    assert torch.equal(dw, dw2)
    if rows % 32 == 0 and rows:
        ct, st, c2, s2 = buf(cols, rows), buf(cols, rows // 32), buf(rows, cols), buf(rows, cols // 32)
        dw2.fill_(5.0)
        sh.moe_combine_backward(dd, yd, wd, place, source, offsets, tokens, top_k, experts, rows, cols, codes=c2,
                                scales=s2, codes_t=ct, scales_t=st, dweights=dw2, **common)
        codes, scales = R.quant_cols(g)
        e32 = -(-end // 32) * 32
        np.testing.assert_array_equal(host(ct)[:, :e32], codes[:, :e32])
        np.testing.assert_array_equal(host(st)[:, :e32 // 32], scales[:, :e32 // 32])
        assert torch.equal(c2, c) and torch.equal(s2, s) and torch.equal(dw, dw2)


def test_combine_of_masked_and_non_finite_rows():
    """A token without any row keeps its residual (or 0); places outside the rows add nothing; infinities follow
    their weights."""
    say("combine, masked")
    y = torch.full((4, 32), float("inf"), device="cuda")
    y[0], y[1] = 1.0, 2.0
    place = torch.tensor([[-1, -1], [0, 1], [4, 1 << 30], [-(1 << 31), 0], [2, 0], [2, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan"), 1], [1, 2], [1, float("nan")], [1, 3], [2, 1], [-1, 1]], device="cuda")
    res = torch.full((6, 32), 0.5, device="cuda")
    out = buf(6, 32, dtype=torch.float32, fill=7.0)
    sh.moe_combine(y, place, out, 6, 2, 4, 32, dtype="fp32", weights=w, residual=res, stream=stream())
    assert host(out)[:, 0].tolist() == [0.5, 5.5, 0.5, 3.5, np.inf, -np.inf]
    sh.moe_combine(y, place, out, 6, 2, 4, 32, dtype="fp32", weights=w, stream=stream())
    assert host(out)[:, 31].tolist() == [0.0, 5.0, 0.0, 3.0, np.inf, -np.inf]
    dw = buf(6, 2, dtype=torch.float32, fill=7.0)
    y[2:] = 3.0
    sh.moe_combine_backward(res, y, None, place, None, None, 6, 2, 1, 4, 32, dtype="fp32", dweights=dw, stream=stream())
    assert host(dw).tolist() == [[0, 0], [16, 32], [0, 0], [0, 16], [48, 16], [48, 0]]


def test_combine_of_no_rows():
    say("combine of nothing")
    out = buf(3, 64, dtype=torch.float32, fill=7.0)
    place = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    sh.moe_combine(None, place, out, 3, 2, 0, 64, dtype="fp32", stream=stream())
    assert not host(out).any()


def test_foreign_and_host_pointers_are_refused():
    """Memory that the runtime does not know is an ARG error, not a fault."""
    say("foreign pointers")
    cpu = torch.zeros(4096, dtype=torch.int32)
    d = torch.zeros(4096, dtype=torch.int32, device="cuda")
    for call in (lambda: sh.moe_sort(cpu, 4, 2, 4, d, d, d, 8, stream=stream()),
                 lambda: sh.moe_gather_mxfp8(d, cpu, d, 4, 2, 4, 32, 32, y=d, stream=stream()),
                 lambda: sh.moe_combine(d, cpu, d, 4, 2, 8, 32, stream=stream()),
                 lambda: sh.moe_combine_backward(d, cpu, d, d, d, d, 4, 2, 4, 8, 32, dweights=d, stream=stream())):
        with pytest.raises(sh.SshdpError) as e:
            call()
        assert e.value.name == "ARG"
