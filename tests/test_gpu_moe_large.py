"""The expert layer's operators where elements pass 2^32: what lies there is compared to a small call on the same data,
to the bit, or to exact sums (codes of 0 and of 1 and -1 under scale 1)."""

import pytest

import mxfp8_weight_repack_amd as sh

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

COLS, MORE = 16384, 224
ROWS = (1 << 18) + MORE                                # ROWS x COLS: the last 224 rows lie past 2^32 elements


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()
    yield
    torch.cuda.empty_cache()


def stream():
    return torch.cuda.current_stream().cuda_stream


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pair(rows, cols=COLS):
    """Buffers of a matrix's codes and scales both ways."""
    return u8(rows, cols), u8(rows, cols // 32), u8(cols, rows), u8(cols, rows // 32)


def same_tail(large, small, rows):
    """The last rows of `large` and all of `small`, both ways."""
    (c, s, ct, st), (d, t, dt, tt) = large, small
    assert torch.equal(c[-rows:], d) and torch.equal(s[-rows:], t)
    assert torch.equal(ct[:, -rows:], dt) and torch.equal(st[:, -rows // 32:], tt)


@pytest.mark.parametrize("weighted", [False, True])
def test_gather(weighted):
    tokens = 1024
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(tokens, COLS, device="cuda", generator=g).bfloat16()
    w = torch.randn(tokens, 1, device="cuda", generator=g) if weighted else None
    source = (torch.arange(ROWS, device="cuda") * 37 % tokens).int()
    source[-5] = -1

    def run(src, rows):
        y, out = torch.empty(rows, COLS, dtype=torch.bfloat16, device="cuda"), pair(rows)
        sh.moe_gather_mxfp8(x, src, ints(0, rows), tokens, 1, 1, rows, COLS, weights=w, y=y, codes=out[0],
                            scales=out[1], codes_t=out[2], scales_t=out[3], stream=stream())
        return y, out

    y, large = run(source, ROWS)
    few, small = run(source[-MORE:].contiguous(), MORE)
    assert torch.equal(y[-MORE:].view(torch.int16), few.view(torch.int16))
    same_tail(large, small, MORE)


def test_combine_and_its_weights_gradient():
    tokens = 64
    y = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    y[-MORE:] = torch.randn(MORE, COLS, device="cuda").bfloat16()
    w, dout = torch.randn(tokens, 2, device="cuda"), torch.randn(tokens, COLS, device="cuda").bfloat16()
    place = torch.randint(0, MORE, (tokens, 2), device="cuda", dtype=torch.int32)

    def run(y, place, rows):
        out, dw = torch.empty_like(dout), torch.empty_like(w)
        sh.moe_combine(y, place, out, tokens, 2, rows, COLS, weights=w, stream=stream())
        sh.moe_combine_backward(dout, y, w, place, None, None, tokens, 2, 1, rows, COLS, dweights=dw, stream=stream())
        return out.view(torch.int16), dw

    for a, b in zip(run(y, place + (ROWS - MORE), ROWS), run(y[-MORE:].contiguous(), place, MORE)):
        assert torch.equal(a, b)


def test_activation_gradient():
    src = [torch.randn(MORE, COLS, device="cuda").bfloat16() for _ in range(3)]

    def run(dh, gate, up, rows):
        outs = [pair(rows) for _ in range(2)]
        sh.swiglu_backward_mxfp8(dh, gate, up, rows, COLS, dgate=sh.mx_pair(*outs[0]), h=sh.mx_pair(*outs[1]), stream=stream())
        return outs

    whole = []
    for s in src:
        t = torch.zeros(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
        t[-MORE:] = s
        whole.append(t)
    for large, small in zip(run(*whole, ROWS), run(*src, MORE)):
        same_tail(large, small, MORE)
    rows = [(u8(n, COLS), u8(n, COLS // 32)) for n in (ROWS, MORE)]
    for (dh, gate, up), (c, s) in zip((whole, src), rows):
        sh.swiglu_backward_mxfp8(None, gate, up, c.shape[0], COLS, h=sh.mx_pair(c, s), stream=stream())
    assert torch.equal(rows[0][0][-MORE:], rows[1][0]) and torch.equal(rows[0][1][-MORE:], rows[1][1])


def signs(rows, cols, where=None):
    """Codes of 0, 1 and -1 in the rows `where` (all), zeros elsewhere; their values there."""
    table = torch.tensor([0x00, 0x38, 0xB8], dtype=torch.uint8, device="cuda")
    n = rows if where is None else where
    pick = torch.randint(0, 3, (n, cols), device="cuda")
    codes = torch.zeros(rows, cols, dtype=torch.uint8, device="cuda")
    codes[-n:] = table[pick]
    return codes, torch.full((rows, cols // 32), 127, dtype=torch.uint8, device="cuda"), torch.tensor([0., 1., -1.], device="cuda")[pick]


def test_rows_of_a_long_operand():
    """A past 2^32 codes; whole numbers up to 256 are exact in bfloat16 as well, larger ones rounded once."""
    a, sa, va = signs(ROWS, COLS, MORE)
    b, sb, vb = signs(2 * 160, COLS)
    off = ints(0, ROWS - 100, ROWS)
    ref = torch.cat([va[:-100].double() @ vb[:160].double().t(), va[-100:].double() @ vb[160:].double().t()])
    for dtype, td in (("fp32", torch.float32), ("bf16", torch.bfloat16)):
        out = torch.empty(ROWS, 160, dtype=td, device="cuda")
        sh.gemm_mxfp8_grouped(sh.mx_matrix(a, sa, ROWS, COLS), sh.mx_matrix(b, sb, 2 * 160, COLS), out, off, 2,
                              out_dtype=dtype, stream=stream())
        assert torch.equal(out[-MORE:], ref.to(td)) and not bool(out[:-MORE].any())


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_rows_of_a_long_result(op):
    a, sa, va = signs(ROWS, 128)
    b, sb, vb = signs(*((2 * COLS, 128) if op == "nt" else (2 * 128, COLS)))
    if op == "nn":
        sb = torch.full((2 * 128 // 32, COLS // 32), 127, dtype=torch.uint8, device="cuda")
    B = sh.mx_matrix(b, sb, *b.shape, layout="rowmajor" if op == "nt" else "block32x32")
    off = ints(0, ROWS - 100, ROWS)
    out = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    sh.gemm_mxfp8_grouped(sh.mx_matrix(a, sa, ROWS, 128), B, out, off, 2, op=op, addend=None, stream=stream())
    w = [vb[:COLS].t(), vb[COLS:].t()] if op == "nt" else [vb[:128], vb[128:]]
    ref = torch.cat([va[-MORE:-100] @ w[0], va[-100:] @ w[1]])          # sums up to 128: exact
    assert torch.equal(out[-MORE:].float(), ref)


def test_gated_pair_of_a_long_result():
    a, sa, _ = signs(ROWS, 128)
    bg, sg, _ = signs(COLS, 128)
    bu, su, _ = signs(COLS, 128)
    m = [sh.mx_matrix(b, s, COLS, 128) for b, s in ((bg, sg), (bu, su))]

    def run(first, rows):
        c, s = u8(rows, COLS), u8(rows, COLS // 32)
        kept = [torch.empty(rows, COLS, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sh.gemm_mxfp8_swiglu(sh.mx_matrix(a[first:], sa[first:], rows, 128), *m, codes=c, scales=s, offsets=None,
                             groups=1, gate=kept[0], up=kept[1], stream=stream())
        return c, s, kept[0].view(torch.int16), kept[1].view(torch.int16)

    first = ROWS - 256 * 8                             # a call of the same tiles
    large, small = run(0, ROWS), run(first, ROWS - first)
    for x, y in zip(large[2:], small[2:]):
        assert torch.equal(x[-MORE:], y[-MORE:])
    for x, y in zip(large[:2], small[:2]):
        assert torch.equal(x[-MORE:], y[-MORE:])


def test_weight_gradients_past_two_to_the_32():
    groups, m, n, p = 40, 8192, 16384, 2560            # 5.4e9 results
    a, sa, va = signs(m, p)
    b, sb, vb = signs(n, p)
    off = torch.arange(groups + 1, device="cuda", dtype=torch.int32) * 64
    out = torch.ones(groups * m, n, device="cuda")
    sh.gemm_mxfp8_grouped(sh.mx_matrix(a, sa, m, p), sh.mx_matrix(b, sb, n, p), out, off, groups, out_dtype="fp32",
                          op="tn", addend=out, stream=stream())
    for e in (0, 31, 32, groups - 1):
        k = slice(64 * e, 64 * e + 64)
        assert torch.equal(out[e * m:(e + 1) * m], va[:, k] @ vb[:, k].t() + 1)
