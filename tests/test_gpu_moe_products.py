"""MXFP8 products grouped by expert against exact sums on the GPU: codes of small whole numbers under scales near 1, so
every partial sum is exact in float32 and float32 output must equal the float64 product (bfloat16: that, rounded once).
Experts without rows, of one row, of many tiles; rows behind the last expert; NaN blocks, which stay in their expert."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
from gpu_util import say
from grouped_sizes import SIZES
from test_gpu_gemm_shapes import Operand

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3_HALF = 2.0 ** -4                                  # half a step of a code, relative


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def stream():
    return torch.cuda.current_stream().cuda_stream


def offsets_of(counts):
    return torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def small(o, by):
    """The operand times 2^-by."""
    o.blocks -= by
    o.values *= 2.0 ** -by
    return o


def reference(a, b, counts, op):
    """float64 rows (or, op "tn", the experts' matrices one above the other)."""
    at, e, out = 0, len(counts), []
    rows_b = b.rows // e
    for i, c in enumerate(counts):
        if op == "tn":
            out.append(a.values[:, at:at + c] @ b.values[:, at:at + c].t())
        else:
            w = b.values[i * rows_b:(i + 1) * rows_b]
            out.append(a.values[at:at + c] @ (w if op == "nn" else w.t()))
        at += c
    return torch.cat(out)


def run(a, b, counts, op, dtype, pad=0, addend=None, in_place=True):
    """The product in a frame that must stay as it was; twice, with the same bits."""
    e = len(counts)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows = e * a.rows if op == "tn" else a.rows
    used = rows if op == "tn" else sum(counts)
    n = b.cols if op == "nn" else b.rows if op == "tn" else b.rows // e
    A, B, off = a.matrix(), b.matrix(), None if e == 1 and pad else offsets_of(counts)
    if off is None:
        used = rows
    runs = []
    for _ in range(2):
        out = torch.full((rows + 1, n + pad), 3.0, dtype=td, device="cuda")
        add = None
        if addend is not None:
            add = out if in_place else torch.full_like(out, 9.0)
            add[:used, :n] = addend
        sh.gemm_mxfp8_grouped(A, B, out, off, e, out_dtype=dtype, op=op, addend=add, ld_out=n + pad, stream=stream())
        assert bool((out[used:] == 3.0).all()) and bool((out[:, n:] == 3.0).all())
        runs.append(out[:used, :n])
    assert torch.equal(bits(runs[0]), bits(runs[1]))
    return runs[0]


def check(op, counts, n, k, dtype, lb="rowmajor", tail=0):
    e, p = len(counts), sum(counts) + tail
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    lb = "block32x32" if op == "nn" else lb
    a = Operand(*((n, p) if op == "tn" else (p, k)), "rowmajor", n + k + p)
    b = Operand(*((k, p) if op == "tn" else (e * k, n) if op == "nn" else (e * n, k)), "rowmajor" if op == "tn" else lb,
                n + k + p + 1)
    ref = reference(a, b, counts, op)
    off = [0] + np.cumsum(counts).tolist()
    if tail:                                           # what lies behind the last expert spoils nothing
        if op == "tn":
            a.blocks[:, off[-1] // 32:], b.blocks[:, off[-1] // 32:] = 255, 255
        else:
            a.blocks[off[-1]:] = 255
    assert torch.equal(run(a, b, counts, op, dtype, pad=0 if tail else 3), ref.to(td))
    add = torch.randint(-50, 50, ref.shape, device="cuda").to(td)
    for in_place in (True, False):
        got = run(a, b, counts, op, dtype, pad=0 if tail else 1, addend=add, in_place=in_place)
        assert torch.equal(got, (ref + add.double()).to(td))
    live = [i for i, c in enumerate(counts) if c]
    if not live:
        return
    # a NaN block of a row of A, and of an expert's B: its row, and its columns in its expert's rows
    x = live[len(live) // 2]
    bad = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    if op == "tn":
        a.blocks[n // 2, off[x] // 32] = 255
        b.blocks[0, off[x + 1] // 32 - 1] = 255
        bad[x * n + n // 2] = True
        bad[x * n:(x + 1) * n, 0] = True
    else:
        a.blocks[off[x + 1] - 1, -1] = 255
        bad[off[x + 1] - 1] = True
        per = b.blocks.shape[0] // e
        b.blocks[x * per, 0] = 255
        if op == "nn":
            bad[off[x]:off[x + 1], :32] = True
        else:
            bad[off[x]:off[x + 1], :b.br] = True
    got = run(a, b, counts, op, dtype)
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], ref.to(td)[~bad])


@pytest.mark.parametrize("name,layout", [(n, lay) for n in SIZES if " gated " not in n
                                         for lay in ("rowmajor", "tile32x4", "block32x32")
                                         if " nn " not in n or lay == "block32x32"])
def test_every_kernel_of_rows(name, layout):
    """Edges that no tile divides; in the layouts that group rows and columns, the next ones those take."""
    counts, n, k = SIZES[name]
    words = name.split()
    if layout != "rowmajor":
        n = -(-n // 32) * 32
    if layout == "tile32x4":
        k = -(-k // 128) * 128
    say(f"{name} {layout}: {counts} {n} x {k}")
    check(words[1], counts, n, k, words[2], lb=layout)


MANY = [0, 1, 0, 5, 33, 0, 0, 2] * 12 + [130]          # over 64 experts
ROWS = [
    ([37], 96, 64, 0), ([1], 32, 32, 0), ([0, 1, 0], 64, 96, 3), ([0, 0], 64, 64, 5), ([5, 0, 16, 17, 1], 96, 544, 2),
    ([128, 129, 0, 300, 127], 160, 416, 0), ([3, 200, 31], 352, 1056, 7), (MANY, 64, 160, 1), ([600, 1, 257], 288, 2080, 0),
    ([1, 2, 0, 3] * 20, 96, 4256, 0), ([7, 1, 12], 64, 8192, 0), ([9, 2], 64, 8224, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_rows_by_expert(case, op, dtype):
    counts, n, k, tail = ROWS[case]
    if op == "nn" and n * k < 4096:
        n = k = 64
    say(f"grouped {op} {len(counts)} experts, {sum(counts)} rows, {n} x {k}, {dtype}")
    check(op, counts, n, k, dtype, tail=tail)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("layout", ["tile32x4", "block32x32"])
@pytest.mark.parametrize("counts,n,k", [([1, 0, 9], 64, 640), ([150, 20, 0, 140], 96, 384), ([300], 128, 1152),
                                        ([2, 17, 1], 160, 2176), ([600, 700], 416, 1024)])
def test_banks_in_every_layout(counts, n, k, layout, dtype):
    say(f"grouped {counts} {n} x {k} {layout} {dtype}")
    check("nt", counts, n, k, dtype, lb=layout)


def test_columns_that_end_anywhere():
    """Row-major banks of experts whose rows are no multiple of anything."""
    say("grouped, odd columns")
    for counts, n in (([3, 20], 1), ([150, 40], 71), ([260], 131), ([1, 2, 1], 45)):
        for dtype in ("bf16", "fp32"):
            check("nt", counts, n, 160, dtype)


COLUMNS = [([32, 0, 64, 32], 96, 64, 0), ([128], 1, 33, 0), ([0, 0], 40, 64, 128), ([0, 160, 32, 0, 288, 32], 130, 257, 0),
           ([544, 32, 0, 64], 260, 130, 128), ([32, 1056, 64], 71, 129, 0), ([32] * 70 + [64], 33, 32, 64),
           ([96, 512, 640], 256, 384, 32), ([32], 257, 64, 96)]


@pytest.mark.parametrize("case", range(len(COLUMNS)))
def test_weight_gradients(case):
    counts, m, n, tail = COLUMNS[case]
    tail += -(sum(counts) + tail) % 128
    say(f"grouped tn {len(counts)} experts, {sum(counts)} rows, {m} x {n}")
    check("tn", counts, m, n, "fp32", tail=tail)


def test_weight_gradient_of_no_rows():
    """No sorted rows at all: the addend, or zeros."""
    say("grouped tn, nothing")
    e, m, n = 3, 40, 64
    a, b = sh.mx_matrix(None, None, m, 0), sh.mx_matrix(None, None, n, 0)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    add = torch.randn(e * m, n, device="cuda")
    out = torch.full_like(add, 3.0)
    sh.gemm_mxfp8_grouped(a, b, out, off, e, out_dtype="fp32", op="tn", addend=add, stream=stream())
    assert torch.equal(out, add)
    sh.gemm_mxfp8_grouped(a, b, out, off, e, out_dtype="fp32", op="tn", stream=stream())
    assert not bool(out.any())


# --------------------------------------------------------------------------------------------------------------- gated

def decode(codes, scales):
    """float64 values, half the distance to the next code, of MXFP8 rows."""
    v = codes.view(torch.float8_e4m3fn).double()
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return v * s, torch.clamp(v.abs() * E4M3_HALF, min=2.0 ** -10) * s


def scale_byte(amax):
    """The scale rule in float64: the least e with amax <= 448 2^e."""
    frac, ex = torch.frexp(amax)
    e = torch.where(frac > 0.875, ex - 8, ex - 9)
    return torch.where(amax == 0, 0, e.clamp(-127, 127) + 127)


def check_codes(codes, scales, h, eh):
    """Codes of values within eh of h: each block's scale is the rule's for some such value, each code off by no more
    than half a step (and eh)."""
    rows = h.shape[0]
    a, d = (t.view(rows, h.shape[1] // 32, 32) for t in (h.abs(), eh))
    lo, hi = scale_byte((a - d).clamp_min(0).amax(-1)), scale_byte((a + d).amax(-1))
    assert bool(((scales >= lo) & (scales <= hi)).all())
    v, step = decode(codes, scales)
    assert bool(((v - h).abs() <= eh + step * (1 + 2.0 ** -20)).all())


GATED = ROWS[:2] + ROWS[2:9] + [([1, 2, 0, 3] * 20, 96, 4256, 0), ([7, 1, 12], 64, 8192, 0), ([9, 2], 64, 8224, 0),
                                ([40, 1], 32, 512, 4), ([700, 300], 704, 256, 9)] + \
    [(*s, 0) for name, s in SIZES.items() if " gated " in name]


@pytest.mark.parametrize("layout", ["rowmajor", "tile32x4", "block32x32"])
@pytest.mark.parametrize("case", range(len(GATED)))
def test_gated(case, layout):
    counts, n, k, tail = GATED[case]
    if layout == "tile32x4":
        k = -(-k // 128) * 128
    say(f"gated {len(counts)} experts, {sum(counts)} rows, {n} x {k}, {layout}")
    e, used = len(counts), sum(counts)
    p = used + tail
    # gates of a few units: both sides of the activation and its tails
    a = small(Operand(p, k, "rowmajor", k + p), 3 + int(np.log2(k)) // 2)
    g, u = Operand(e * n, k, layout, k + p + 1), Operand(e * n, k, layout, k + p + 2)
    gate, up = reference(a, g, counts, "nt"), reference(a, u, counts, "nt")
    a.blocks[used:] = 255
    h = gate / (1 + torch.exp(-gate)) * up
    off = offsets_of(counts) if e > 1 or tail else None
    A, G, U = a.matrix(), g.matrix(), u.matrix()

    def call(keep, codes=True):
        s = dict(codes=torch.full((p, n), 0xA5, dtype=torch.uint8, device="cuda"),
                 scales=torch.full((p, n // 32), 0xA5, dtype=torch.uint8, device="cuda")) if codes else {}
        if keep:
            s.update(gate=torch.full((p, n), 3.0, dtype=torch.bfloat16, device="cuda"),
                     up=torch.full((p, n), 3.0, dtype=torch.bfloat16, device="cuda"))
        sh.gemm_mxfp8_swiglu(A, G, U, offsets=off, groups=e, **s, stream=stream())
        return s

    s = call(True)
    assert torch.equal(s["gate"][:used], gate.bfloat16()) and torch.equal(s["up"][:used], up.bfloat16())
    # silu's argument is exact: 1.23 |gate| + 7 halves of a step from the exponent on
    check_codes(s["codes"][:used], s["scales"][:used], h, h.abs() * (1.25 * gate.abs() + 8) * 2.0 ** -24)
    assert bool((s["gate"][used:] == 3.0).all()) and bool((s["up"][used:] == 3.0).all())
    assert bool((s["codes"][used:] == 0xA5).all()) and bool((s["scales"][used:] == 0xA5).all())
    for other in (call(False), call(True), call(True, codes=False)):
        for name, t in other.items():
            assert torch.equal(t, s[name]), name
    # a NaN block of one expert's up spoils that expert's 32 columns
    if used:
        x = max(range(e), key=lambda i: counts[i])
        u.blocks[x * u.blocks.shape[0] // e, 0] = 255
        U = u.matrix()
        t = call(True)
        rows = slice(sum(counts[:x]), sum(counts[:x + 1]))
        assert bool((t["scales"][rows, 0] == 255).all()) and bool((t["codes"][rows, :32] == 0x7F).all())
        same = torch.ones(used, n // 32, dtype=torch.bool, device="cuda")
        same[rows, 0] = False
        assert torch.equal(t["scales"][:used][same], s["scales"][:used][same])
        assert torch.equal(t["codes"][:used][same.repeat_interleave(32, 1)], s["codes"][:used][same.repeat_interleave(32, 1)])


def test_gates_far_out():
    """Gates whose exponential leaves float32's range: the activation is the gate itself, or a zero."""
    say("gated, far gates")
    k, n = 32, 64
    a = Operand(2, k, "rowmajor", 1)
    a.codes.fill_(0x38)
    a.blocks.fill_(127)                                # rows of ones
    g, u = Operand(n, k, "rowmajor", 2), Operand(n, k, "rowmajor", 3)
    g.codes.fill_(0x38)
    g.codes[1::2] = 0xB8                               # gates of +-32 * 2^e
    g.blocks[:] = 127 + torch.arange(n, device="cuda", dtype=torch.uint8).unsqueeze(1) // 2
    u.codes.fill_(0x38)
    u.blocks.fill_(122)                                # ups of one
    out = {m: torch.zeros(2, n, dtype=torch.bfloat16, device="cuda") for m in ("gate", "up")}
    codes, scales = torch.zeros(2, n, dtype=torch.uint8, device="cuda"), torch.zeros(2, 2, dtype=torch.uint8, device="cuda")
    sh.gemm_mxfp8_swiglu(a.matrix(), g.matrix(), u.matrix(), codes, scales, **out, stream=stream())
    gate = out["gate"].double()
    h = gate * torch.special.expit(gate)
    assert bool(torch.isfinite(decode(codes, scales)[0]).all())
    check_codes(codes, scales, h, h.abs() * (1.25 * gate.abs() + 8) * 2.0 ** -24 + 2.0 ** -118)


# ------------------------------------------------------------------------------------------------------------ limits

def test_offsets_outside_the_rows_stay_inside_the_buffers():
    """Offsets that leave the rows, run backwards or are no multiples write a part of out and nothing else."""
    say("grouped, wild offsets")
    a, b = Operand(200, 64, "rowmajor", 1), Operand(4 * 64, 64, "block32x32", 2)
    at, bt = Operand(64, 256, "rowmajor", 3), Operand(32, 256, "rowmajor", 4)
    codes, scales = torch.zeros(200, 64, dtype=torch.uint8, device="cuda"), torch.zeros(200, 2, dtype=torch.uint8, device="cuda")
    for wild in ([-5, 100, 50, 1 << 30, 7], [1 << 30, -(1 << 31), 3, 200, 201], [0, 13, 77, 199, 200], [250, 255, 260, 5, 1]):
        off = torch.tensor(wild, dtype=torch.int32, device="cuda")
        for op in ("nt", "nn"):
            for dtype in (torch.bfloat16, torch.float32):
                out = torch.full((201, 64), 3.0, dtype=dtype, device="cuda")
                sh.gemm_mxfp8_grouped(a.matrix(), b.matrix(), out, off, 4, op=op,
                                      out_dtype="bf16" if dtype == torch.bfloat16 else "fp32", stream=stream())
                assert bool((out[200] == 3.0).all())
        sh.gemm_mxfp8_swiglu(a.matrix(), b.matrix(), b.matrix(), codes, scales, offsets=off, groups=4, stream=stream())
        out = torch.full((4 * 64 + 1, 32), 3.0, device="cuda")
        sh.gemm_mxfp8_grouped(at.matrix(), bt.matrix(), out, off, 4, out_dtype="fp32", op="tn", stream=stream())
        assert bool((out[-1] == 3.0).all())
    torch.cuda.synchronize()
