"""Products grouped by expert with bfloat16 output, and the gated pair, take every code under every scale: elements beyond
bfloat16's range (from 2^128 on) and under its normal numbers, in each kernel, against exact sums.  Rows and columns of
ordinary elements beside them keep theirs."""

import pytest

import mxfp8_weight_repack_amd as sh
from grouped_sizes import SIZES
from gpu_util import say
from test_gpu_gemm_shapes import Operand
from test_gpu_moe_products import check_codes, offsets_of, reference, run, stream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def remake(o):
    """The operand's values from its codes and blocks."""
    f = torch.exp2(o.blocks.double() - 127).repeat_interleave(o.br, 0).repeat_interleave(32, 1)
    o.values = o.codes.view(torch.float8_e4m3fn).double() * f
    return o


def spread(o, extreme, ordinary, along_k=False):
    """Every third block row (along_k: column) under the `extreme` scale byte, the others under `ordinary`, and blocks of
    zeros under byte 0, as G makes them.  K runs along the rows, or down the columns: a sum has elements of one kind, so
    that it is exact."""
    codes, blocks, br = o.codes, o.blocks, (o.br, 32)
    if along_k:
        codes, blocks, br = codes.t(), blocks.t(), (32, o.br)
    blocks[:] = ordinary
    blocks[::3] = extreme
    if blocks.shape[0] > 1 and blocks.shape[1] > 1:
        blocks[1::3, -1] = 0
        codes[torch.arange(codes.shape[0], device="cuda") // br[0] % 3 == 1, -br[1]:] = 0
    return remake(o)


# extreme and ordinary scale byte of one operand, the other's.  In the last two the codes are the format's smallest, 1 to
# 7 times 2^-9: 2^-136 to 2^-133 of byte 0.
WAYS = [(254, 127, 100), (250, 127, 100), (0, 127, 200), (3, 127, 200)]


@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("way", WAYS, ids=str)
@pytest.mark.parametrize("name", [n for n in SIZES if "bf16" in n and "gated" not in n])
def test_products_of_elements_of_any_size(name, way, swapped):
    say(f"{name}, scale bytes {way}, {'B' if swapped else 'A'}")
    extreme, ordinary, other = way
    counts, n, k = SIZES[name]
    op = name.split()[1]
    e, p = len(counts), sum(counts)
    a = Operand(p, k, "rowmajor", 1)
    b = Operand(*((e * k, n) if op == "nn" else (e * n, k)), "block32x32" if op == "nn" else "rowmajor", 2)
    x, y = (b, a) if swapped else (a, b)
    if extreme < 10:
        g = torch.Generator(device="cuda").manual_seed(3)
        x.codes = torch.randint(0, 8, x.codes.shape, generator=g, device="cuda", dtype=torch.uint8)
    y.blocks[:] = other
    spread(x, extreme, ordinary, along_k=swapped and op == "nn")
    remake(y)
    ref = reference(a, b, counts, op)
    assert bool((ref.abs() < 2.0 ** 127).all())
    assert torch.equal(run(a, b, counts, op, "bf16"), ref.to(torch.bfloat16))


@pytest.mark.parametrize("bytes_", [(254, 0), (254, 10), (0, 254), (5, 246), (246, 5)], ids=str)
@pytest.mark.parametrize("name", [n for n in SIZES if "gated" in n])
def test_gated_pair_of_elements_of_any_size(name, bytes_):
    """One operand huge, the other tiny: gates and ups of ordinary size, in rows and columns beside zeros."""
    say(f"{name}, scale bytes {bytes_}")
    counts, n, k = SIZES[name]
    e, p = len(counts), sum(counts)
    a, g, u = Operand(p, k, "rowmajor", 1), Operand(e * n, k, "rowmajor", 2), Operand(e * n, k, "rowmajor", 3)
    a.codes[:, 3:k - 1] = 0                            # sums of a few terms
    if bytes_ == (254, 0):
        a.codes[:, 1:] = 0
    a.blocks[:], g.blocks[:], u.blocks[:] = bytes_[0], bytes_[1], bytes_[1]
    a.codes[::4], a.blocks[::4] = 0, 0                 # padding rows
    for o in (a, g, u):
        remake(o)
    gate, up = reference(a, g, counts, "nt"), reference(a, u, counts, "nt")
    assert float(gate.abs().max()) < 2.0 ** 20
    gs, us = (torch.zeros(p, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    codes, scales = (torch.zeros(p, c, dtype=torch.uint8, device="cuda") for c in (n, n // 32))
    sh.gemm_mxfp8_swiglu(a.matrix(), g.matrix(), u.matrix(), codes, scales, offsets=offsets_of(counts), groups=e, gate=gs,
                         up=us, stream=stream())
    assert torch.equal(gs, gate.bfloat16()) and torch.equal(us, up.bfloat16())
    h = gate * torch.special.expit(gate) * up
    under = torch.where(gate < -87.336, 2.0 ** -126 * gate.abs() * up.abs(), 0.0)
    check_codes(codes, scales, h, h.abs() * (1.25 * gate.abs() + 8) * 2.0 ** -24 * (gate >= -87.336) + under)


@pytest.mark.parametrize("layout", ["tile32x4", "block32x32"])
@pytest.mark.parametrize("way", [WAYS[0], WAYS[2]], ids=str)
@pytest.mark.parametrize("counts,n,k", [([3, 0, 17, 1], 96, 640), ([5, 20], 64, 4352), ([40], 32, 128)])
def test_few_rows_by_banks_in_every_layout(counts, n, k, way, layout):
    """The second pass finds a step's scales where each layout has them."""
    say(f"few rows {counts} {n} x {k} {layout}, scale bytes {way}")
    extreme, ordinary, other = way
    e = len(counts)
    a, b = Operand(sum(counts), k, "rowmajor", 1), Operand(e * n, k, layout, 2)
    for x, y in ((a, b), (b, a)):
        if extreme < 10:
            g = torch.Generator(device="cuda").manual_seed(3)
            x.codes = torch.randint(0, 8, x.codes.shape, generator=g, device="cuda", dtype=torch.uint8)
        y.blocks[:] = other
        spread(x, extreme, ordinary)
        remake(y)
        ref = reference(a, b, counts, "nt")
        assert bool((ref.abs() < 2.0 ** 127).all())
        assert torch.equal(run(a, b, counts, "nt", "bf16"), ref.to(torch.bfloat16))


@pytest.mark.parametrize("name", ["few nt bf16 4", "few nt bf16 8"])
def test_ordinary_rows_keep_their_bits(name):
    """Elements of any size in one row, or in one column's weights, change no bit of another's result."""
    say(f"{name}, neighbours")
    counts, n, k = SIZES[name]
    e, p = len(counts), sum(counts)
    r = torch.Generator(device="cuda").manual_seed(5)

    def operand(rows, seed):
        o = Operand(rows, k, "rowmajor", seed)
        o.codes = torch.randint(0, 0x7E, o.codes.shape, generator=r, device="cuda", dtype=torch.uint8)
        o.codes += 128 * torch.randint(0, 2, o.codes.shape, generator=r, device="cuda", dtype=torch.uint8)
        return o
    a, b = operand(p, 1), operand(e * n, 2)
    want = run(a, b, counts, "nt", "bf16").clone()
    row, col = p - 1, 7
    a.blocks[row, ::2], b.blocks[col::n, 1::2] = 2, 250
    got = run(a, b, counts, "nt", "bf16")
    rows = torch.arange(p, device="cuda") != row
    cols = torch.arange(n, device="cuda") != col
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])
    assert not torch.equal(got[row], want[row])
