"""MXFP8 products in every way the library may run one, against exact sums on the
GPU: codes of small whole numbers under scales 1 and 2, so every partial sum is a
whole number below 2^24 and float32 output must equal the float64 product (bfloat16:
that, rounded once; a group of 8 products spans less than 2^14, so none is cut off)."""

import pytest

import mxfp8_weight_repack_amd as sh
from gemm_sizes import INSTANCES
from gpu_util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


CODES = [0x00, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0x48]     # 0 1 2 3 -1 -2 4
VALUES = [0.0, 1.0, 2.0, 3.0, -1.0, -2.0, 4.0]


class Operand:
    """A random rows x cols operand in `layout`: codes, blocks (scale bytes as a matrix), values."""

    def __init__(self, rows, cols, layout, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        pick = torch.randint(0, len(CODES), (rows, cols), generator=g, device="cuda")
        br = 32 if layout == "block32x32" else 1
        self.rows, self.cols, self.layout, self.br = rows, cols, layout, br
        self.codes = torch.tensor(CODES, dtype=torch.uint8, device="cuda")[pick]
        self.blocks = torch.randint(127, 129, (rows // br, cols // 32), generator=g, device="cuda", dtype=torch.uint8)
        scale = torch.exp2((self.blocks.double() - 127)).repeat_interleave(br, 0).repeat_interleave(32, 1)
        self.values = torch.tensor(VALUES, dtype=torch.float64, device="cuda")[pick] * scale

    def matrix(self):
        s = self.blocks
        if self.layout == "tile32x4":                  # 32 rows x 4 blocks: one word a row, rows in order
            s = s.view(self.rows // 32, 32, self.cols // 128, 4).permute(0, 2, 1, 3)
        odd = torch.empty(s.numel() + 1, dtype=torch.uint8, device="cuda")[1:]     # scales lie at any address
        return sh.mx_matrix(self.codes, odd.copy_(s.reshape(-1)), self.rows, self.cols, self.layout)


def product(a, b, op, dtype, pad=0, addend=None):
    """The product in a frame that must stay as it was; twice, with the same bits."""
    m, n = a.rows, b.cols if op == "nn" else b.rows
    A, B = a.matrix(), b.matrix()
    nb = sh.gemm_mxfp8_workspace(A, B, op=op)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    runs = []
    for _ in range(2):
        out = torch.full((m + 1, n + pad), 3.0, dtype=td, device="cuda")
        if addend is not None:
            out[:m, :n] = addend
        ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        sh.gemm_mxfp8(A, B, out, dtype, op=op, addend=None if addend is None else out, ld_out=n + pad, workspace=ws,
                      workspace_bytes=nb, stream=torch.cuda.current_stream().cuda_stream)
        assert bool((out[m] == 3.0).all()) and bool((out[:, n:] == 3.0).all())
        runs.append(out[:m, :n])
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(runs[0].contiguous().view(bits), runs[1].contiguous().view(bits))
    return runs[0]


def check(op, m, n, k, dtype, la="rowmajor", lb="rowmajor"):
    """Plain, over an addend (float32), and with NaN blocks, which spoil their own rows and columns alone."""
    lb = "block32x32" if op == "nn" else lb
    a = Operand(m, k, la, m + 3 * n + k)
    b = Operand(*((k, n) if op == "nn" else (n, k)), lb, m + 3 * n + k + 1)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    ref = a.values @ (b.values if op == "nn" else b.values.t())
    assert torch.equal(product(a, b, op, dtype, pad=3), ref.to(td))
    if dtype == "fp32":
        add = torch.randint(-50, 50, (m, n), device="cuda").float()
        assert torch.equal(product(a, b, op, dtype, pad=1, addend=add), (ref + add).float())
    a.blocks[a.blocks.shape[0] // 2, -1] = 255
    b.blocks[-1, 0] = 255
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    r = a.blocks.shape[0] // 2 * a.br
    bad[r:r + a.br] = True
    if op == "nn":
        bad[:, :32] = True
    else:
        bad[:, n - b.br:] = True
    got = product(a, b, op, dtype)
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], ref.to(td)[~bad])


@pytest.mark.parametrize("op,m,n,k", [("nt", 5896, 32, 960), ("nn", 78, 2432, 928), ("nt", 35, 40, 5824),
                                      ("nn", 5, 160, 2080)])
def test_float32_by_two_wave_groups(op, m, n, k):
    """One product over two runs of K at once, their sums joined in LDS; the last two with K split besides."""
    say(f"gemm two groups {op} {m}x{n}x{k}")
    check(op, m, n, k, "fp32")


@pytest.mark.parametrize("layout", ["rowmajor", "tile32x4", "block32x32"])
def test_an_expert_of_a_bank(layout):
    """Products read an expert's rows where G left the bank's, as from the expert quantised by itself."""
    say(f"gemm expert {layout}")
    d = dict(is_unit=False, quantize=None, cols=256, row_stride=256)
    bank = dict(d, parent=-1, offset=1024, rows=288, quantize=True)
    experts = [(0, 96), (96, 64), (160, 128)]
    nodes = [bank] + [dict(d, parent=0, offset=r * 256, rows=n) for r, n in experts]
    numel = 1024 + 288 * 256
    plan = sh.Plan(nodes, numel, layout=layout)
    s = torch.cuda.current_stream().cuda_stream
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(numel, generator=g, device="cuda")
    codes = torch.zeros(numel, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(plan.stats()["scale_bytes"], dtype=torch.uint8, device="cuda")
    sh.requant_mxfp8(plan, w, codes, scales, s)
    x = Operand(50, 256, "rowmajor", 6).matrix()
    for i, (r, n) in enumerate(experts, 1):
        own = sh.Plan([dict(bank, offset=0, rows=n)], n * 256, layout=layout)
        oc = torch.zeros(n * 256, dtype=torch.uint8, device="cuda")
        os_ = torch.zeros(own.stats()["scale_bytes"], dtype=torch.uint8, device="cuda")
        ow = w[1024 + r * 256:1024 + (r + n) * 256].clone()
        sh.requant_mxfp8(own, ow, oc, os_, s)
        outs = []
        for m in (plan.mx_matrix(i, codes, scales), own.mx_matrix(0, oc, os_)):
            assert sh.gemm_mxfp8_workspace(x, m) == 0
            outs.append(torch.full((50, n), 3.0, device="cuda"))
            sh.gemm_mxfp8(x, m, outs[-1], "fp32", stream=s)
        assert torch.equal(*outs) and bool(outs[0].abs().sum() > 0)


@pytest.mark.parametrize("name", sorted(INSTANCES))
def test_every_instance(name):
    """Each compiled kernel, K whole and split, at a ragged size, and in every scale layout that the operands may have."""
    odd, whole = INSTANCES[name]
    op, dtype = "nn" if " nn" in name else "nt", "bf16" if "bf16" in name else "fp32"
    say(f"gemm instance {name}: {odd}")
    check(op, *odd, dtype)
    m, n, k = whole
    allowed = lambda layout, rows: layout == "rowmajor" or rows % 32 == 0 and (layout != "tile32x4" or k % 128 == 0)   # noqa: E731
    pairs = [(la, "block32x32") for la in ("tile32x4", "block32x32")] if op == "nn" else \
        [("rowmajor", "tile32x4"), ("rowmajor", "block32x32"), ("tile32x4", "block32x32"), ("block32x32", "tile32x4")]
    ran = 0
    for la, lb in pairs:
        if allowed(la, m) and (op == "nn" or allowed(lb, n)):
            say(f"gemm instance {name}: {whole} {la} {lb}")
            check(op, *whole, dtype, la, lb)
            ran += 1
    assert ran >= (1 if name.startswith("rows nn") else 2)


@pytest.mark.parametrize("name", sorted(INSTANCES))
def test_scales_at_both_ends(name):
    """One operand's values near 2^125, the other's near 2^-117, and the other way round: results 2^6 times the plain
    ones, to the bit."""
    op, dtype = "nn" if " nn" in name else "nt", "bf16" if "bf16" in name else "fp32"
    m, n, k = INSTANCES[name][0]
    say(f"gemm extreme scales {name}")
    a = Operand(m, k, "rowmajor", m + n)
    b = Operand(*((k, n) if op == "nn" else (n, k)), "block32x32" if op == "nn" else "rowmajor", m + k)
    ref = (a.values @ (b.values if op == "nn" else b.values.t()) * 64).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    for up in (123, -117):
        a.blocks.add_(up)
        b.blocks.add_(6 - up)
        assert torch.equal(product(a, b, op, dtype), ref)
        a.blocks.sub_(up)
        b.blocks.sub_(6 - up)
