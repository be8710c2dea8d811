"""The gated activation where its exponential matters, in every kernel that computes it: gates far out on both sides, and
many gates whose results lie next to codes' rounding borders.  Products are exact sums, so the gates are known to the bit."""

import pytest

import mxfp8_weight_repack_amd as sh
from gate_sizes import GATE_COLUMNS, GATE_SIZES
from gpu_util import say
from test_gpu_moe_products import check_codes, offsets_of, stream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CUT = -87.336                                          # where the sigmoid leaves float32's normal range: ln 2^-126


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def digits(x, least):
    """Powers of two, `least` and up, that add up to |x|, with x's sign."""
    out, d = [], 64.0
    while d >= least:
        if abs(x) >= d:
            out.append(d if x > 0 else -d)
            x = x - out[-1]
        d /= 2
    assert x == 0
    return out


def mx(values, scale_exponents=None):
    """An operand of these values (float32, each an E4M3 one times its block's scale; scale 1 unless given)."""
    rows, k = values.shape
    e = torch.zeros(rows, k // 32, dtype=torch.int32, device="cuda") if scale_exponents is None else scale_exponents
    f = torch.exp2(e.double()).repeat_interleave(32, 1)
    codes = (values.double() / f).float().to(torch.float8_e4m3fn)
    assert torch.equal(codes.double() * f, values.double())
    return sh.mx_matrix(codes.view(torch.uint8), (e + 127).to(torch.uint8), rows, k)


def call(a, g, u, counts, n):
    rows = sum(counts)
    codes = torch.full((rows, n), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, n // 32), 0xA5, dtype=torch.uint8, device="cuda")
    gate, up = (torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sh.gemm_mxfp8_swiglu(a, g, u, codes, scales, offsets=offsets_of(counts), groups=len(counts), gate=gate, up=up,
                         stream=stream())
    return codes, scales, gate, up


def near(g):
    """The activation's error relative to itself, as sshdp.h states it."""
    return (1.25 * g.abs() + 8) * 2.0 ** -24


FAR = [-20, -30, -40, -50, -60, -70, -80, -84, -86, -86.5, -87, -87.25, -87.5, -88, -88.5, -89, -100, -(2.0 ** 20),
       20, 60, 87.25, 88.5, 100, 2.0 ** 20]


@pytest.mark.parametrize("name", GATE_SIZES)
def test_far_gates(name):
    """A gate to a block of 32 columns, so a block's scale is its own: h is as near as stated down to -87.336, and no
    further from the formula's than that value under it, where the sigmoid leaves float32's normal range."""
    say(f"{name}, far gates")
    counts, k = GATE_SIZES[name]
    n, e = GATE_COLUMNS, len(counts)
    assert n == 32 * len(FAR)
    a = torch.zeros(sum(counts), k, device="cuda")
    a[:, :32] = 1
    gv, ge, uv, ue = (torch.zeros(n, c, dtype=t, device="cuda") for c, t in
                      ((k, torch.float32), (k // 32, torch.int32), (k, torch.float32), (k // 32, torch.int32)))
    for i, x in enumerate(FAR):
        at = slice(32 * i, 32 * i + 32)
        if abs(x) > 128:
            gv[at, 0], ge[at, 0] = x, 20
        else:
            d = digits(x, 0.25)
            gv[at, :len(d)] = torch.tensor(d, device="cuda")
        ue[at, 0] = 40 if -1000 < x < -45 else 0       # h far above the smallest code
        uv[at, 0] = 2.0 ** (40 if -1000 < x < -45 else 0)
    bank = lambda t: t.repeat(e, 1)                    # noqa: E731
    codes, scales, gate, up = call(mx(a), mx(bank(gv), bank(ge)), mx(bank(uv), bank(ue)), counts, n)
    g = torch.tensor(FAR, dtype=torch.float64, device="cuda").repeat_interleave(32).expand(sum(counts), n)
    u = uv[:, 0].double().expand_as(g)
    assert torch.equal(gate, g.bfloat16()) and torch.equal(up.double(), u)
    h = g * torch.special.expit(g) * u
    under = torch.where(g < CUT, 2.0 ** -126 * g.abs() * u, 0.0)
    check_codes(codes, scales, h.contiguous(), h.abs() * near(g) * (g >= CUT) + under)


@pytest.mark.parametrize("name", GATE_SIZES)
def test_gates_of_many_sizes(name):
    """Gates -88 to -20 and ups 0.5 to 8, both from a row's part and a column's: of many values many lie next to a code's
    rounding border, and none may leave it further than stated."""
    say(f"{name}, many gates")
    counts, k = GATE_SIZES[name]
    n, e, rows = GATE_COLUMNS, len(counts), sum(counts)
    r = torch.Generator(device="cuda").manual_seed(k + rows)
    pick = lambda top, size: torch.randint(0, top, (size,), generator=r, device="cuda")   # noqa: E731
    # gate -(c + d), quarters; neighbouring columns' are alike, so few of a block's values vanish beside its largest
    c, d = 20 + torch.sort(pick(36 * 4, n)).values / 4.0, pick(31 * 4, rows) / 4.0
    a, gv, uv = torch.zeros(rows, k, device="cuda"), torch.zeros(n, k, device="cuda"), torch.zeros(n, k, device="cuda")
    a[:, :8] = 1                                       # the columns' part: c's digits times one
    gv[:, 8:16] = -1                                   # the rows' part
    for j in range(8):                                 # 32 .. 1/4
        p = 2.0 ** (5 - j)
        gv[:, j] = -p * (torch.floor(c / p) % 2)
        a[:, 8 + j] = p * (torch.floor(d / p) % 2)
    a[:, 16], a[:, 24] = 1, 1 + pick(8, rows) / 8.0
    uv[:, 16], uv[:, 24] = 0.5 + pick(8, n) / 16.0, (1 + pick(8, n) / 8.0) * 2
    g = -(c.double().unsqueeze(0) + d.double().unsqueeze(1))
    u = uv[:, 16].double().unsqueeze(0) + a[:, 24].double().unsqueeze(1) * uv[:, 24].double().unsqueeze(0)
    bank = lambda t: t.repeat(e, 1)                    # noqa: E731
    codes, scales, gate, up = call(mx(a), mx(bank(gv)), mx(bank(uv)), counts, n)
    assert torch.equal(gate, g.bfloat16()) and torch.equal(up, u.bfloat16())
    h = g * torch.special.expit(g) * u
    check_codes(codes, scales, h, h.abs() * near(g))


def gradient_with_bounds(d, g, u):
    """{output: (float64 value, bound)}: the sigmoid s to 2^-21, other roundings 2^-24 each.  dup, h: s and two products.
    dgate = d u (s f), f = 1 + g (1 - s): s, three products and f's sum relative to the result; 1 - s is off by s's own error
    and its rounding, which is by no more than s."""
    s, eps = torch.special.expit(g), 2.0 ** -24
    f = 1 + g * (1 - s)
    one = 2.0 ** -21 + 2 * eps
    return {"dgate": (d * u * s * f, (d * u * s).abs() * ((2.0 ** -21 + 4 * eps) * f.abs() +
                                                          g.abs() * (2.0 ** -21 * s + s.clamp_max(eps)))),
            "dup": (d * g * s, one * (d * g * s).abs()), "h": (g * s * u, one * (g * s * u).abs())}


def test_gradient_within_its_own_bound():
    """4 million gates of -87 to 30 in the activation's gradient: the sigmoid to 2^-21 and the products behind it, which
    codes next to a rounding border tell from a sigmoid whose error grows with the gate (dgate's, whose factors have the
    most bits)."""
    say("swiglu gradient, many gates")
    r = torch.Generator(device="cuda").manual_seed(11)
    rows, cols = 2048, 2048
    gate = (torch.rand(rows, cols, generator=r, device="cuda") * 117 - 87).bfloat16()
    up, dh = ((torch.rand(rows, cols, generator=r, device="cuda") + 0.5).bfloat16() for _ in range(2))
    # blocks of like gates along both directions, so that most values are far above their block's smallest code
    gate = torch.sort(gate.view(-1)).values.view(rows // 32, cols // 32, 32, 32).permute(0, 2, 1, 3).reshape(rows, cols).contiguous()
    out = {}
    for name in ("dgate", "dup", "h"):
        out[name] = [torch.zeros(*s, dtype=torch.uint8, device="cuda") for s in
                     ((rows, cols), (rows, cols // 32), (cols, rows), (cols, rows // 32))]
    sh.swiglu_backward_mxfp8(dh, gate, up, rows, cols, **{k: sh.mx_pair(*v) for k, v in out.items()}, stream=stream())
    d, g, u = dh.double(), gate.double(), up.double()
    ref = gradient_with_bounds(d, g, u)
    for name, (v, e) in ref.items():
        t = out[name]
        check_codes(t[0], t[1], v, e + 2.0 ** -148)
        check_codes(t[2], t[3], v.t().contiguous(), e.t().contiguous() + 2.0 ** -148)
