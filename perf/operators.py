"""Timed cases of the operators around the update step: the gradient's global norm and clipping before it, and what
reads the MXFP8 weights it leaves behind -- quantising matrices, the residual RMS norm that feeds a product, and the
MXFP8 products of a linear layer in its three directions.

`own` False computes each operator with elementary torch operations; `own` True calls the library.  Sizes follow the
workloads of this repository (blocks of d = 2048 and d = 8192, the expert bank, the flat ragged shard of 5e8 elements).
"""

import random

import torch

own = False

W_STD, G_STD = 0.02, 1e-3


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a small attention block's gradients (heads, output matrix, norm): latency of the calls before a tiny update
        dict(name="clip-block", op="clip", tensors=14, numel=262400, max_norm=0.25),
        # one GPU's ragged shard of a large model: every gradient read for the norm, read and rewritten by the clip
        dict(name="clip-shard", op="clip", tensors=180, numel=500_000_000, max_norm=1.0),
        # the output gradient of a linear layer, quantised both ways for its two backward products; ragged token count
        dict(name="quant-gradient", op="quant", rows=4093, cols=8192, dtype="bf16", along="both"),
        # a main weight's transpose, the operand of the input gradient where its own scales run along the rows
        dict(name="quant-weight", op="quant", rows=8192, cols=2048, dtype="fp32", along="cols"),
        # one new token: the norm ahead of each projection while generating
        dict(name="norm-token", op="norm", rows=1, cols=8192, dtype="bf16", residual=True, keep_y=False),
        # a training batch through the d = 8192 block's norm, normalised rows kept for the weight gradient
        dict(name="norm-batch", op="norm", rows=8191, cols=8192, dtype="bf16", residual=True, keep_y=True),
        # a short sequence in full precision
        dict(name="normgrad-few", op="norm_grad", rows=33, cols=2048, dtype="fp32", through=False),
        # the same training batch backwards, the residual stream's gradient joining in
        dict(name="normgrad-batch", op="norm_grad", rows=8191, cols=8192, dtype="bf16", through=True),
        # one new token through the packed query/key/value projection of the d = 8192 block
        dict(name="linear-token", op="linear", way="fwd", m=1, n=10240, k=8192, layout="tile32x4", out="bf16"),
        # a prompt of 8192 tokens through the d = 8192 block's gate projection
        dict(name="linear-prompt", op="linear", way="fwd", m=8192, n=28672, k=8192, layout="rowmajor", out="bf16"),
        # input gradient of the d = 2048 block's up projection, read from the forward's own 32 x 32-block codes
        dict(name="linear-dgrad", op="linear", way="dgrad", m=1999, n=8192, k=2048, layout="block32x32", out="bf16"),
        # weight gradient of the same layer on a ragged batch, added to the gradients of earlier microbatches
        dict(name="linear-wgrad", op="linear", way="wgrad", m=4093, n=8192, k=2048, layout="rowmajor", out="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["clip", "quant", "norm", "norm_grad", "linear", "linear", "linear"])
    if op == "clip":
        return dict(op=op, tensors=_log(rng, 1, 400), numel=_log(rng, 100_000, 400_000_000),
                    max_norm=rng.choice([0.01, 1.0, 100.0]))
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 16000), cols=32 * _log(rng, 1, 256), dtype=rng.choice(["bf16", "fp32"]),
                    along=rng.choice(["rows", "cols", "both"]))
    if op in ("norm", "norm_grad"):
        c = dict(op=op, rows=_log(rng, 1, 8000), cols=32 * _log(rng, 2, 256), dtype=rng.choice(["bf16", "fp32"]))
        if op == "norm":
            c.update(residual=rng.random() < 0.7, keep_y=rng.random() < 0.5)
        else:
            c.update(through=rng.random() < 0.5)
        return c
    way = rng.choice(["fwd", "fwd", "dgrad", "wgrad"])
    layout = {"fwd": rng.choice(["rowmajor", "tile32x4", "block32x32"]), "dgrad": "block32x32", "wgrad": "rowmajor"}[way]
    n, k = 32 * _log(rng, 2, 512), 32 * _log(rng, 2, 256)
    if layout == "tile32x4":
        k = max(128, k // 128 * 128)
    elif layout == "rowmajor" and way == "fwd":
        n -= rng.choice([0, 1, 16])
    return dict(op=op, way=way, m=_log(rng, 1, 8000), n=n, k=k, layout=layout,
                out="fp32" if way == "wgrad" else rng.choice(["bf16", "fp32"]))


# --------------------------------------------------------------------------------------------------------------- inputs

def _randn(seed, stream, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + stream)
    return torch.randn(*shape, generator=g, device="cuda")


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pad32(n):
    return (n + 31) // 32 * 32


def _sizes(case):
    """Ragged tensor sizes, log-uniform like the flat shard's, and their 32-aligned offsets in one root."""
    r = random.Random(case["tensors"] * 1_000_003 + case["numel"])
    w = [4000.0 ** r.random() for _ in range(case["tensors"])]
    sizes = [max(1, int(case["numel"] * x / sum(w))) for x in w]
    ends, offsets = 0, []
    for s in sizes:
        offsets.append(ends)
        ends += _pad32(s)
    return sizes, offsets, ends


def _pow2(e):
    """2^e of whole numbers -127 .. 127 as float32, from its bits: exact where a power function need not be."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x):
    """MXFP8 of x along its last dimension (a multiple of 32): E4M3FN codes and one E8M0 byte per 32 elements, the
    least power of two that brings the block's largest magnitude to 448 or below."""
    b = x.float().unflatten(-1, (-1, 32))
    frac, exp = torch.frexp(b.abs().amax(-1))
    e = torch.where(frac > 0.875, exp - 8, exp - 9)
    e = torch.where(frac == 0, -127, e.clamp(-127, 127))
    codes = (b * _pow2(-e).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _quantise_weight(w, layout):
    """A weight's codes and its scale bytes, flat, in one of the three scale layouts."""
    n, k = w.shape
    if layout == "block32x32":
        # 1 x 32 rules on rows that hold a whole 32 x 32 block give the block's scale
        amax = w.view(n // 32, 32, k // 32, 32).abs().amax((1, 3))
        _, s = _quantise(amax.reshape(-1, 1).expand(-1, 32))
        s = s.view(n // 32, k // 32)
        e = s.int().sub(127).repeat_interleave(32, 0).repeat_interleave(32, 1)
        return (w * _pow2(-e)).to(torch.float8_e4m3fn), s.reshape(-1)
    codes, s = _quantise(w)
    if layout == "tile32x4":
        s = s.view(n // 32, 32, k // 128, 4).permute(0, 2, 1, 3)
    return codes, s.reshape(-1)


def _inputs(case, seed):
    op = case["op"]
    if op == "clip":
        sizes, offsets, numel = _sizes(case)
        g = _randn(seed, 0, numel).mul_(G_STD)
        pad = torch.tensor([[o + s, o + _pad32(s)] for o, s in zip(offsets, sizes)])
        holes = torch.cat([torch.arange(a, b) for a, b in pad.tolist()])
        g[holes.cuda()] = 0
        return dict(grad=g)
    if op == "quant":
        x = _randn(seed, 0, case["rows"], case["cols"]).mul_(W_STD if case["dtype"] == "fp32" else G_STD)
        return dict(src=x.to(_dtype(case["dtype"])))
    if op in ("norm", "norm_grad"):
        t, shape = _dtype(case["dtype"]), (case["rows"], case["cols"])
        # rows of different sizes, as a residual stream has them, and a trained norm's weights
        size = torch.exp(_randn(seed, 3, case["rows"], 1))
        d = dict(weight=_randn(seed, 1, case["cols"]).mul_(0.1).add_(1.0))
        if op == "norm":
            d["x"] = (_randn(seed, 0, *shape) * size).to(t)
            if case["residual"]:
                d["residual"] = (_randn(seed, 2, *shape) * size).to(t)
            return d
        d["h"] = (_randn(seed, 0, *shape) * size).to(t)
        d["rstd"] = d["h"].double().square().mean(1).add(1e-6).rsqrt().float()
        d["dy"] = _randn(seed, 2, *shape).mul_(G_STD).to(t)
        if case["through"]:
            d["dh"] = _randn(seed, 4, *shape).mul_(G_STD).to(t)
        return d
    m, n, k = case["m"], case["n"], case["k"]
    if case["way"] == "wgrad":
        # both operands with the tokens last, a ragged token count padded with zeros to whole blocks
        a = torch.zeros(n, _pad32(m), device="cuda")
        a[:, :m] = _randn(seed, 0, n, m).mul_(G_STD)
        b = torch.zeros(k, _pad32(m), device="cuda")
        b[:, :m] = _randn(seed, 1, k, m)
        (ac, as_), (bc, bs) = _quantise(a), _quantise(b)
        return dict(a=ac, a_scales=as_.reshape(-1), b=bc, b_scales=bs.reshape(-1),
                    addend=_randn(seed, 2, n, k).mul_(G_STD))
    fwd = case["way"] == "fwd"
    ac, as_ = _quantise(_randn(seed, 0, m, k if fwd else n).mul_(1.0 if fwd else G_STD))
    bc, bs = _quantise_weight(_randn(seed, 1, n, k).mul_(W_STD), case["layout"])
    return dict(a=ac, a_scales=as_.reshape(-1), b=bc, b_scales=bs)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], op = case, case["op"]
    # output buffers that a training or serving program keeps
    if op == "clip":
        s["out"], s["stats"] = torch.zeros_like(s["grad"]), torch.zeros(2, device="cuda")
    elif op == "quant":
        r, c, rp = case["rows"], case["cols"], _pad32(case["rows"])
        u8 = dict(dtype=torch.uint8, device="cuda")
        if case["along"] != "cols":
            s["codes"], s["scales"] = torch.empty(r, c, **u8), torch.empty(r, c // 32, **u8)
        if case["along"] != "rows":
            s["codes_t"], s["scales_t"] = torch.empty(c, rp, **u8), torch.empty(c, rp // 32, **u8)
    elif op == "norm":
        r, c, x = case["rows"], case["cols"], s["x"]
        s["h"] = torch.empty_like(x) if case["residual"] else None
        s["y"] = torch.empty_like(x) if case["keep_y"] else None
        s["codes"] = torch.empty(r, c, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(r, c // 32, dtype=torch.uint8, device="cuda")
        s["rstd"] = torch.empty(r, device="cuda")
    elif op == "norm_grad":
        s["dx"], s["dweight"] = torch.empty_like(s["h"]), torch.empty(case["cols"], device="cuda")
    else:
        rows, cols = {"fwd": ("m", "n"), "dgrad": ("m", "k"), "wgrad": ("n", "k")}[case["way"]]
        s["out"] = torch.empty(case[rows], case[cols], dtype=_dtype(case["out"]), device="cuda")
    if own:
        _prepare_own(s, case)
    return s


def _prepare_own(s, case):
    """The library's plan, operand descriptions and workspace, which a program makes once."""
    import mxfp8_weight_repack_amd as sh
    s["sh"], op, need = sh, case["op"], 0
    if op == "clip":
        sizes, offsets, numel = _sizes(case)
        nodes = [dict(parent=-1, offset=o, rows=1, cols=n, row_stride=n, is_unit=True, optimizer="adamw")
                 for o, n in zip(offsets, sizes)]
        s["plan"] = sh.Plan(nodes, numel)
        need = sh.grad_workspace(s["plan"])
    elif op == "norm_grad":
        need = sh.rmsnorm_backward_workspace(case["rows"], case["cols"])
    elif op == "linear":
        s["op"] = "nn" if case["way"] == "dgrad" else "nt"
        s["A"] = sh.mx_matrix(s["a"], s["a_scales"], s["a"].shape[0], s["a"].shape[1])
        s["B"] = sh.mx_matrix(s["b"], s["b_scales"], s["b"].shape[0], s["b"].shape[1], layout=case["layout"])
        need = sh.gemm_mxfp8_workspace(s["A"], s["B"], op=s["op"])
    s["ws"], s["ws_bytes"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda"), need


# ----------------------------------------------------------------------------------------------------------- plain form

def _scale_matrix(scales, layout, rows, cols):
    """Exponents of the 1 x 32 blocks of a rows x cols matrix, whatever the layout its bytes are kept in."""
    kb = cols // 32
    if layout == "tile32x4":
        s = scales.view(rows // 32, kb // 4, 32, 4).permute(0, 2, 1, 3).reshape(rows, kb)
    elif layout == "block32x32":
        s = scales.view(rows // 32, kb).repeat_interleave(32, 0)
    else:
        s = scales.view(rows, kb)
    return s.int() - 127


def _values(codes, scales, layout="rowmajor"):
    rows, cols = codes.shape
    e = _scale_matrix(scales, layout, rows, cols)
    return (codes.float().view(rows, cols // 32, 32) * _pow2(e).unsqueeze(-1)).view(rows, cols)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "clip":
        g = s["grad"]
        norm = (g * g).sum(dtype=torch.float64).sqrt()
        coef = torch.where(norm > case["max_norm"], case["max_norm"] / norm, torch.ones_like(norm))
        return [g * coef.float(), torch.stack([norm, coef]).float()]
    if op == "quant":
        x, out = s["src"].float(), []
        if case["along"] != "cols":
            out += _as_values(*_quantise(x))
        if case["along"] != "rows":
            pad = _pad32(case["rows"]) - case["rows"]
            out += _as_values(*_quantise(torch.nn.functional.pad(x.t(), (0, pad))))
        return out
    if op == "norm":
        h = s["x"]
        if case["residual"]:
            h = (h.float() + s["residual"].float()).to(h.dtype)
        # in 64 bits, then rounded once: a code's rounding follows from the value next to its border
        hd = h.double()
        rstd = hd.square().mean(1, keepdim=True).add(1e-6).rsqrt()
        y = (hd * rstd * s["weight"].double()).float()
        out = _as_values(*_quantise(y)) + [rstd.float().view(-1)]
        return out + ([h] if case["residual"] else []) + ([y.to(h.dtype)] if case["keep_y"] else [])
    if op == "norm_grad":
        h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"].unsqueeze(1)
        xhat, wdy = h * rstd, dy * s["weight"]
        dx = (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) * rstd
        if case["through"]:
            dx = dx + s["dh"].float()
        return [dx.to(s["h"].dtype), (dy * xhat).sum(0)]
    a, b = _values(s["a"], s["a_scales"]), _values(s["b"], s["b_scales"], case["layout"])
    out = a @ (b if case["way"] == "dgrad" else b.t())
    if "addend" in s:
        out = out + s["addend"]
    return [out.to(_dtype(case["out"]))]


def _as_values(codes, scales):
    return [codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)]


# -------------------------------------------------------------------------------------------------------- library calls

def _library(s):
    case, op, sh = s["case"], s["case"]["op"], s["sh"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "clip":
        sh.grad_clip_norm(s["plan"], s["grad"], s["out"], case["max_norm"], s["stats"], s["ws"], s["ws_bytes"], stream)
        return [s["out"], s["stats"]]
    if op == "quant":
        sh.quant_mxfp8(s["src"], case["dtype"], case["rows"], case["cols"], s.get("codes"), s.get("scales"),
                       s.get("codes_t"), s.get("scales_t"), stream=stream)
        return (_as_values(s["codes"], s["scales"]) if "codes" in s else []) + \
            (_as_values(s["codes_t"], s["scales_t"]) if "codes_t" in s else [])
    if op == "norm":
        sh.rmsnorm_mxfp8(s["x"], s["weight"], case["rows"], case["cols"], dtype=case["dtype"],
                         residual=s.get("residual"), h=s["h"], y=s["y"], codes=s["codes"], scales=s["scales"],
                         rstd=s["rstd"], eps=1e-6, stream=stream)
        return _as_values(s["codes"], s["scales"]) + [s["rstd"]] + [t for t in (s["h"], s["y"]) if t is not None]
    if op == "norm_grad":
        sh.rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], case["rows"],
                            case["cols"], dtype=case["dtype"], dh=s.get("dh"), first=True, workspace=s["ws"],
                            workspace_bytes=s["ws_bytes"], stream=stream)
        return [s["dx"], s["dweight"]]
    sh.gemm_mxfp8(s["A"], s["B"], s["out"], case["out"], op=s["op"], addend=s.get("addend"), workspace=s["ws"],
                  workspace_bytes=s["ws_bytes"], stream=stream)
    return [s["out"]]


def run(s):
    return _library(s) if own else _plain(s)


# ------------------------------------------------------------------------------------------------------- work and exact

def work(case):
    op = case["op"]
    if op == "clip":
        return dict(bytes=8 * case["numel"], flops=3 * case["numel"])
    size = 2 if case.get("dtype") == "bf16" else 4
    if op == "quant":
        r, c, rp = case["rows"], case["cols"], _pad32(case["rows"])
        out = (r * c if case["along"] != "cols" else 0) + (rp * c if case["along"] != "rows" else 0)
        return dict(bytes=r * c * size + out * 33 / 32, flops=3 * out)
    if op in ("norm", "norm_grad"):
        r, c = case["rows"], case["cols"]
        if op == "norm":
            per = size * (1 + 2 * case["residual"] + case["keep_y"]) + 33 / 32
            return dict(bytes=r * c * per + 4 * (r + c), flops=6 * r * c)
        return dict(bytes=r * c * size * (3 + case["through"]) + 4 * (r + 2 * c), flops=12 * r * c)
    m, n, k = case["m"], case["n"], case["k"]
    size = 2 if case["out"] == "bf16" else 4
    inputs = {"fwd": m * k + n * k, "dgrad": m * n + n * k, "wgrad": (n + k) * _pad32(m)}[case["way"]]
    outputs = {"fwd": m * n, "dgrad": m * k, "wgrad": n * k}[case["way"]]
    return dict(bytes=inputs * 33 / 32 + outputs * size * (2 if case["way"] == "wgrad" else 1), flops=2 * m * n * k)


_E4M3 = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)]


def _mx64(x):
    """Codes' values and scales of the MX format, from the definition, in 64 bits."""
    power = torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device="cuda")
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().max(-1).values
    bounds = 448 * power[160 - 127:160 + 127]
    e = torch.searchsorted(bounds, amax.contiguous()) - 127      # the least e with amax <= 448 * 2^e
    y = b * power[160 - e].unsqueeze(-1)
    binades = power[160 - 6:160 + 10]
    at = torch.searchsorted(binades, y.abs().contiguous(), right=True).clamp_min(1) - 1
    step = power[160 - 9 + at]                                   # 2^-3 of the binade, the lowest's below it
    return [(torch.round(y / step) * step).reshape(x.shape), power[160 + e]]


def _values64(codes, scales, layout):
    rows, kb = codes.shape[0], codes.shape[1] // 32
    table = torch.tensor(_E4M3[:127] + [float("nan")] + [-v for v in _E4M3[:127]] + [float("nan")],
                         dtype=torch.float64, device="cuda")
    i, j = torch.arange(rows, device="cuda").unsqueeze(1), torch.arange(kb, device="cuda").unsqueeze(0)
    at = {"rowmajor": i * kb + j, "tile32x4": (i // 32 * (kb // 4) + j // 4) * 128 + i % 32 * 4 + j % 4,
          "block32x32": i // 32 * kb + j}[layout]
    power = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [float("nan")], dtype=torch.float64, device="cuda")
    factor = power[scales[at].int()]
    v = table[codes.view(torch.uint8).int()].reshape(rows, kb, 32)
    return v.mul_(factor.unsqueeze(2)).reshape(rows, kb * 32)


def exact(case, seed):
    s, op = _inputs(case, seed), case["op"]
    if op == "clip":
        g = s["grad"].double()
        norm = torch.dot(g, g) ** 0.5
        coef = min(1.0, case["max_norm"] / float(norm))
        return [g.mul_(coef), torch.tensor([float(norm), coef], dtype=torch.float64)]
    if op == "quant":
        x, out = s["src"], []
        if case["along"] != "cols":
            out += _mx64(x)
        if case["along"] != "rows":
            xt = torch.zeros(case["cols"], _pad32(case["rows"]), dtype=x.dtype, device="cuda")
            xt[:, :case["rows"]] = x.t()
            out += _mx64(xt)
        return out
    if op == "norm":
        t = s["x"].dtype
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        h = h.to(torch.float32).to(t).double()           # the residual stream is kept in the input's type
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + 1e-6)
        y = torch.einsum("rc,r,c->rc", h, rstd, s["weight"].double())
        out = _mx64(y.to(torch.float32)) + [rstd]         # codes are those of y in 32 bits
        return out + ([h] if case["residual"] else []) + ([y] if case["keep_y"] else [])
    if op == "norm_grad":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        dot = (h * dy * w).sum(1) * r ** 3 / case["cols"]
        dx = dy * w * r[:, None] - h * dot[:, None]
        if case["through"]:
            dx = dx + s["dh"].double()
        return [dx, (r[:, None] * h * dy).sum(0)]
    a, b = _values64(s["a"], s["a_scales"], "rowmajor"), _values64(s["b"], s["b_scales"], case["layout"])
    out = torch.mm(a, b if case["way"] == "dgrad" else b.t())
    return [out.add_(s["addend"].double()) if "addend" in s else out]
