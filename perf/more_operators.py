"""Timed cases of a mixture-of-experts layer on the library's MXFP8 expert banks: tokens sorted by expert, gathered
into the experts' rows and combined back, the experts' products in their directions, and the gated activation's
gradient.

`own` False computes each operator with elementary torch operations; `own` True calls the library.  Sizes follow this
repository's expert bank (64 experts, d = 2048, width 1408), with generic numbers of tokens and choices.
"""

import torch

own = False

W_STD, G_STD = 0.02, 1e-3


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # sixteen sequences generating: the few slots of one decoding step
        dict(name="sort-tokens", op="sort", tokens=16, top_k=6, experts=64, align=1, padding=0),
        # a training batch whose last tokens are padding, experts' rows aligned for the weight gradient
        dict(name="sort-batch", op="sort", tokens=16381, top_k=6, experts=64, align=32, padding=301),
        # a prompt's tokens on their way to the experts, operands of the forward products alone
        dict(name="gather-prompt", op="gather", tokens=1021, top_k=6, experts=64, align=1, padding=0, cols=2048,
             dtype="bf16", both=False),
        # a training batch, quantised along the tokens too for the weight gradients
        dict(name="gather-batch", op="gather", tokens=4093, top_k=6, experts=64, align=32, padding=61, cols=2048,
             dtype="bf16", both=True),
        # the experts' results back to a batch's residual stream
        dict(name="combine-batch", op="combine", tokens=8191, top_k=6, experts=64, align=32, padding=0, cols=2048,
             dtype="bf16", residual=True),
        # its gradient: the experts' output gradients as product operands, and the router's weights' gradient
        dict(name="combine-grad", op="combine_grad", tokens=4093, top_k=6, experts=64, align=32, padding=61, cols=2048,
             dtype="bf16", both=True),
        # one decoding step of sixteen sequences through gate, up and activation
        dict(name="experts-tokens", op="product", way="gated", tokens=16, top_k=6, experts=64, align=1, n=1408, k=2048,
             layout="tile32x4", keep=False),
        # a training batch through them, gate and up kept for the backward pass
        dict(name="experts-batch", op="product", way="gated", tokens=4093, top_k=6, experts=64, align=32, n=1408,
             k=2048, layout="block32x32", keep=True),
        # the input gradient of the down projection, from the forward's own codes
        dict(name="experts-dgrad", op="product", way="dgrad", tokens=4093, top_k=6, experts=64, align=32, n=2048,
             k=1408, layout="block32x32", addend=False),
        # the weight gradient of the gate projection, added to the gradients of earlier microbatches
        dict(name="experts-wgrad", op="product", way="wgrad", tokens=4093, top_k=6, experts=64, align=32, n=1408,
             k=2048),
        # the activation's gradient of a short batch
        dict(name="actgrad-few", op="act_grad", tokens=129, top_k=2, experts=16, align=32, cols=704),
        # and of a training batch
        dict(name="actgrad-batch", op="act_grad", tokens=4093, top_k=6, experts=64, align=32, cols=1408),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["sort", "gather", "combine", "combine_grad", "product", "product", "product", "act_grad"])
    e = _log(rng, 4, 64)
    k = rng.randint(1, min(8, e))
    t = _log(rng, 1, {"sort": 12000, "combine": 6000}.get(op, 4093) * 6 // max(k, 6))
    c = dict(op=op, tokens=t, top_k=k, experts=e, align=rng.choice([1, 32]))
    if op not in ("product", "act_grad"):
        c["padding"] = rng.choice([0, 0, t // 5])
    if op in ("gather", "combine", "combine_grad"):
        c.update(cols=32 * _log(rng, 2, 64), dtype=rng.choice(["bf16", "bf16", "fp32"]))
        if op == "combine":
            c["residual"] = rng.random() < 0.5
        else:
            c["both"] = c["align"] == 32 and rng.random() < 0.6
    elif op == "product":
        way = rng.choice(["gated", "gated", "forward", "forward", "dgrad", "wgrad"])
        n, kk = 32 * _log(rng, 4, 64), 32 * _log(rng, 4, 64)
        n = min(n, 32 * (1408 * 2048 // (32 * kk)))
        c.update(way=way, n=n, k=kk)
        if way == "wgrad":
            c["align"] = 32
        else:
            c["layout"] = "block32x32" if way == "dgrad" else rng.choice(["rowmajor", "tile32x4", "block32x32"])
            if c["layout"] == "tile32x4":
                c["k"] = max(128, kk // 128 * 128)
            if way == "gated":
                c["keep"] = rng.random() < 0.5
            else:
                c["addend"] = rng.random() < 0.5
    elif op == "act_grad":
        c.update(align=32, cols=32 * _log(rng, 4, 44))
    return c


# --------------------------------------------------------------------------------------------------------------- inputs

def _randn(seed, stream, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + stream)
    return torch.randn(*shape, generator=g, device="cuda")


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rows(case):
    """Rows of the sorted buffers: every slot, and each expert's rows brought up to `align`, in whole tiles of 128."""
    slots = case["tokens"] * case["top_k"]
    if case["align"] == 1:
        return slots
    return (slots + min(slots, case["experts"]) * (case["align"] - 1) + 127) // 128 * 128


def _route(case, seed):
    """Choices of a router whose experts are not equally liked, their softmax weights, padding tokens' choices -1."""
    logits = _randn(seed, 0, case["tokens"], case["experts"]) + 0.7 * _randn(seed, 1, case["experts"])
    v, ids = torch.topk(logits, case["top_k"], dim=1)
    if case.get("padding"):
        ids[-case["padding"]:] = -1
    return ids, torch.softmax(v, 1)


def _sort(ids, experts, align, rows):
    """offsets (experts + 1), place of each slot, slot of each row."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    counts = (key.unsqueeze(1) == torch.arange(experts + 1, device="cuda")).sum(0)
    first = torch.cumsum(counts, 0) - counts                       # of each expert among the sorted slots
    padded = (counts[:experts] + align - 1) // align * align
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(padded, 0)
    order = torch.sort(key, stable=True).indices
    ks = key[order]
    at = offsets[ks] + torch.arange(flat.numel(), device="cuda") - first[ks]
    dropped = ks == experts
    place = torch.empty_like(flat)
    place[order] = torch.where(dropped, -1, at)
    source = torch.full((rows + 1,), -1, dtype=torch.int64, device="cuda")
    source[torch.where(dropped, rows, at)] = torch.where(dropped, -1, order)
    return offsets.int(), place.int(), source[:rows].int()


def _pow2(e):
    """2^e of whole numbers -127 .. 127 as float32, from its bits."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x):
    """MXFP8 of x along its last dimension: E4M3FN codes and one E8M0 byte per 32 elements, the least power of two
    that brings the block's largest magnitude to 448 or below."""
    b = x.float().unflatten(-1, (-1, 32))
    frac, exp = torch.frexp(b.abs().amax(-1))
    e = torch.where(frac > 0.875, exp - 8, exp - 9)
    e = torch.where(frac == 0, -127, e.clamp(-127, 127))
    codes = (b * _pow2(-e).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return codes, (e + 127).to(torch.uint8)


def _quantise_bank(w, layout):
    """A bank's codes (experts n x k) and its scale bytes, flat, in one of the three scale layouts."""
    n, k = w.shape
    if layout == "block32x32":
        amax = w.view(n // 32, 32, k // 32, 32).abs().amax((1, 3))
        _, s = _quantise(amax.reshape(-1, 1).expand(-1, 32))
        s = s.view(n // 32, k // 32)
        e = s.int().sub(127).repeat_interleave(32, 0).repeat_interleave(32, 1)
        return (w * _pow2(-e)).to(torch.float8_e4m3fn), s.reshape(-1)
    codes, s = _quantise(w)
    if layout == "tile32x4":
        s = s.view(n // 32, 32, k // 128, 4).permute(0, 2, 1, 3)
    return codes, s.reshape(-1)


def _sizes(case):
    """Columns of A (what a product sums over), rows and columns of one expert's B, columns of the output."""
    n, k = case["n"], case["k"]
    return (n, (n, k), k) if case["way"] == "dgrad" else (k, (n, k), n)


def _inputs(case, seed):
    op, rows = case["op"], _rows(case)
    ids, weights = _route(case, seed)
    if op == "sort":
        return dict(ids=ids)
    offsets, place, source = _sort(ids, case["experts"], case["align"], rows)
    s = dict(offsets=offsets)
    if op in ("gather", "combine", "combine_grad"):
        t, c = _dtype(case["dtype"]), case["cols"]
        s.update(place=place, source=source)
        if op != "gather":
            s.update(weights=weights, y=_randn(seed, 3, rows, c).to(t))
        if op == "combine":
            if case["residual"]:
                s["residual"] = _randn(seed, 4, case["tokens"], c).to(t)
        else:
            # tokens of different sizes, as a normalised stream times its weights has them
            x = _randn(seed, 2, case["tokens"], c) * torch.exp(0.3 * _randn(seed, 4, case["tokens"], 1))
            s["x"] = (x * (G_STD if op == "combine_grad" else 1.0)).to(t)
        return s
    used = (source >= 0).unsqueeze(1)
    if op == "act_grad":
        c = case["cols"]
        s["dh"] = (_randn(seed, 2, rows, c) * used).mul_(G_STD).bfloat16()
        s["gate"] = (_randn(seed, 3, rows, c) * used).mul_(1.5).bfloat16()
        s["up"] = (_randn(seed, 4, rows, c) * used).bfloat16()
        return s
    e, n, k, way = case["experts"], case["n"], case["k"], case["way"]
    if way == "wgrad":
        a, a_scales = _quantise((_randn(seed, 2, rows, n) * used).mul_(G_STD).t().contiguous())
        b, b_scales = _quantise((_randn(seed, 3, rows, k) * used).t().contiguous())
        return dict(s, a=a, a_scales=a_scales.reshape(-1), b=b, b_scales=b_scales.reshape(-1),
                    addend=_randn(seed, 4, e * n, k).mul_(G_STD))
    ka, _, nout = _sizes(case)
    a, a_scales = _quantise((_randn(seed, 2, rows, ka) * used).mul_(G_STD if way == "dgrad" else 1.0))
    s.update(a=a, a_scales=a_scales.reshape(-1))
    for j, name in enumerate(("b", "b2") if way == "gated" else ("b",)):
        s[name], s[name + "_scales"] = _quantise_bank(_randn(seed, 5 + j, e * n, k).mul_(W_STD), case["layout"])
    if case.get("addend"):
        s["addend"] = _randn(seed, 4, rows, nout).mul_(G_STD if way == "dgrad" else 1.0).bfloat16()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], op, rows = case, case["op"], _rows(case)
    if op not in ("sort", "gather", "combine", "combine_grad"):
        # what a program knows of a batch it has sized its buffers by: the most rows an expert has here
        s["most"] = int(torch.diff(s["offsets"]).max())
    u8 = dict(dtype=torch.uint8, device="cuda")

    # output buffers that a training or serving program keeps, rows behind the last expert's zero
    def pair(name, r, c, both):
        s[name + "codes"], s[name + "scales"] = torch.zeros(r, c, **u8), torch.zeros(r, c // 32, **u8)
        if both:
            s[name + "codes_t"], s[name + "scales_t"] = torch.zeros(c, r, **u8), torch.zeros(c, r // 32, **u8)

    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "sort":
        s["offsets"], s["source"] = torch.zeros(case["experts"] + 1, **i32), torch.zeros(rows, **i32)
        s["place"] = torch.zeros(case["tokens"] * case["top_k"], **i32)
    elif op in ("gather", "combine_grad"):
        pair("", rows, case["cols"], case["both"])
        s["dweights"] = torch.zeros(case["tokens"], case["top_k"], device="cuda")
    elif op == "combine":
        s["out"] = torch.zeros(case["tokens"], case["cols"], dtype=_dtype(case["dtype"]), device="cuda")
    elif op == "act_grad":
        pair("gate_", rows, case["cols"], True)
        pair("up_", rows, case["cols"], True)
        s["h_codes_t"], s["h_scales_t"] = torch.zeros(case["cols"], rows, **u8), torch.zeros(case["cols"], rows // 32, **u8)
    elif case["way"] == "wgrad":
        s["out"] = torch.zeros(case["experts"] * case["n"], case["k"], device="cuda")
    elif case["way"] == "gated":
        pair("", rows, case["n"], False)
        if case["keep"]:
            s["gate"], s["up"] = (torch.zeros(rows, case["n"], dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        s["out"] = torch.zeros(rows, _sizes(case)[2], dtype=torch.bfloat16, device="cuda")
    if own:
        _prepare_own(s, case)
    return s


def _prepare_own(s, case):
    """The library's operand descriptions and workspace, which a program makes once."""
    import mxfp8_weight_repack_amd as sh
    s["sh"], op, need = sh, case["op"], 0
    if op == "sort":
        need = sh.moe_sort_workspace(case["tokens"], case["top_k"], case["experts"])
    elif op == "product":
        layout = case.get("layout", "rowmajor")
        s["A"] = sh.mx_matrix(s["a"], s["a_scales"], s["a"].shape[0], s["a"].shape[1])
        s["B"] = sh.mx_matrix(s["b"], s["b_scales"], s["b"].shape[0], s["b"].shape[1], layout=layout)
        if case["way"] == "gated":
            s["B2"] = sh.mx_matrix(s["b2"], s["b2_scales"], s["b2"].shape[0], s["b2"].shape[1], layout=layout)
    s["ws"], s["ws_bytes"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda"), need


# ----------------------------------------------------------------------------------------------------------- plain form

def _values(codes, scales, layout="rowmajor"):
    """An MXFP8 matrix's float32 values, whatever the layout its scale bytes are kept in."""
    rows, cols = codes.shape
    kb = cols // 32
    if layout == "tile32x4":
        e = scales.view(rows // 32, kb // 4, 32, 4).permute(0, 2, 1, 3).reshape(rows, kb)
    elif layout == "block32x32":
        e = scales.view(rows // 32, kb).repeat_interleave(32, 0)
    else:
        e = scales.view(rows, kb)
    return (codes.float().view(rows, kb, 32) * _pow2(e.int() - 127).unsqueeze(-1)).view(rows, cols)


def _as_values(codes, scales):
    return [codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)]


def _both(x, rows=True, cols=True):
    return (_as_values(*_quantise(x)) if rows else []) + (_as_values(*_quantise(x.t().contiguous())) if cols else [])


def _members(offsets, most, rows):
    """experts x most: each expert's rows, and whether it has that many."""
    at = offsets[:-1].long().unsqueeze(1) + torch.arange(most, device="cuda")
    return at.clamp_max(max(rows - 1, 0)), at < offsets[1:].unsqueeze(1)


def _ungroup(x, at, have, rows):
    """experts x most x columns back to rows x columns, zeros where no expert has the row."""
    out = torch.zeros(rows + 1, x.shape[2], device="cuda")
    out[torch.where(have, at, rows).reshape(-1)] = x.reshape(-1, x.shape[2])
    return out[:rows]


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    rows = _rows(case)
    if op == "sort":
        return list(_sort(s["ids"], case["experts"], case["align"], rows))
    if op in ("gather", "combine_grad"):
        slot = s["source"].long()
        w = (slot >= 0).float()
        if op == "combine_grad":
            w = w * s["weights"].reshape(-1)[slot.clamp_min(0)]
        y = s["x"].float()[slot.clamp_min(0) // case["top_k"]] * w.unsqueeze(1)
        out = _both(y, True, case["both"])
        if op == "combine_grad":
            place = s["place"].long().view(case["tokens"], -1)
            rows_y = s["y"].float()[place.clamp_min(0)] * (place >= 0).unsqueeze(2)
            out.append((rows_y * s["x"].float().unsqueeze(1)).sum(2))
        return out
    if op == "combine":
        place = s["place"].long().view(case["tokens"], -1)
        w = s["weights"] * (place >= 0)
        out = (s["y"].float()[place.clamp_min(0)] * w.unsqueeze(2)).sum(1)
        if case["residual"]:
            out = out + s["residual"].float()
        return [out.to(s["y"].dtype)]
    if op == "act_grad":
        d, g, u = s["dh"].float(), s["gate"].float(), s["up"].float()
        sig = 1 / (1 + torch.exp(-g))
        return _both(d * u * sig * (1 + g * (1 - sig))) + _both(d * g * sig) + _both(g * sig * u, rows=False)
    e, n, k, way = case["experts"], case["n"], case["k"], case["way"]
    a = _values(s["a"], s["a_scales"])
    at, have = _members(s["offsets"], s["most"], rows)
    if way == "wgrad":
        b = _values(s["b"], s["b_scales"])
        ag = (a[:, at] * have).transpose(0, 1).contiguous()                    # experts x n x most
        bg = (b[:, at] * have).permute(1, 2, 0).contiguous()                   # experts x most x k
        return [torch.bmm(ag, bg).view(e * n, k) + s["addend"]]
    ag = a[at] * have.unsqueeze(2)
    banks = [_values(s[name], s[name + "_scales"], case["layout"]).view(e, n, k)
             for name in (("b", "b2") if way == "gated" else ("b",))]
    out = [_ungroup(torch.bmm(ag, w if way == "dgrad" else w.transpose(1, 2).contiguous()), at, have, rows) for w in banks]
    if way == "gated":
        gate, up = out
        h = gate * (1 / (1 + torch.exp(-gate))) * up
        return _as_values(*_quantise(h)) + ([gate.bfloat16(), up.bfloat16()] if case["keep"] else [])
    if "addend" in s:
        inside = torch.arange(rows, device="cuda") < s["offsets"][-1]
        return [(out[0] + s["addend"].float() * inside.unsqueeze(1)).bfloat16()]
    return [out[0].bfloat16()]


# -------------------------------------------------------------------------------------------------------- library calls

def _library(s):
    case, op, sh = s["case"], s["case"]["op"], s["sh"]
    stream = torch.cuda.current_stream().cuda_stream
    t, k, e, rows = case["tokens"], case["top_k"], case["experts"], _rows(case)
    if op == "sort":
        sh.moe_sort(s["ids"], t, k, e, s["offsets"], s["place"], s["source"], rows, align=case["align"],
                    ids_dtype="int64", workspace=s["ws"], workspace_bytes=s["ws_bytes"], stream=stream)
        return [s["offsets"], s["place"], s["source"]]
    if op == "gather":
        sh.moe_gather_mxfp8(s["x"], s["source"], s["offsets"], t, k, e, rows, case["cols"], dtype=case["dtype"],
                            codes=s["codes"], scales=s["scales"], codes_t=s.get("codes_t"),
                            scales_t=s.get("scales_t"), stream=stream)
        return _pairs(s, "", case["both"])
    if op == "combine":
        sh.moe_combine(s["y"], s["place"], s["out"], t, k, rows, case["cols"], dtype=case["dtype"],
                       weights=s["weights"], residual=s.get("residual"), stream=stream)
        return [s["out"]]
    if op == "combine_grad":
        sh.moe_combine_backward(s["x"], s["y"], s["weights"], s["place"], s["source"], s["offsets"], t, k, e, rows,
                                case["cols"], dtype=case["dtype"], codes=s["codes"], scales=s["scales"],
                                codes_t=s.get("codes_t"), scales_t=s.get("scales_t"), dweights=s["dweights"],
                                stream=stream)
        return _pairs(s, "", case["both"]) + [s["dweights"]]
    if op == "act_grad":
        sh.swiglu_backward_mxfp8(s["dh"], s["gate"], s["up"], rows, case["cols"], offsets=s["offsets"], groups=e,
                                 dgate=sh.mx_pair(*(s["gate_" + n] for n in _NAMES)),
                                 dup=sh.mx_pair(*(s["up_" + n] for n in _NAMES)),
                                 h=sh.mx_pair(None, None, s["h_codes_t"], s["h_scales_t"]), stream=stream)
        return _pairs(s, "gate_", True) + _pairs(s, "up_", True) + _as_values(s["h_codes_t"], s["h_scales_t"])
    if case["way"] == "gated":
        sh.gemm_mxfp8_swiglu(s["A"], s["B"], s["B2"], s["codes"], s["scales"], offsets=s["offsets"], groups=e,
                             gate=s.get("gate"), up=s.get("up"), stream=stream)
        return _pairs(s, "", False) + ([s["gate"], s["up"]] if case["keep"] else [])
    op = {"forward": "nt", "dgrad": "nn", "wgrad": "tn"}[case["way"]]
    sh.gemm_mxfp8_grouped(s["A"], s["B"], s["out"], s["offsets"], e, out_dtype="fp32" if op == "tn" else "bf16", op=op,
                          addend=s.get("addend"), stream=stream)
    return [s["out"]]


_NAMES = ("codes", "scales", "codes_t", "scales_t")


def _pairs(s, name, both):
    return _as_values(s[name + "codes"], s[name + "scales"]) + \
        (_as_values(s[name + "codes_t"], s[name + "scales_t"]) if both else [])


def run(s):
    return _library(s) if own else _plain(s)


# ------------------------------------------------------------------------------------------------------- work and exact

def work(case):
    op, t, slots, e = case["op"], case["tokens"], case["tokens"] * case["top_k"], case["experts"]
    rows = _rows(case)
    if op == "sort":
        return dict(bytes=8 * slots + 4 * (slots + rows + e + 1), flops=0)
    size = 2 if case.get("dtype", "bf16") == "bf16" else 4
    live = (t - case.get("padding", 0)) * case["top_k"]                  # slots that reach an expert
    c = case.get("cols")
    if op == "combine":
        return dict(bytes=c * size * (live + t * (1 + case["residual"])) + 8 * slots, flops=2 * live * c)
    if op in ("gather", "combine_grad"):
        out = live * c * 33 / 32 * (1 + case["both"])
        per = 3 * (1 + case["both"])
        if op == "gather":
            return dict(bytes=t * c * size + out + 4 * rows, flops=per * live * c)
        return dict(bytes=(t + live) * c * size + out + 4 * rows + 12 * slots, flops=(per + 3) * live * c)
    if op == "act_grad":
        return dict(bytes=slots * c * (3 * 2 + 5 * 33 / 32), flops=30 * slots * c)
    n, k, way = case["n"], case["k"], case["way"]
    flops = 2 * slots * n * k * (2 if way == "gated" else 1)
    if way == "wgrad":
        return dict(bytes=slots * (n + k) * 33 / 32 + 8 * e * n * k, flops=flops)
    banks = 2 if way == "gated" else 1
    used = e * (1 - (1 - case["top_k"] / e) ** t)                        # experts that some token chose
    ka, _, nout = _sizes(case)
    out = nout * (33 / 32 + 4 * case["keep"]) if way == "gated" else nout * 2 * (1 + case["addend"])
    return dict(bytes=used * n * k * banks * 33 / 32 + slots * (ka * 33 / 32 + out), flops=flops)


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
    """Values of an MXFP8 matrix in 64 bits: the format's bits taken apart."""
    rows, kb = codes.shape[0], codes.shape[1] // 32
    c = codes.view(torch.uint8).int()
    mant, ex = c & 7, c >> 3 & 15
    table = torch.tensor([2.0 ** (max(i, 1) - 10) for i in range(16)], dtype=torch.float64, device="cuda")
    v = torch.where(ex > 0, mant + 8, mant).double() * table[ex] * torch.where(c > 127, -1.0, 1.0)
    i, j = torch.arange(rows, device="cuda").unsqueeze(1), torch.arange(kb, device="cuda").unsqueeze(0)
    at = {"rowmajor": i * kb + j, "tile32x4": (i // 32 * (kb // 4) + j // 4) * 128 + i % 32 * 4 + j % 4,
          "block32x32": i // 32 * kb + j}[layout]
    power = torch.tensor([2.0 ** (i - 127) for i in range(255)], dtype=torch.float64, device="cuda")
    return v.reshape(rows, kb, 32).mul_(power[scales[at].int()].unsqueeze(2)).reshape(rows, kb * 32)


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    s, rows, top_k = _inputs(case, seed), _rows(case), case["top_k"]
    if op == "combine":
        out = s["residual"].double() if case["residual"] else torch.zeros(case["tokens"], case["cols"], device="cuda",
                                                                          dtype=torch.float64)
        for j in range(top_k):
            at = s["place"].view(-1, top_k)[:, j].long()
            some = at >= 0
            out[some] += s["weights"][some, j].double().unsqueeze(1) * s["y"][at[some]].double()
        return [out]
    if op in ("gather", "combine_grad"):
        live = torch.nonzero(s["source"] >= 0).view(-1)
        slot = s["source"][live].long()
        y = torch.zeros(rows, case["cols"], dtype=torch.float64, device="cuda")
        y[live] = s["x"].double()[torch.div(slot, top_k, rounding_mode="floor")]
        if op == "combine_grad":
            y[live] *= s["weights"].double().view(-1)[slot].unsqueeze(1)
        out = _mx64(y.to(torch.float32)) + (_mx64(y.to(torch.float32).t()) if case["both"] else [])
        if op == "combine_grad":
            dw = torch.zeros(case["tokens"] * top_k, dtype=torch.float64, device="cuda")
            dw[slot] = torch.einsum("rc,rc->r", s["x"].double()[torch.div(slot, top_k, rounding_mode="floor")],
                                    s["y"][live].double())
            out.append(dw.view(-1, top_k))
        return out
    if op == "act_grad":
        d, g, u = s["dh"].double(), s["gate"].double(), s["up"].double()
        sig = torch.sigmoid(g)
        du = d * torch.nn.functional.silu(g)
        dg = d * u * (sig + g * torch.exp(-g) * sig * sig)
        h = torch.nn.functional.silu(g) * u
        return _mx64(dg) + _mx64(dg.t()) + _mx64(du) + _mx64(du.t()) + _mx64(h.t())
    n, k, way = case["n"], case["k"], case["way"]
    ends = s["offsets"].tolist()
    a = _values64(s["a"], s["a_scales"], "rowmajor")
    if way == "wgrad":
        b = _values64(s["b"], s["b_scales"], "rowmajor")
        out = s["addend"].double()
        for i in range(case["experts"]):
            at = slice(ends[i], ends[i + 1])
            out[i * n:(i + 1) * n] += torch.mm(a[:, at], b[:, at].t())
        return [out]
    out = []
    for name in ("b", "b2") if way == "gated" else ("b",):
        b = _values64(s[name], s[name + "_scales"], case["layout"]).view(-1, n, k)
        o = torch.zeros(rows, _sizes(case)[2], dtype=torch.float64, device="cuda")
        for i in range(case["experts"]):
            at = slice(ends[i], ends[i + 1])
            o[at] = torch.mm(a[at], b[i] if way == "dgrad" else b[i].t())
        out.append(o)
    if way == "gated":
        gate, up = out
        return _mx64(torch.nn.functional.silu(gate) * up) + ([gate, up] if case["keep"] else [])
    if "addend" in s:
        out[0][:ends[-1]] += s["addend"].double()[:ends[-1]]
    return out
