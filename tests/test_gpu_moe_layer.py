"""An expert layer as it is used, forwards and backwards on a plan's banks: each stage against float64 of what it was
given; captured into a graph and replayed on new tokens; two of them on two streams at once; and a training step's
gradients taken up by the update."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import moe_ref as M
import ops_ref as R
from gpu_util import say
from test_gpu_moe_products import check_codes, decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


class Layer:
    """One layer's weights and the buffers that a program keeps for it.  The roots hold gate, up and down banks."""

    def __init__(self, tokens, top_k, experts, d, f, seed):
        self.t, self.k, self.e, self.d, self.f = tokens, top_k, experts, d, f
        g = torch.Generator(device="cuda").manual_seed(seed)
        nodes, at = [], 0
        for rows, cols in ((f, d), (f, d), (d, f)):
            nodes.append(dict(parent=-1, offset=at, rows=experts * rows, cols=cols, row_stride=cols, is_unit=False,
                              optimizer=None, quantize=True))
            bank = len(nodes) - 1
            nodes += [dict(parent=bank, offset=i * rows * cols, rows=rows, cols=cols, row_stride=cols, is_unit=True,
                           optimizer="muon") for i in range(experts)]
            at += experts * rows * cols
        self.banks = (0, 1 + experts, 2 + 2 * experts)
        self.plan = sh.Plan(nodes, at, layout="block32x32")
        self.numel = at
        st = self.plan.stats()
        self.w = torch.randn(at, generator=g, device="cuda") * 0.05
        self.grad, self.mom = torch.zeros(at, device="cuda"), torch.zeros(at, device="cuda")
        self.codes, self.scales = u8(at), u8(st["scale_bytes"])
        self.ws = u8(max(st["workspace_bytes"], 256))
        sh.requant_mxfp8(self.plan, self.w, self.codes, self.scales, torch.cuda.current_stream().cuda_stream)
        self.W = [self.plan.mx_matrix(b, self.codes, self.scales) for b in self.banks]
        self.G = [self.grad[nodes[b]["offset"]:nodes[b]["offset"] + nodes[b]["rows"] * nodes[b]["cols"]] for b in self.banks]
        p = self.p = sh.moe_rows(tokens, top_k, experts, 32)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ids = torch.zeros(tokens, top_k, dtype=torch.int64, device="cuda")
        self.weights = torch.zeros(tokens, top_k, device="cuda")
        self.x, self.dout = bf(tokens, d), bf(tokens, d)
        self.offsets, self.place = torch.zeros(experts + 1, **i32), torch.zeros(tokens, top_k, **i32)
        self.source, self.sort_bytes = torch.zeros(p, **i32), sh.moe_sort_workspace(tokens, top_k, experts)
        self.sort_ws = u8(max(self.sort_bytes, 16))
        both = lambda c: (u8(p, c), u8(p, c // 32), u8(c, p), u8(c, p // 32))   # noqa: E731
        self.xs, self.dys, self.dgate, self.dup = both(d), both(d), both(f), both(f)
        self.h, self.h_t = (u8(p, f), u8(p, f // 32)), (u8(f, p), u8(f, p // 32))
        self.gate, self.up, self.dh, self.y, self.dxs = bf(p, f), bf(p, f), bf(p, f), bf(p, d), bf(p, d)
        self.out, self.dx, self.dweights = bf(tokens, d), bf(tokens, d), torch.zeros(tokens, top_k, device="cuda")

    def tokens(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits = torch.randn(self.t, self.e, generator=g, device="cuda")
        v, ids = torch.topk(logits, self.k, dim=1)
        ids[-2:] = -1                                  # padding tokens
        x = torch.randn(self.t, self.d, generator=g, device="cuda").bfloat16()
        dout = (torch.randn(self.t, self.d, generator=g, device="cuda") * 1e-2).bfloat16()
        return ids, torch.softmax(v, 1), x, dout

    def take(self, seed):
        for buf, new in zip((self.ids, self.weights, self.x, self.dout), self.tokens(seed)):
            buf.copy_(new)

    def run(self):
        """Forwards and backwards on the current stream; gradients added to the root."""
        s = torch.cuda.current_stream().cuda_stream
        t, k, e, d, f, p = self.t, self.k, self.e, self.d, self.f, self.p
        mx = lambda pair, r, c: sh.mx_matrix(pair[0], pair[1], r, c)   # noqa: E731
        names = ("codes", "scales", "codes_t", "scales_t")
        sh.moe_sort(self.ids, t, k, e, self.offsets, self.place, self.source, p, align=32, ids_dtype="int64",
                    workspace=self.sort_ws, workspace_bytes=self.sort_bytes, stream=s)
        sh.moe_gather_mxfp8(self.x, self.source, self.offsets, t, k, e, p, d, **dict(zip(names, self.xs)), stream=s)
        sh.gemm_mxfp8_swiglu(mx(self.xs, p, d), self.W[0], self.W[1], *self.h, offsets=self.offsets, groups=e,
                             gate=self.gate, up=self.up, stream=s)
        sh.gemm_mxfp8_grouped(mx(self.h, p, f), self.W[2], self.y, self.offsets, e, stream=s)
        sh.moe_combine(self.y, self.place, self.out, t, k, p, d, weights=self.weights, residual=self.x, stream=s)
        sh.moe_combine_backward(self.dout, self.y, self.weights, self.place, self.source, self.offsets, t, k, e, p, d,
                                **dict(zip(names, self.dys)), dweights=self.dweights, stream=s)
        sh.gemm_mxfp8_grouped(mx(self.dys, p, d), self.W[2], self.dh, self.offsets, e, op="nn", stream=s)
        sh.swiglu_backward_mxfp8(self.dh, self.gate, self.up, p, f, offsets=self.offsets, groups=e,
                                 dgate=sh.mx_pair(*self.dgate), dup=sh.mx_pair(*self.dup),
                                 h=sh.mx_pair(None, None, *self.h_t), stream=s)
        sh.gemm_mxfp8_grouped(mx(self.dgate, p, f), self.W[0], self.dxs, self.offsets, e, op="nn", stream=s)
        sh.gemm_mxfp8_grouped(mx(self.dup, p, f), self.W[1], self.dxs, self.offsets, e, op="nn", addend=self.dxs, stream=s)
        sh.moe_combine(self.dxs, self.place, self.dx, t, k, p, d, residual=self.dout, stream=s)
        for a, b, m, n, g in ((self.dgate[2:], self.xs[2:], f, d, 0), (self.dup[2:], self.xs[2:], f, d, 1),
                              (self.dys[2:], self.h_t, d, f, 2)):
            sh.gemm_mxfp8_grouped(mx(a, m, p), mx(b, n, p), self.G[g], self.offsets, e, op="tn", out_dtype="fp32",
                                  addend=self.G[g], stream=s)

    def results(self):
        return [self.out, self.dx, self.dweights, self.grad, self.gate, self.h[0], self.dgate[2], self.y]


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def values(pair):
    return decode(*pair)[0].cpu().numpy()


def test_each_stage_of_a_layer():
    say("expert layer, forwards and backwards")
    L = Layer(53, 2, 5, 128, 160, 1)
    L.take(7)
    L.run()
    off = host(L.offsets)
    for got, want in zip((L.offsets, L.place, L.source), M.sort(host(L.ids), L.e, 32, L.p)):
        np.testing.assert_array_equal(host(got).reshape(-1), want)
    end = off[-1]
    x, dout, w = host(L.x), host(L.dout), host(L.weights)
    place, source = host(L.place), host(L.source)

    def both(pair, v):
        codes, scales = R.quant_rows(v)
        np.testing.assert_array_equal(host(pair[0])[:end], codes[:end])
        np.testing.assert_array_equal(host(pair[1])[:end], scales[:end])
        codes, scales = R.quant_cols(v)
        np.testing.assert_array_equal(host(pair[2])[:, :end], codes[:, :end])
        np.testing.assert_array_equal(host(pair[3])[:, :end // 32], scales[:, :end // 32])
    both(L.xs, M.gather(x, None, source, off, L.k))
    both(L.dys, M.gather(dout, w, source, off, L.k))

    blocks = host(L.scales)
    banks = []
    for m in L.W:
        c0 = m.codes - L.codes.data_ptr()
        c = host(L.codes)[c0:c0 + m.rows * m.cols].reshape(m.rows, m.cols)
        s = blocks[c0 // 1024:(c0 + m.rows * m.cols) // 1024]
        banks.append(R.decode(c, s, "block32x32").reshape(L.e, -1, m.cols))

    def product(a, bank, nn, dtype="bf16", addend=None):
        out, bound = np.zeros((L.p, bank.shape[2] if nn else bank.shape[1])), 0.0
        bound = np.zeros_like(out)
        for i in range(L.e):
            r = slice(off[i], off[i + 1])
            out[r], bound[r] = R.product(a[r], bank[i].T if nn else bank[i], None, dtype)
            if addend is not None:                     # joined in float32: one more rounding of the sum
                out[r] += addend[r]
                bound[r] += (R.HALF[dtype] + 2 * R.U) * np.abs(addend[r])
        return out, bound

    def near(got, want):
        assert np.all(np.abs(host(got)[:end] - want[0][:end]) <= want[1][:end])
    xs = values(L.xs[:2])
    gate, up = product(xs, banks[0], False), product(xs, banks[1], False)
    near(L.gate, gate)
    near(L.up, up)
    # h of the sums: what is between them and the float64 products moves it by silu's slope, at most 1.1
    s = 1 / (1 + np.exp(-gate[0]))
    eg, eu = gate[1], up[1]
    h = gate[0] * s * up[0]
    eh = 1.1 * eg * (np.abs(up[0]) + eu) + np.abs(gate[0] * s) * eu + np.abs(h) * (1.25 * np.abs(gate[0]) + 8) * 2.0 ** -24
    check_codes(L.h[0][:end], L.h[1][:end], torch.from_numpy(h).cuda()[:end], torch.from_numpy(eh).cuda()[:end])
    near(L.y, product(values(L.h), banks[2], False))
    y = host(L.y)
    out, bound = M.combine(y, place, w, x, L.k, "bf16")
    assert np.all(np.abs(host(L.out) - out) <= bound)
    dw, bound = M.dweights(dout, y, place, L.k)
    assert np.all(np.abs(host(L.dweights) - dw) <= bound)
    near(L.dh, product(values(L.dys[:2]), banks[2], True))
    dxs, bound = product(values(L.dgate[:2]), banks[0], True)
    more = product(values(L.dup[:2]), banks[1], True, addend=dxs)
    near(L.dxs, (more[0], more[1] + bound * (1 + R.HALF["bf16"])))
    dx, bound = M.combine(host(L.dxs), place, None, dout, L.k, "bf16")
    assert np.all(np.abs(host(L.dx) - dx) <= bound)
    for a, b, g, m in ((L.dgate, L.xs[2:], 0, L.f), (L.dup, L.xs[2:], 1, L.f), (L.dys, L.h_t, 2, L.d)):
        at, bt = values(a[2:]), values(b)
        got = host(L.G[g]).reshape(L.e, m, -1)
        for i in range(L.e):
            r = slice(off[i], off[i + 1])
            want, bound = R.product(at[:, r], bt[:, r], None, "fp32")
            assert np.all(np.abs(got[i] - want) <= bound)


@pytest.mark.parametrize("tokens,experts", [(53, 5), (3, 70)])
def test_a_captured_layer_follows_its_tokens(tokens, experts):
    """One graph of a layer, replayed on other tokens, whose experts have other rows: each replay's bits are those of
    eager calls, with eager work between the replays."""
    say(f"expert layer captured, {tokens} tokens")
    L, ref = (Layer(tokens, 2, experts, 128, 96, 2) for _ in range(2))
    L.take(1)
    L.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    for seed in (3, 4, 5, 3):
        for z in (L, ref):
            z.take(seed)
            z.grad.zero_()
        graph.replay()
        ref.run()
        torch.cuda.synchronize()
        end = int(ref.offsets[-1])
        for a, b in zip(L.results(), ref.results()):
            if a.shape[0] == L.p and a.dim() == 2:
                a, b = a[:end], b[:end]
            if a.dim() == 2 and a.shape[1] == L.p:
                a, b = a[:, :end], b[:, :end]
            assert torch.equal(a, b)


def test_two_layers_on_two_streams():
    """Two layers at once, each on a stream of its own, have the bits of one after the other."""
    say("two expert layers at once")
    layers = [Layer(211, 3, 6, 256, 192, s) for s in (1, 2)]
    want = []
    for i, L in enumerate(layers):
        L.take(10 + i)
        L.run()
        torch.cuda.synchronize()
        want.append([r.clone() for r in L.results()])
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for L in layers:
            L.grad.zero_()
        torch.cuda.synchronize()
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.run()
        torch.cuda.synchronize()
        for L, w in zip(layers, want):
            for a, b in zip(L.results(), w):
                assert torch.equal(a, b)


def test_an_update_takes_the_layers_gradients():
    """The banks' gradients, norm and clip and update: experts no token chose keep their weights."""
    say("expert layer, update")
    L = Layer(9, 1, 6, 128, 96, 3)
    L.take(2)
    L.ids.clamp_(max=3)                                # experts 4 and 5 get nothing
    L.run()
    s = torch.cuda.current_stream().cuda_stream
    before = L.w.clone()
    n = sh.grad_workspace(L.plan)
    stats, ws = torch.zeros(2, device="cuda"), u8(max(n, 16))
    sh.grad_clip_norm(L.plan, L.grad, L.grad, 1.0, stats, ws, n, s)
    sh.update_step(L.plan, sh.buffers(L.w, L.grad, L.mom, None, L.codes, L.scales), sh.muon_hp(), None, 1, L.ws,
                   L.ws.numel(), s)
    torch.cuda.synchronize()
    norm = float(np.sqrt(np.sum(host(L.grad).astype(np.float64) ** 2)))
    assert float(stats[0]) > 0 and norm <= 1.0 + 1e-6
    used = set(host(L.ids).reshape(-1).tolist()) - {-1}
    moved = (host(L.w) != host(before)).reshape(3, L.e, -1).any(axis=2)
    assert moved.tolist() == [[e in used for e in range(L.e)]] * 3
