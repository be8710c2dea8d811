"""The operators around the update where calls share the GPU: a layer's step captured
and replayed, and calls on two streams that run at the same time, compared to the bit
with the same calls alone."""

import pytest

import mxfp8_weight_repack_amd as sh
from gpu_util import say
from test_gpu_ops import Layer, unit

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def same(a, b):
    """Equal bits, NaN and the sign of zero included."""
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


def test_a_captured_step_to_the_bit():
    """A step captured once and replayed on new inputs, with eager work between, leaves an eager step's very bits."""
    say("layer graph to the bit")
    G, E = Layer(4), Layer(4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        G.step()
    torch.cuda.current_stream().wait_stream(side)
    E.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        G.step()
    for rep in range(4):
        for L in (G, E):
            g = torch.Generator(device="cuda").manual_seed(20 + rep)
            for t in L.x + L.dy:
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        E.step()
        torch.cuda.synchronize()
        a, b = G.state(), E.state()
        for k in a:
            assert same(a[k], b[k]), (rep, k)
            assert not (a[k].is_floating_point() and bool(a[k].isnan().any())), (rep, k)


class Calls:
    """One user's calls, each long enough to meet the other user's: products with K split (both output types, both
    forms) and whole, a norm and its gradient by partial rows, quantising both ways, and the clip."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")   # noqa: E731
        M, D, self.n = 4090, 2048, 6_000_001
        self.M, self.D = M, D
        self.x, self.res, self.dy, self.w = r(M, D).bfloat16(), r(M, D).bfloat16(), r(M, D).bfloat16(), r(D)
        self.grad = r(self.n + 7)
        self.plan = sh.Plan([unit(3, 1, self.n)], self.n + 7)
        wm, xm = r(256, 8192), r(200, 8192)
        self.b = sh.mx_matrix(u8(256, 8192), u8(256, 256), 256, 8192)
        self.a = sh.mx_matrix(u8(200, 8192), u8(200, 256), 200, 8192)
        for src, m in ((wm, self.b), (xm, self.a)):
            sh.quant_mxfp8(src, "fp32", m.rows, m.cols, *m._keep, stream=torch.cuda.current_stream().cuda_stream)
        nn = torch.randint(0, 120, (8192, 256), generator=g, device="cuda").to(torch.uint8)
        self.bn = sh.mx_matrix(nn, torch.full((256, 8), 122, dtype=torch.uint8, device="cuda"), 8192, 256, "block32x32")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.o = dict(h=torch.zeros(M, D, **bf), y=torch.zeros(M, D, **bf), c=u8(M, D), s=u8(M, D // 32),
                      rstd=torch.zeros(M, device="cuda"), dx=torch.zeros(M, D, **bf), dw=torch.zeros(D, device="cuda"),
                      qc=u8(M, D), qs=u8(M, D // 32), ct=u8(D, 4096), st=u8(D, 128), p32=torch.zeros(200, 256, device="cuda"),
                      p16=torch.zeros(200, 256, **bf), n32=torch.zeros(200, 256, device="cuda"),
                      n16=torch.zeros(200, 256, **bf), clip=torch.zeros(self.n + 7, device="cuda"),
                      stats=torch.zeros(2, device="cuda"))
        self.ws = {}
        for op, b in (("nt", self.b), ("nn", self.bn)):
            assert sh.gemm_mxfp8_workspace(self.a, b, op=op) > 0       # K is split
            self.ws[op] = u8(sh.gemm_mxfp8_workspace(self.a, b, op=op))
        self.ws["norm"], self.ws["clip"] = u8(sh.rmsnorm_backward_workspace(M, D)), u8(sh.grad_workspace(self.plan))

    def each(self):
        """The calls, one at a time, on the current stream."""
        o, M, D, w = self.o, self.M, self.D, self.ws
        st = lambda: torch.cuda.current_stream().cuda_stream   # noqa: E731
        yield lambda: sh.rmsnorm_mxfp8(self.x, self.w, M, D, residual=self.res, h=o["h"], y=o["y"], codes=o["c"],
                                       scales=o["s"], rstd=o["rstd"], stream=st())
        for op, b, out, dtype in (("nt", self.b, "p32", "fp32"), ("nn", self.bn, "n16", "bf16"),
                                  ("nt", self.b, "p16", "bf16"), ("nn", self.bn, "n32", "fp32")):
            yield lambda op=op, b=b, out=out, dtype=dtype: sh.gemm_mxfp8(
                self.a, b, o[out], dtype, op=op, workspace=w[op], workspace_bytes=w[op].numel(), stream=st())
        yield lambda: sh.rmsnorm_backward(self.dy, o["h"], self.w, o["rstd"], o["dx"], o["dw"], M, D,
                                          workspace=w["norm"], workspace_bytes=w["norm"].numel(), stream=st())
        yield lambda: sh.quant_mxfp8(o["y"], "bf16", M, D, o["qc"], o["qs"], o["ct"], o["st"], stream=st())
        yield lambda: sh.grad_clip_norm(self.plan, self.grad, o["clip"], 0.5, o["stats"], w["clip"], w["clip"].numel(), st())

    def clear(self):
        for t in self.o.values():
            t.zero_()


def test_two_streams_in_turn():
    """Two users' calls, issued in turn, one a call behind, behind an event that both streams wait for: when it comes
    the GPU has both queues full.  Each user's outputs are the bits that it gets alone."""
    say("two streams in turn")
    users = [Calls(1), Calls(2)]
    torch.cuda.synchronize()
    alone = []
    for u in users:
        for call in u.each():
            call()
        torch.cuda.synchronize()
        alone.append({k: v.clone() for k, v in u.o.items()})
        assert all(bool(v.any()) for v in alone[-1].values())
    gate, streams = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    big = torch.randn(8192, 8192, device="cuda")
    for rep in range(4):
        for u in users:
            u.clear()
        torch.cuda.synchronize()
        with torch.cuda.stream(gate):
            big @ big
            event = gate.record_event()
        for s in streams:
            s.wait_event(event)
        queues = [list(u.each()) for u in users]
        queues[rep % 2] = [None] + queues[rep % 2]     # one a call behind: different calls side by side
        for i in range(max(map(len, queues))):
            for q, s in zip(queues, streams):
                if i < len(q) and q[i]:
                    with torch.cuda.stream(s):
                        q[i]()
        torch.cuda.synchronize()
        for u, a in zip(users, alone):
            for k in a:
                assert same(u.o[k], a[k]), (rep, k)
