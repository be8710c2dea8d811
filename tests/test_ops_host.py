"""The operators around the update on the host (no GPU): their refusals (every
argument error comes before anything touches the device), their workspace sizes,
a plan's regions as product operands, the gradient norm's work items, and the
norm gradient's formula against differences."""

import os
import shutil
import struct
import subprocess

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
from mxfp8_weight_repack_amd._lib import LAYOUT, node_array
import ops_ref as R
import workloads
from oracle.mxfp8 import scale_index

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20                                            # an aligned address that no refused call follows


def refused(name, call):
    with pytest.raises(sh.SshdpError) as e:
        call()
    assert e.value.name == name, (e.value.name, name)


def test_quant_refusals():
    q = lambda *a, **k: (lambda: sh.quant_mxfp8(*a, **k))   # noqa: E731
    refused("ARG", q(P, "fp16", 4, 32, P, P))
    refused("ARG", q(P, "fp32", -1, 32, P, P))
    refused("ARG", q(None, "fp32", 4, 32, P, P))
    refused("ARG", q(P, "fp32", 4, 32, P, None))
    refused("ARG", q(P, "fp32", 4, 32, None, None, None, P))
    refused("ARG", q(P, "fp32", 4, 32))
    refused("SCHEMA", q(P, "fp32", 4, 48, P, P))
    refused("SCHEMA", q(P, "fp32", 4, 64, P, P, ld=32))
    refused("SCHEMA", q(P, "bf16", 4, 64, P, P, ld=68))
    refused("SCHEMA", q(P, "fp32", (1 << 30) + 1, 32, P, P))
    refused("ALIGN", q(P + 4, "fp32", 4, 32, P, P))
    refused("ALIGN", q(P, "fp32", 4, 32, P + 8, P))
    refused("ALIGN", q(P, "fp32", 4, 32, None, None, P + 8, P))
    sh.quant_mxfp8(None, "fp32", 0, 32)                # nothing to do
    sh.quant_mxfp8(None, "fp32", 5, 0)


def test_rmsnorm_refusals():
    q = lambda *a, **k: (lambda: sh.rmsnorm_mxfp8(*a, **k))   # noqa: E731
    refused("ARG", q(P, P, 4, 32, dtype="x", y=P))
    refused("ARG", q(P, P, 4, 32, weight_dtype="x", y=P))
    refused("ARG", q(P, P, 4, 32, y=P, eps=-1.0))
    refused("ARG", q(P, P, 4, 32, y=P, eps=float("nan")))
    refused("ARG", q(P, P, 4, 32))                     # no output
    refused("ARG", q(None, P, 4, 32, y=P))
    refused("ARG", q(P, None, 4, 32, y=P))
    refused("ARG", q(P, P, 4, 32, codes=P))
    refused("ARG", q(P, P, 4, 32, h=P))                # h without a residual
    refused("SCHEMA", q(P, P, 4, 40, y=P))
    refused("SCHEMA", q(P, P, 4, 32800, y=P))
    refused("SCHEMA", q(P, P, 4, 64, y=P, ld_x=32))
    refused("SCHEMA", q(P, P, 4, 64, y=P, ld_x=68))
    refused("SCHEMA", q(P, P, 4, 64, y=P, residual=P, ld_residual=60))
    for k in ("y", "codes", "rstd"):
        refused("ALIGN", q(P, P, 4, 32, **dict({"scales": P} if k == "codes" else {}, **{k: P + 4})))
    refused("ALIGN", q(P, P, 4, 32, y=P, residual=P + 8))
    sh.rmsnorm_mxfp8(None, None, 0, 64)


def test_rmsnorm_in_place_needs_dense_rows():
    """h is dense: over x or a residual with gaps it would overwrite rows not read yet."""
    for kw in (dict(h=P, ld_x=64), dict(h=P + 4096, residual=P + 4096, ld_residual=40)):
        refused("SCHEMA", lambda: sh.rmsnorm_mxfp8(P, P, 4, 32, **dict(dict(residual=P + 8192), **kw)))


def test_rmsnorm_backward_refusals():
    nb = sh.rmsnorm_backward_workspace(4, 64)
    assert nb >= 64 * 4 and nb % 16 == 0
    assert sh.rmsnorm_backward_workspace(0, 64) == 0
    ok = dict(workspace=P, workspace_bytes=nb)
    q = lambda *a, **k: (lambda: sh.rmsnorm_backward(*a, **k))   # noqa: E731
    refused("ARG", q(P, P, P, P, P, None, 4, 64, **ok))
    for i in range(5):
        args = [P] * 6
        args[i] = None
        refused("ARG", q(*args, 4, 64, **ok))
    refused("ARG", q(P, P, P, P, P, P, 4, 64, dtype="x", **ok))
    refused("SCHEMA", q(P, P, P, P, P, P, 4, 70, **ok))
    refused("SCHEMA", q(P, P, P, P, P, P, 4, 32800, **ok))
    refused("ALIGN", q(P, P + 8, P, P, P, P, 4, 64, **ok))
    refused("ALIGN", q(P, P, P, P, P, P, 4, 64, dh=P + 2, **ok))
    refused("WORKSPACE", q(P, P, P, P, P, P, 4, 64))
    refused("WORKSPACE", q(P, P, P, P, P, P, 4, 64, workspace=P, workspace_bytes=nb - 1))
    refused("ALIGN", q(P, P, P, P, P, P, 4, 64, workspace=P + 8, workspace_bytes=nb))
    sh.rmsnorm_backward(None, None, None, None, None, None, 0, 64, first=False)


def test_rmsnorm_weight_gradient_at_any_element():
    """A norm unit may start at any element of the gradient root: past the alignment check, the missing workspace
    is what is left to refuse."""
    for at in (4, 8, 12, 20):
        refused("WORKSPACE", lambda: sh.rmsnorm_backward(P, P, P, P, P, P + at, 4, 64))
    refused("ALIGN", lambda: sh.rmsnorm_backward(P, P, P, P, P, P + 2, 4, 64))


def test_rmsnorm_weight_at_any_element():
    """The weight may start at any element of its root; what is refused then is what comes after its alignment."""
    for dtype, at in (("fp32", 4), ("fp32", 12), ("bf16", 2), ("bf16", 10)):
        refused("WORKSPACE", lambda: sh.rmsnorm_backward(P, P, P + at, P, P, P, 4, 64, weight_dtype=dtype))
        refused("ALIGN", lambda: sh.rmsnorm_backward(P, P, P + at - 1, P, P, P, 4, 64, weight_dtype=dtype))
        refused("ALIGN", lambda: sh.rmsnorm_mxfp8(P, P + at - 1, 4, 64, weight_dtype=dtype, y=P))
    refused("ALIGN", lambda: sh.rmsnorm_mxfp8(P, P + 2, 4, 64, weight_dtype="fp32", y=P))


def test_gemm_refusals():
    mat = lambda r, c, layout="rowmajor", codes=P, scales=P: sh.mx_matrix(codes, scales, r, c, layout)   # noqa: E731

    def g(a, b, out=P, **k):
        return lambda: sh.gemm_mxfp8(a, b, out, **k)

    a, b = mat(8, 64), mat(16, 64)
    refused("ARG", g(mat(8, 64, "other"), b))
    refused("ARG", g(mat(-1, 64), b))
    refused("ARG", g(mat(8, 64, codes=None), b))
    refused("ARG", g(a, mat(16, 64, scales=None)))
    refused("ARG", g(a, b, op="tn"))
    refused("ARG", g(a, b, out_dtype="fp16"))
    refused("ARG", g(a, b, out_dtype="bf16", addend=P))
    refused("ARG", g(a, b, out=None))
    refused("SCHEMA", g(a, mat(16, 96)))
    refused("SCHEMA", g(mat(8, 48), mat(16, 48)))
    refused("SCHEMA", g(a, mat(64, 64, "rowmajor"), op="nn"))             # needs 32 x 32 blocks
    refused("SCHEMA", g(a, mat(16, 64, "block32x32")))                    # 16 rows
    refused("SCHEMA", g(a, mat(48, 64, "block32x32"), op="nn"))
    refused("SCHEMA", g(a, mat(96, 64, "block32x32"), op="nn"))           # K differs
    refused("SCHEMA", g(mat(8, 96), mat(32, 96, "tile32x4")))             # cols % 128
    refused("SCHEMA", g(a, b, ld_out=15))
    refused("SCHEMA", g(mat(8, (1 << 22) + 32), mat(8, (1 << 22) + 32)))
    refused("SCHEMA", g(mat((1 << 30) + 1, 32), mat(8, 32)))
    refused("ALIGN", g(a, b, out=P + 8))
    refused("ALIGN", g(mat(8, 64, codes=P + 4), b))
    refused("ALIGN", g(a, b, out_dtype="fp32", addend=P + 8))
    big_a, big_b = mat(64, 1 << 16), mat(64, 1 << 16)
    nb = sh.gemm_mxfp8_workspace(big_a, big_b)
    if nb:
        refused("WORKSPACE", g(big_a, big_b, workspace=P, workspace_bytes=nb - 1))
        refused("ALIGN", g(big_a, big_b, workspace=P + 4, workspace_bytes=nb))
    sh.gemm_mxfp8(mat(0, 64, codes=None, scales=None), b, None)           # no rows: nothing to do


def test_gemm_workspace_of_every_small_size():
    """Down to empty operands: none divides by nothing, and each answer holds a whole number of partial outputs."""
    for m in (0, 1, 16, 17, 300, 5000):
        for n in (0, 1, 32, 96, 128, 8192):
            for k in (0, 32, 96, 128, 544, 4096):
                for op in ("nt", "nn"):
                    if op == "nn" and n % 32:
                        continue
                    a = sh.mx_matrix(P, P, m, k)
                    b = sh.mx_matrix(P, P, *((k, n, "block32x32") if op == "nn" else (n, k)))
                    size = sh.gemm_mxfp8_workspace(a, b, op=op)
                    assert size >= 0 and size % max(4 * m * ((n + 3) // 4 * 4), 1) == 0


def test_grad_refusals_on_a_host_only_plan():
    node = dict(parent=-1, offset=0, rows=1, cols=64, row_stride=64, is_unit=True, optimizer="adamw", quantize=None)
    p = sh.Plan([node], 64, host_only=True)
    assert sh.grad_workspace(p) > 0
    refused("STATE", lambda: sh.grad_clip_norm(p, P, P, 1.0, P, P, 1 << 20))
    refused("STATE", lambda: sh.grad_sumsq(p, P, P, P, 1 << 20))
    refused("STATE", lambda: sh.grad_clip(p, P, P, P, 1.0, P))


@pytest.mark.parametrize("layout", ["rowmajor", "tile32x4", "block32x32"])
def test_plan_regions_as_operands(layout):
    """A region's operand points at its own codes and scales inside the roots."""
    nodes = [dict(parent=-1, offset=0, rows=64, cols=256, row_stride=256, is_unit=True, optimizer="muon", quantize=True),
             dict(parent=-1, offset=64 * 256, rows=32, cols=128, row_stride=128, is_unit=False, quantize=True),
             dict(parent=-1, offset=20480, rows=1, cols=128, row_stride=128, is_unit=True, optimizer="adamw")]
    p = sh.Plan(nodes, 20608, layout=layout, host_only=True)
    m = p.mx_matrix(1, P, 2 * P)
    assert (m.codes, m.rows, m.cols, m.layout) == (P + 64 * 256, 32, 128, LAYOUT[layout])
    assert m.scales == 2 * P + 64 * 256 // (1024 if layout == "block32x32" else 32)
    refused("SCHEMA", lambda: p.mx_matrix(2, P, P))    # no MXFP8 region
    refused("ARG", lambda: p.mx_matrix(3, P, P))
    refused("ARG", lambda: p.mx_matrix(0, None, P))


@pytest.mark.parametrize("layout", ["rowmajor", "tile32x4", "block32x32"])
def test_views_of_a_region_as_operands(layout):
    """Whole rows of a region (an expert of a bank, a head of a packed projection) are operands of their own:
    codes from their first element on, and the very scales that the region's formula gives those rows."""
    view = lambda offset, rows, cols=256, stride=256, parent=1: dict(   # noqa: E731
        parent=parent, offset=offset, rows=rows, cols=cols, row_stride=stride, is_unit=False, quantize=None)
    base, rows, cols = 4096, 160, 256
    nodes = [dict(parent=-1, offset=0, rows=1, cols=4096, row_stride=4096, is_unit=True, optimizer="adamw"),
             dict(parent=-1, offset=base, rows=rows, cols=cols, row_stride=cols, is_unit=False, quantize=True),
             view(0, 64), view(64 * 256, 96), view(160, 1, 96, 96, 0), view(32 * 256, 64, 128), view(128, 2, 256),
             view(32 * 256, 16, 256, 512), view(0, 160), view(33 * 256, 1), view(32 * 256, 32, 256, 256, 1)]
    nodes.append(dict(nodes[10], parent=3, offset=32 * 256))           # a view of a view: rows 96 .. 127
    p = sh.Plan(nodes, base + rows * cols, layout=layout, host_only=True)
    index = scale_index(layout, base, rows, cols)
    br = 32 if layout == "block32x32" else 1
    good = {2: (0, 64), 3: (64, 96), 8: (0, 160), 10: (32, 32), 11: (96, 32)}
    if layout == "rowmajor":
        good[9] = (33, 1)
    for i, (first, n) in good.items():
        m = p.mx_matrix(i, P, 2 * P)
        assert (m.codes, m.rows, m.cols, m.layout) == (P + base + first * cols, n, cols, LAYOUT[layout])
        assert np.array_equal(m.scales - 2 * P + scale_index(layout, 0, n, cols), index[first // br:(first + n) // br])
    for i in set(range(12)) - set(good) - {1}:         # outside, part of the columns, across rows, with gaps
        refused("SCHEMA", lambda: p.mx_matrix(i, P, P))


def test_every_expert_of_a_bank_is_an_operand():
    """The expert bank's node carries `quantize`; its experts are views inside it."""
    wl = workloads.config(3)
    p = sh.Plan(wl.nodes, wl.root_numel, layout=wl.scale_layout, host_only=True)
    bank = [i for i, n in enumerate(wl.nodes) if n["quantize"]]
    experts = [i for i, n in enumerate(wl.nodes) if n["parent"] in bank and not n["quantize"]]
    assert len(experts) >= 64
    for i in experts:
        m, o = p.mx_matrix(i, P, 2 * P), p.node(i)[0]
        assert (m.codes, m.scales, m.rows, m.cols) == (P + o, 2 * P + o // 32, wl.nodes[i]["rows"], wl.nodes[i]["cols"])


def test_gradient_chunks_cover_every_unit_element_once(tmp_path):
    """The norm's work items of every workload: each unit element once, nothing else."""
    if not (os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h") and shutil.which("g++")):
        pytest.skip("ROCm headers or g++ missing")
    exe, data = tmp_path / "gradchk", tmp_path / "trees.bin"
    csrc = os.path.join(ROOT, "mxfp8_weight_repack_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(ROOT, "include"), "-I", csrc, "-I", "/opt/rocm/include",
                        os.path.join(csrc, "plan.cpp"), os.path.join(ROOT, "tests", "host_grad_check.cpp"),
                        "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    wls = [workloads.config(c, small=c != 1) for c in (1, 2, 3, 4, 5)] + [workloads.ragged_mix(), workloads.random_units()]
    with open(data, "wb") as f:
        for wl in wls:
            f.write(struct.pack("<iqiI", len(wl.nodes), wl.root_numel, LAYOUT["rowmajor"], 0))
            f.write(bytes(node_array([dict(n, quantize=None) for n in wl.nodes])))
    r = subprocess.run([str(exe), str(data)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0, (r.stdout[-2000:], r.stderr[-3000:])
    lines = [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    assert [line[0] for line in lines] == [wl.params for wl in wls]
    tiny = lines[0]                                    # head views tile their matrix: whole chunks, few of them
    assert tiny[1] <= wls[0].params // 4096 + 4


def test_norm_gradient_formula_against_differences():
    """The float64 formula the kernels are held to, against central differences of the norm itself."""
    rng = np.random.default_rng(11)
    rows, cols, eps = 3, 32, 1e-3
    x, w, dy = rng.standard_normal((rows, cols)), 1 + 0.3 * rng.standard_normal(cols), rng.standard_normal((rows, cols))

    def loss(x, w):
        return np.sum(dy * x * w / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps))

    rstd = 1 / np.sqrt(np.mean(x * x, axis=1) + eps)
    dx, _, dw, _ = R.rmsnorm_grad(dy, x, w, rstd, None, "fp32")
    step = 1e-5
    # central differences: step^2 of the third derivative (order 1 here) and 2^-53 / step of the loss
    for i in range(rows):
        for j in range(cols):
            d = np.zeros_like(x)
            d[i, j] = step
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * step) - dx[i, j]) < 1e-8
    for j in range(cols):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * step) - dw[j]) < 1e-8
