"""The residual RMS norm and its gradient beside a plan's own norm units: weight and
weight gradient at any element of the roots, and how the weight gradient's sums are
joined, against float64 references."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import ops_ref as R
from gpu_util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def stream():
    return torch.cuda.current_stream().cuda_stream


def dev(a, dtype="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy()


def matrix(rng, rows, cols, dtype):
    return R.as_dtype((rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)))).astype(np.float32), dtype)


def backward(dy, h, w, rstd, dw, rows, cols, first=True, dtype="fp32", weight_dtype="fp32"):
    dx = torch.full((rows + 1, cols), 3.0, dtype=dy.dtype, device="cuda")
    nb = sh.rmsnorm_backward_workspace(rows, cols)
    ws = torch.full((max(nb, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    sh.rmsnorm_backward(dy, h, w, rstd, dx, dw, rows, cols, dtype=dtype, weight_dtype=weight_dtype, first=first,
                        workspace=ws, workspace_bytes=nb, stream=stream())
    assert bool((dx[rows] == 3.0).all())
    return dx[:rows]


@pytest.mark.parametrize("at", [1, 2, 3, 6])
@pytest.mark.parametrize("rows,cols", [(1, 32), (40, 2048), (1100, 96), (70, 16416)])
def test_weight_gradient_at_any_element(rows, cols, at):
    """The unit's place and nothing around it, by one launch or two, set and added to."""
    say(f"dweight at {at} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols + at)
    dy, h = matrix(rng, rows, cols, "fp32"), matrix(rng, rows, cols, "fp32")
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    rstd = R.rmsnorm(h, None, w, 1e-6, "fp32")[1].astype(np.float32)
    _, _, dw, bdw = R.rmsnorm_grad(dy, h, w, rstd, None, "fp32")
    g = torch.full((cols + 9,), 7.0, device="cuda")
    args = [dev(v) for v in (dy, h, w, rstd)]
    backward(*args, g[at:], rows, cols)
    backward(*args, g[at:], rows, cols, first=False)
    got = host(g)
    assert np.all(np.abs(got[at:at + cols] - 2 * dw) <= 2 * bdw + R.U * np.abs(2 * dw))
    assert np.all(got[:at] == 7.0) and np.all(got[at + cols:] == 7.0)


@pytest.mark.parametrize("wdtype,at", [("fp32", 1), ("fp32", 2), ("bf16", 1), ("bf16", 3), ("bf16", 6)])
@pytest.mark.parametrize("rows,cols", [(1, 8192), (33, 544), (1100, 96), (3, 20512)])
def test_weight_at_any_element(rows, cols, wdtype, at):
    """Codes, scales and gradient of a weight inside a root that is NaN around it: bit for bit those of an aligned copy."""
    say(f"norm weight at {at} {wdtype} {rows}x{cols}")
    rng = np.random.default_rng(rows + cols + at)
    x, dy = matrix(rng, rows, cols, "bf16"), matrix(rng, rows, cols, "bf16")
    w = R.as_dtype(1 + 0.2 * rng.standard_normal(cols), wdtype)
    root = dev(np.concatenate([np.full(at, np.nan), w, np.full(9, np.nan)]), wdtype)
    _, rstd, y = R.rmsnorm(x, None, w, 1e-6, "bf16")
    qc, qs = R.quant_rows(y)
    xd, dyd, runs = dev(x, "bf16"), dev(dy, "bf16"), []
    for weight in (root[at:], dev(w, wdtype)):
        c = torch.full((rows, cols), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device="cuda")
        rs = torch.zeros(rows, device="cuda")
        sh.rmsnorm_mxfp8(xd, weight, rows, cols, weight_dtype=wdtype, codes=c, scales=s, rstd=rs, stream=stream())
        assert np.array_equal(host(c), qc) and np.array_equal(host(s), qs)
        assert np.all(np.abs(host(rs) - rstd) <= 1.01 * R.U * rstd)
        dw = torch.full((cols,), 3.0, device="cuda")
        runs.append((backward(dyd, xd, weight, rs, dw, rows, cols, dtype="bf16", weight_dtype=wdtype), dw))
    dx, bdx, dw, bdw = R.rmsnorm_grad(dy, x, w, host(rs), None, "bf16")
    assert np.all(np.abs(host(runs[0][0]) - dx) <= bdx) and np.all(np.abs(host(runs[0][1]) - dw) <= bdw)
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


@pytest.mark.parametrize("rows,picked", [(64, range(1, 64)), (1100, range(4, 128, 4))])
def test_weight_gradient_sums_in_pairs(rows, picked):
    """One large term and many of half its last place, each alone in its slice of the rows: a chain of additions
    loses all of them (63 and 31 half steps of the sum).  Adding zeros is exact, and adding the slices in pairs
    rounds a value once a level (6 and 5 levels) before the store, whose sum with nothing is exact."""
    say(f"dweight in pairs {rows}")
    cols = 64
    h = np.ones((rows, cols), np.float32)
    dy = np.zeros((rows, cols), np.float32)
    dy[0] = 1.0
    dy[list(picked)] = R.U
    dw = torch.full((cols,), 3.0, device="cuda")
    backward(dev(dy), dev(h), dev(np.ones(cols)), dev(np.ones(rows)), dw, rows, cols)
    exact = 1.0 + len(picked) * R.U
    levels = 6 if rows == 64 else 5
    assert np.all(np.abs(host(dw).astype(np.float64) - exact) <= levels * R.U * exact)
