"""G of the expert layer's operators is made by gfx950's scaled conversions: their codes against the oracle's for every
bfloat16 value under every scale byte, and for float32 values at and beside the rounding borders, subnormal ones among
them, along the rows and along the columns, weighted (float32 arithmetic ahead) and not."""

import numpy as np
import pytest

import mxfp8_weight_repack_amd as sh
import ops_ref as R
from gpu_util import say
from test_gpu_moe import buf, dev, host, stream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

COLS = 2048


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sh.lib()


def anchor(byte):
    """The largest magnitude of a block whose scale byte this is, as a bfloat16 value."""
    if byte == 247:                                    # float32's end: bfloat16's largest
        return np.float32(np.ldexp(255.0, 120))
    return np.float32(np.ldexp(448.0, byte - 127))


def blocks_of(values, byte):
    """Blocks of 32 of these magnitudes (none above the anchor) with alternating signs, the anchor at the end of each."""
    v = values[values <= anchor(byte)]
    v = np.concatenate([v, np.zeros(-v.size % 31, np.float32)]).reshape(-1, 31)
    v = np.concatenate([v, np.full((v.shape[0], 1), anchor(byte), np.float32)], axis=1)
    v[:, 1::2] *= -1
    v[::2] *= -1
    return v


def every_bfloat16():
    """Each scale byte's values from 2^-20 of its anchor on, and 2^-20 of it and less by a stride."""
    all_ = (np.arange(0x7F80, dtype=np.uint32) << 16).view(np.float32)
    out = []
    for byte in range(248):
        small = all_ < anchor(byte) * np.float32(2.0 ** -20)
        out.append(blocks_of(np.concatenate([all_[~small], all_[small]]), byte))
    return np.concatenate(out)


def float32_borders():
    """Around codes' rounding borders of each scale: the border and its two neighbours; and values of random bits."""
    rng = np.random.default_rng(2)
    mags = np.sort(np.unique(np.abs(R._TABLE[np.isfinite(R._TABLE)])))
    mids = (mags[1:] + mags[:-1]) / 2
    out = []
    for byte in range(248):
        with np.errstate(over="ignore"):
            b = np.ldexp(np.concatenate([mids, mags]), byte - 127).astype(np.float32)
        b = b[np.isfinite(b)]
        some = rng.integers(0, int(anchor(byte).view(np.uint32)) + 1, 1000, dtype=np.uint32).view(np.float32)
        near = (anchor(byte) * np.exp2(-24 * rng.random(1000, dtype=np.float32))).astype(np.float32)
        out.append(blocks_of(np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(np.inf)), some, near]),
                             byte))
    return np.concatenate(out)


@pytest.mark.parametrize("which,dtype", [("every bfloat16", "bf16"), ("borders", "fp32")])
def test_codes_of_every_value(which, dtype):
    say(f"encode, {which}")
    v = every_bfloat16() if dtype == "bf16" else float32_borders()
    per = 32 * COLS
    v = np.concatenate([v.reshape(-1), np.zeros(-v.size % per, np.float32)]).reshape(-1, 32)
    codes, scales = R.quant_rows(v)
    rows = v.size // COLS
    assert rows // 128 * (COLS // 128) < 768
    x = v.reshape(rows, COLS)
    # the same blocks along the columns: 32 rows of a column each
    xt = np.ascontiguousarray(v.reshape(rows // 32, COLS, 32).transpose(0, 2, 1)).reshape(rows, COLS)
    want = codes.reshape(rows, COLS), scales.reshape(rows, COLS // 32)
    want_t = (codes.reshape(rows // 32, COLS, 32).transpose(1, 0, 2).reshape(COLS, rows),
              scales.reshape(rows // 32, COLS).T)
    source = torch.arange(rows, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ones = torch.ones(rows, device="cuda")
    xd, td = dev(x, dtype), dev(xt, dtype)
    for weights in (None, ones):
        for y in (None, torch.zeros_like(xd)):         # by tiles, and (with y, few tiles) by runs
            c, s = buf(rows, COLS), buf(rows, COLS // 32)
            sh.moe_gather_mxfp8(xd, source, offsets, rows, 1, 1, rows, COLS, dtype=dtype, weights=weights, codes=c, scales=s,
                                y=y, stream=stream())
            np.testing.assert_array_equal(host(s), want[1])
            np.testing.assert_array_equal(host(c), want[0])
        c, s = buf(COLS, rows), buf(COLS, rows // 32)
        sh.moe_gather_mxfp8(td, source, offsets, rows, 1, 1, rows, COLS, dtype=dtype, weights=weights, codes_t=c, scales_t=s,
                            stream=stream())
        np.testing.assert_array_equal(host(s), want_t[1])
        np.testing.assert_array_equal(host(c), want_t[0])
