"""Float64 references of the operators around the update, in NumPy, and the
error bounds their float32 arithmetic allows.  u = 2^-24 is half a step of
float32 relative to the value."""

import numpy as np

import oracle
from oracle.mxfp8 import quantize_blocks_fast, quantize_blocks_32x32, scale_index
from oracle.numerics import bf16_rne

U = 2.0 ** -24
HALF = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}        # half a step, relative, of a stored result


def as_dtype(x, dtype):
    """float32 values rounded to dtype (kept in float32)."""
    x = np.asarray(x, np.float32)
    return x if dtype == "fp32" else bf16_rne(x)


def quant_rows(x):
    with np.errstate(all="ignore"):
        return quantize_blocks_fast(np.ascontiguousarray(x, dtype=np.float32))


def quant_cols(x):
    """(codes_t, scales_t): the transpose, rows padded to 32 with zeros (code 0 there)."""
    r, c = x.shape
    rp = (r + 31) // 32 * 32
    t = np.zeros((c, rp), np.float32)
    t[:, :r] = x.T
    codes, s = quant_rows(t)
    codes[:, r:] = 0
    return codes, s


def rmsnorm(x, residual, weight, eps, dtype):
    """h (float32 values of dtype), rstd (float64), y (float32)."""
    h = np.asarray(x, np.float32)
    if residual is not None:
        h = as_dtype(h + np.asarray(residual, np.float32), dtype)
    h64 = h.astype(np.float64)
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt(np.mean(h64 * h64, axis=1) + np.float64(np.float32(eps)))
        y = (h64 * rstd[:, None] * np.asarray(weight, np.float64)).astype(np.float32)
    return h, rstd, y


def rmsnorm_grad(dy, h, weight, rstd, dh, dtype):
    """dx, dweight in float64 and the bounds of their float32 computation.

    A lane adds at most 32 products w dy xhat in float32 before float64 takes
    over, each product off by 3 roundings: the mean is off by (32 + 4) u mean|w dy
    xhat|.  dx then takes 3 products and 2 sums, 5 u of every term, and its own
    rounding to dtype.  dweight adds dy xhat over at most `rows` rows in a chain
    and up to 64 partial rows: (rows + 64 + 2) u sum|dy xhat|, rounded once."""
    dy, h, w, r = (np.asarray(v, np.float64) for v in (dy, h, weight, rstd))
    xhat = h * r[:, None]
    wdy = dy * w
    mean = np.mean(wdy * xhat, axis=1, keepdims=True)
    amean = np.mean(np.abs(wdy * xhat), axis=1, keepdims=True)
    d = 0.0 if dh is None else np.asarray(dh, np.float64)
    dx = r[:, None] * (wdy - xhat * mean) + d
    e = r[:, None] * (np.abs(xhat) * 36 * U * amean + 5 * U * (np.abs(wdy) + np.abs(xhat * mean))) + 2 * U * np.abs(d)
    bdx = e + HALF[dtype] * (np.abs(dx) + e) + 2.0 ** -133
    dw = np.sum(dy * xhat, axis=0)
    bdw = (dy.shape[0] + 66) * U * np.sum(np.abs(dy * xhat), axis=0) + U * np.abs(dw)
    return dx, bdx, dw, bdw


_TABLE = np.asarray(oracle.e4m3_decode(np.arange(256, dtype=np.uint8)), np.float64)


def decode(codes, scales, layout):
    """Float64 values of an MXFP8 matrix; scales flat in `layout`."""
    rows, cols = codes.shape
    s = np.asarray(scales, np.uint8).reshape(-1)
    if rows == 0 or cols == 0:
        return np.zeros((rows, cols))
    if layout == "block32x32":
        sm = np.repeat(s[scale_index(layout, 0, rows, cols)], 32, axis=0)
    else:
        sm = s[scale_index(layout, 0, rows, cols)]
    f = np.where(sm == 255, np.nan, np.ldexp(1.0, sm.astype(int) - 127))
    return _TABLE[codes] * np.repeat(f, 32, axis=1)


def quant_weight(w, layout):
    """Codes and flat scales of a float32 matrix in a scale layout."""
    if layout == "block32x32":
        c, s = quantize_blocks_32x32(w)
        return c, s.reshape(-1)
    c, s = quant_rows(w)
    out = np.zeros(s.size, np.uint8)
    out[scale_index(layout, 0, *w.shape)] = s
    return c, out


def product(a, b, addend, dtype):
    """a b^T (+ addend) in float64, and the bound on its computation.

    Float32 output: exact products added in float32 in any order: each of the K
    additions off by at most a whole step 2u (whether it rounds or truncates) of a
    sum no larger than sum|a b|, then the stored result's rounding.  bfloat16
    output: besides that, the 8-bit matrix instruction cuts the products of each 8
    consecutive k off at 2^-14 of the binade of their largest; the largest itself
    (8 significant bits) loses nothing, so a group loses less than 7 * 2^-14 of it."""
    with np.errstate(all="ignore"):
        out = a @ b.T
        mag = np.abs(a) @ np.abs(b).T
        if addend is not None:
            out = out + addend
            mag = mag + np.abs(addend)
        e = (a.shape[1] + 1) * 2 * U * mag
        if dtype == "bf16":
            for k in range(0, a.shape[1], 8):
                e += 7 * 2.0 ** -14 * np.max(np.abs(a[:, None, k:k + 8] * b[None, :, k:k + 8]), axis=2)
        return out, e + HALF[dtype] * (np.abs(out) + e) + 2.0 ** -133
