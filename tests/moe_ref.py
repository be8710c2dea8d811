"""Plain NumPy references of the expert layer's operators, in 64 bits, and the error bounds their float32 arithmetic
allows (U and HALF as in ops_ref: half a step, relative)."""

import numpy as np

import ops_ref as R


def rows_for(tokens, top_k, experts, align):
    slots = tokens * top_k
    n = slots + min(slots, experts) * (align - 1)
    return n if align < 32 else -(-n // 128) * 128


def sort(ids, experts, align, rows):
    """offsets, place, source, slot by slot."""
    flat = [int(i) for i in np.asarray(ids).reshape(-1)]
    members = [[s for s, e in enumerate(flat) if e == x] for x in range(experts)] if experts < 8 else None
    if members is None:
        members = [[] for _ in range(experts)]
        for s, e in enumerate(flat):
            if 0 <= e < experts:
                members[e].append(s)
    offsets, place, source = [0], [-1] * len(flat), [-1] * rows
    for m in members:
        at = offsets[-1]
        for i, s in enumerate(m):
            place[s], source[at + i] = at + i, s
        offsets.append(at + -(-len(m) // align) * align)
    return np.array(offsets, np.int32), np.array(place, np.int32), np.array(source, np.int32)


def gather(x, weights, source, offsets, top_k):
    """Float32 rows, correctly rounded products, and which rows are in use."""
    source = np.asarray(source)
    y = np.zeros((source.size, x.shape[1]), np.float32)
    slots = x.shape[0] * top_k
    for p in range(int(offsets[-1])):
        s = source[p]
        if 0 <= s < slots:
            w = 1.0 if weights is None else float(weights.reshape(-1)[s])
            with np.errstate(all="ignore"):
                y[p] = (x[s // top_k].astype(np.float64) * w).astype(np.float32)
    return y


def combine(y, place, weights, residual, top_k, dtype):
    """out and its bound: a fused multiply-add a choice and the residual's sum, a rounding each of a partial sum no
    larger than the terms' magnitudes, then the result's own."""
    place = np.asarray(place).reshape(-1, top_k)
    out = np.zeros((place.shape[0], y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(place.shape[0]):
        for j in range(top_k):
            p = place[t, j]
            if 0 <= p < y.shape[0]:
                v = y[p].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
                out[t] += v
                mag[t] += np.abs(v)
    if residual is not None:
        out += residual
        mag += np.abs(residual)
    e = (top_k + 1) * R.U * (1 + 1e-6) * mag
    return out, e + R.HALF[dtype] * (np.abs(out) + e) + 2.0 ** -133


def dweights(dout, y, place, top_k):
    """A lane adds its columns' products in a chain of cols / 64 (at least 8), then six sums of lanes."""
    place = np.asarray(place).reshape(-1, top_k)
    out, mag = np.zeros(place.shape), np.zeros(place.shape)
    for t in range(place.shape[0]):
        for j in range(top_k):
            p = place[t, j]
            if 0 <= p < y.shape[0]:
                v = dout[t].astype(np.float64) * y[p].astype(np.float64)
                out[t, j], mag[t, j] = v.sum(), np.abs(v).sum()
    chain = -(-y.shape[1] // 512) * 8 + 6
    return out, chain * R.U * (1 + 1e-6) * mag + 2.0 ** -149
