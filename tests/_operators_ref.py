"""Plain 64-bit forms of the routing and the low-rank adapters, and the bounds
their tests use (not a test module)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of f32, relative to the value
# half a step of each output type, and its smallest subnormal (below it a rounding is absolute)
HALF = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -24, "bfloat16": 2.0 ** -133}


def sort(ids, E):
    """(offsets, order, slot): a stable sort by id, ids outside [0, E) last."""
    flat = np.asarray(ids).reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    slot = np.empty_like(order)
    slot[order] = np.arange(flat.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    return offsets.astype(np.int32), order.astype(np.int32), slot.reshape(np.shape(ids)).astype(np.int32)


def gather(x, offsets, slot):
    T = x.shape[0]
    slot = slot.reshape(T, -1)
    rows = np.zeros((slot.size, x.shape[1]))
    for t in range(T):
        for at in slot[t]:
            if at < offsets[-1]:
                rows[at] = x[t]
    return rows


def combine(z, offsets, slot, weights=None):
    """(y, the sum of the absolute terms)."""
    T = slot.shape[0]
    slot = slot.reshape(T, -1)
    y, mag = np.zeros((T, z.shape[1])), np.zeros((T, z.shape[1]))
    for t in range(T):
        for j, at in enumerate(slot[t]):
            if at < offsets[-1]:
                v = (1.0 if weights is None else float(weights[t, j])) * z[at]
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def combine_backward(dy, z, offsets, slot, weights=None):
    """(dz, dw, the sum of dw's absolute terms)."""
    T, k = slot.reshape(dy.shape[0], -1).shape
    slot = slot.reshape(T, k)
    dz = np.zeros((T * k, dy.shape[1]))
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j, at in enumerate(slot[t]):
            if at < offsets[-1]:
                dz[at] = (1.0 if weights is None else float(weights[t, j])) * dy[t]
                if z is not None:
                    dw[t, j] = dy[t] @ z[at]
                    mag[t, j] = np.abs(dy[t]) @ np.abs(z[at])
    return dz, dw, mag


def adapters_forward(x, down, up, ids, scale):
    """((s, y), their sums of absolute terms): y without what it is added to."""
    M, (E, r, _), d_out = x.shape[0], down.shape, up.shape[1]
    s, y = np.zeros((M, r)), np.zeros((M, d_out))
    sm, ym = np.zeros((M, r)), np.zeros((M, d_out))
    for e in range(E):
        m = np.nonzero(ids == e)[0]
        if m.size:
            c = 1.0 if scale is None else float(scale[e])
            s[m] = x[m] @ down[e].T
            sm[m] = np.abs(x[m]) @ np.abs(down[e]).T
            y[m] = c * (s[m] @ up[e].T)
            ym[m] = abs(c) * (sm[m] @ np.abs(up[e]).T)
    return (s, y), (sm, ym)


def adapters_backward(x, dy, down, up, ids, scale, s):
    """((grad_down, grad_up, dx), their sums of absolute terms); s is the tape."""
    E = down.shape[0]
    got = [np.zeros(down.shape), np.zeros(up.shape), np.zeros(x.shape)]
    mag = [np.zeros(down.shape), np.zeros(up.shape), np.zeros(x.shape)]
    for e in range(E):
        m = np.nonzero(ids == e)[0]
        if m.size:
            c = 1.0 if scale is None else float(scale[e])
            ds, dm = c * (dy[m] @ up[e]), abs(c) * (np.abs(dy[m]) @ np.abs(up[e]))
            got[0][e], mag[0][e] = ds.T @ x[m], dm.T @ np.abs(x[m])
            got[1][e], mag[1][e] = c * (dy[m].T @ s[m]), abs(c) * (np.abs(dy[m]).T @ np.abs(s[m]))
            got[2][m], mag[2][m] = ds @ down[e], dm @ np.abs(down[e])
    return got, mag


def within(got, want, mag, terms, dtype="float32"):
    """Every element of got within its bound of want. A sum of n products in
    f32, in any order, is off by at most n U (1 + n U) times the sum of their
    absolute values: each product is rounded once and passes at most n - 1
    additions. `terms` counts the roundings of the whole chain (a sum inside a
    sum: both); one rounding to the output's type is added."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape
    bound = terms * U * (1 + terms * U) * mag + (1 + terms * U) * HALF[dtype] * np.abs(want) + TINY[dtype]
    off = np.abs(got - want)
    bad = ~(off <= bound)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, off / np.maximum(bound, 1e-300), 0)), got.shape)
        raise AssertionError(f"{int(bad.sum())} of {bad.size} elements out of bound; worst at {at}: got {got[at]!r}, "
                             f"want {want[at]!r}, bound {bound[at]:.3g}")
