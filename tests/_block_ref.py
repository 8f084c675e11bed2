"""Plain 64-bit forms of the norms, the gated feed-forward and the 8-bit
checkpoints (not a test module). Functions that return a pair give the value
and the sum of its absolute terms, for `_operators_ref.within`."""
from __future__ import annotations

import math

import numpy as np

MOST = {"float32": 254, "float16": 142, "bfloat16": 254}  # a type's widest step


def pack(x, dtype):
    """(q, b) of rows x [M][d], by the definition: the least step 2^(b - 133)
    of which the block's largest value rounds to at most 127."""
    v = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, 32)
    q, b = np.zeros(v.shape, np.int8), np.zeros(v.shape[:2], np.uint8)
    for t in range(v.shape[0]):
        for j in range(v.shape[1]):
            block = v[t, j]
            if not np.isfinite(block).all():
                b[t, j] = 255
                continue
            top = float(np.abs(block).max())
            e = max(0, (math.frexp(top)[1] - 7 if top else -133) + 133 - 2)
            while e < MOST[dtype] and np.rint(math.ldexp(top, 133 - e)) > 127:
                e += 1
            b[t, j] = e
            q[t, j] = np.clip(np.rint(np.ldexp(block, 133 - e)), -127, 127)
    return q.reshape(x.shape), b


def unpack(q, b):
    e = np.repeat(np.asarray(b).astype(np.int64), 32, axis=-1)
    return np.where(e == 255, np.nan, np.ldexp(np.asarray(q).astype(np.float64), e - 133))


def phi(kind, z):
    """(phi(z), slope, the slope's terms); kind 0 linear, 1 sigmoid, 2 silu.
    silu's slope s + z s (1 - s) is a sum of two roundings' worth of terms that
    cancel near z = -1.28: an f32 result is off by so many 2^-24 of |s| +
    |z s (1 - s)|, not of what is left of them."""
    if kind == 0:
        return z, np.ones_like(z), np.ones_like(z)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    if kind == 1:
        return s, s * (1 - s), s * (1 - s)
    return z * s, s + z * s * (1 - s), s + np.abs(z * s * (1 - s))


def norm_after(x, f, c):
    """(out, its terms, rstd_f) of the stream x after a block's f."""
    rf = np.ones(len(f))
    if c["norm_f"]:
        rf = 1 / np.sqrt((f * f).mean(1) + c["eps"])
    v = f * rf[:, None] * (1.0 if c["w_after"] is None else c["w_after"])
    if c["gate"] is not None:
        v = v * np.repeat(phi(c["kind"], c["gate"])[0], c["span"], axis=0)[:len(f)]
    return c["skip"] * x + c["scale"] * v, np.abs(c["skip"] * x) + np.abs(c["scale"] * v), rf


def norm_before(out, w, eps):
    r = 1 / np.sqrt((out * out).mean(1) + eps)
    return out * r[:, None] * (1.0 if w is None else w), r


def norm_backward(dn, dout, out, f, stats, c):
    """{name: (value, terms)} of every gradient; dn, dout, f may be None."""
    M, d = (dn if dn is not None else dout).shape
    zero = np.zeros((M, d))
    dO, mO = (zero, zero) if dout is None else (dout, np.abs(dout))
    got = {}
    if dn is not None:
        w = 1.0 if c["w"] is None else c["w"]
        r = stats[0][:, None]
        hat, u = out * r, w * dn
        dO = dO + r * (u - hat * (u * hat).mean(1, keepdims=True))
        mO = mO + r * (np.abs(u) + np.abs(hat) * np.abs(u * hat).mean(1, keepdims=True))
        got["dw"] = ((dn * hat).sum(0), np.abs(dn * hat).sum(0))
    if not c["has_f"]:
        got["dx"] = (dO, mO)
        return got
    got["dx"] = (c["skip"] * dO, abs(c["skip"]) * mO)
    ph, sl, ms = np.ones((M, d)), zero, zero
    if c["gate"] is not None:
        ph, sl, ms = (np.repeat(t, c["span"], axis=0)[:M] for t in phi(c["kind"], c["gate"]))
    wa = 1.0 if c["w_after"] is None else c["w_after"]
    p, mp = c["scale"] * ph * dO, np.abs(c["scale"] * ph) * mO
    hat = zero if f is None else f * (stats[1][:, None] if c["norm_f"] else 1.0)
    if c["norm_f"]:
        rf = stats[1][:, None]
        got["df"] = (rf * (wa * p - hat * (wa * p * hat).mean(1, keepdims=True)),
                     rf * (np.abs(wa) * mp + np.abs(hat) * (np.abs(wa * hat) * mp).mean(1, keepdims=True)))
    else:
        got["df"] = (wa * p, np.abs(wa) * mp)
    got["dw_after"] = ((p * hat).sum(0), (mp * np.abs(hat)).sum(0))
    if c["gate"] is not None:
        dz, mz = c["scale"] * sl * wa * hat * dO, np.abs(c["scale"] * ms * wa * hat) * mO
        if c["span"] > 1:
            cut = range(0, M, c["span"])
            dz, mz = (np.add.reduceat(t, list(cut), axis=0) for t in (dz, mz))
        got["dgate"] = (dz, mz)
    return got


def act(kind, g):
    """(act(g), its slope, the terms of both): silu, or gelu by tanh, as
    g sigmoid(y) with y = g or 2 sqrt(2 / pi) (g + 0.044715 g^3). The slope is
    s + g y' s (1 - s), whose terms cancel at act's least value; an f32 y is off
    by a few 2^-24 of itself, which moves act by |g y s (1 - s)| of them, and
    its slope by at most |y| (1 + |g y'|) s (1 - s)."""
    y, dy = g, np.ones_like(g)
    if kind == 1:
        c = 2 * math.sqrt(2 / math.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    with np.errstate(over="ignore", under="ignore"):
        e = np.exp(-np.abs(y))
    big, small = 1 / (1 + e), e / (1 + e)
    s, r = np.where(y >= 0, big, small), big * small
    with np.errstate(over="ignore", invalid="ignore"):
        second = np.where(r == 0, 0.0, g * dy * r)
        moved = np.where(r == 0, 0.0, np.abs(y) * r)
    return g * s, s + second, np.abs(g * s) + np.abs(g) * moved, s + np.abs(second) + moved * (1 + np.abs(g * dy))
