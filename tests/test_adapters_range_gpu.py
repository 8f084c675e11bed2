"""GPU tests of the low-rank adapters on rows of 16 bits whose s or ds spans many
binades, or cancels: every rank takes part with all its bits."""
from __future__ import annotations

import numpy as np
import pytest

import _operators_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import host, say


def num(t):
    return host(t.double())


def wide_case(dev, M, d_in, d_out, r, act, kind, seed):
    """(x, down, up, ids, s): s of 24 bits each, exact in f32, over 30 binades.

    s_j = n 2^(k - 23) with 2^23 <= n < 2^24 comes from three elements of x, of
    8 bits each, so that the sum x down^T is exact in any order. "zeros": of a
    column's ranks only the smaller ones have weights, of 2^-k, so that the
    sum is near one beside ranks up to 2^30 times as large. "cancel": ranks in
    pairs whose s differ by less than 2^-16, with weights of opposite sign."""
    import torch
    rng = np.random.default_rng(seed)
    x, down, up = np.zeros((M, d_in)), np.zeros((2, r, d_in)), np.zeros((2, d_out, r))
    assert d_in >= 3 * r
    k = rng.integers(-5, 25, r)  # of rank j, shared with its partner
    k[1::2] = k[::2]
    n = rng.integers(1 << 23, 1 << 24, (M, r))
    n[:, 1::2] = n[:, ::2] ^ rng.integers(1, 128, (M, r // 2))
    kx = np.clip(k, -14, 8)  # what x holds of the scale; the rest is down's
    for i, shift in enumerate((16, 8, 0)):
        x[:, i:3 * r:3] = (n >> shift & 255) * 2.0 ** kx
        down[:, np.arange(r), 3 * np.arange(r) + i] = 2.0 ** (shift - 23 + k - kx)
    for o in range(d_out):
        w = rng.integers(1, 256, (2, r)) * 2.0 ** (3 - k)
        if kind == "zeros":
            up[:, o] = np.where(k <= rng.integers(-5, 25), w * 2.0 ** -10, 0.0)
        else:
            up[:, o] = np.repeat(w[:, ::2], 2, axis=1) * np.tile([1.0, -1.0], r // 2)
    ids = np.zeros(M, np.int32)
    ids[M // 2] = 1
    put = lambda a: torch.from_numpy(a).to(dev).to(getattr(torch, act))  # noqa: E731
    x, down, up = put(x), put(down), put(up)
    s = np.stack([num(x)[t] @ num(down)[e].T for t, e in enumerate(ids)])
    assert np.array_equal(s, n * 2.0 ** (k - 23.0))  # nothing was lost to the types
    return x, down, up, ids, s


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["zeros", "cancel"])
@pytest.mark.parametrize("r", [8, 16, 24, 64, 104, 128])
@pytest.mark.parametrize("M", [5, 17, 70])
@pytest.mark.parametrize("act", ["float16", "bfloat16"])
def test_small_ranks_beside_large_ones(dev, act, M, r, kind):
    """Forward, and dx by the same numbers (dy as x, up as down^T, down as
    up^T). s is exact, so what is left is the second sum: an element of s
    meets a weight in at most five products, of parts whose absolute values
    add up to at most (1 + 2^-6) of the whole, and what is left out is 2^-25 of
    it: 5 r + 1 roundings, with 2 r for the parts' 2^-6, and the addition to y."""
    import torch
    say(f"adapters, s over 30 binades, M={M} r={r} {act} {kind}")
    d_in, d_out = 384, 256
    x, down, up, ids, s = wide_case(dev, M, d_in, d_out, r, act, kind, seed=M + r)
    W = num(up)
    want = np.stack([W[e] @ s[t] for t, e in enumerate(ids)])
    mag = np.stack([np.abs(W[e]) @ np.abs(s[t]) for t, e in enumerate(ids)])
    offsets, order, _ = blr.blr_route_sort(torch.from_numpy(ids).to(dev), 2)
    y0 = torch.randn((M, d_out), device=dev).to(x.dtype)
    terms = 7 * r + 2

    y, tape = blr.blr_adapters_forward(x, down, up, offsets, order, keep_tape=True)
    assert np.array_equal(num(tape), s)
    ref.within(num(y), want, mag, terms, act)
    y, _ = blr.blr_adapters_forward(x, down, up, offsets, order, y=y0.clone(), accumulate_y=True)
    ref.within(num(y), num(y0) + want, mag + np.abs(num(y0)), terms, act)

    up_t, down_t = down.transpose(1, 2).contiguous(), up.transpose(1, 2).contiguous()
    _, _, dx = blr.blr_adapters_backward(None, x, down_t, up_t, offsets, order, grads=False)
    ref.within(num(dx), want, mag, terms, act)
    gd, gu, dx2 = blr.blr_adapters_backward(y0, x, down_t, up_t, offsets, order, None, tape)
    assert torch.equal(dx2, dx)
    _, _, dx = blr.blr_adapters_backward(None, x, down_t, up_t, offsets, order, grads=False, dx=y0.clone(),
                                         accumulate_dx=True)
    ref.within(num(dx), num(y0) + want, mag + np.abs(num(y0)), terms, act)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("act", ["float16", "bfloat16"])
def test_the_largest_values_stay_finite(dev, act, M):
    """s, ds and the tape at 2^128 - 2^118, past the largest bf16, with other
    factors of 2^-20: results of 2^108 - 2^98, one product each, so exact but
    for the rounding to the output's type."""
    import torch
    say(f"adapters with s past the largest bf16, M={M} {act}")
    t = getattr(torch, act)
    top = 2.0 ** 128 - 2.0 ** 118
    z = lambda *s: torch.zeros(s, dtype=t, device=dev)  # noqa: E731
    # the sum of two products, exact in f32; f16 reaches it by way of the scale
    big = (2.0 ** 127, 2.0 ** 119) if act == "bfloat16" else (2.0 ** 15, 2.0 ** 7)
    scale = torch.tensor([1.0 if act == "bfloat16" else 2.0 ** 112], device=dev)
    a, ends = z(M, 256), z(1, 8, 256)
    a[:, 5], a[:, 9] = big
    ends[0, 2, 5], ends[0, 2, 9] = 255 / 128, 1.5  # 255 2^120 + 1.5 2^119
    other = z(1, 128, 8)
    other[0, :, 2] = 2.0 ** -20
    offsets = torch.tensor([0, M], dtype=torch.int32, device=dev)
    # the gradients take one row (the others' are zero), of x or dy 2^-20
    small = z(M, 128)
    small[M - 1] = 2.0 ** -20
    tape = torch.zeros((M, 8), device=dev)
    tape[M - 1, 2] = top
    down, up = other.transpose(1, 2).contiguous(), ends.transpose(1, 2).contiguous()
    gd, _, dx = blr.blr_adapters_backward(small, a, down, up, offsets, None, scale, tape)
    _, gu, _ = blr.blr_adapters_backward(a, small, ends, other, offsets, None, None, tape)
    assert (num(gd)[0, 2] == top * 2.0 ** -20).all() and not num(gd)[0, 3].any()
    assert (num(gu)[0, :, 2] == top * 2.0 ** -20).all() and not num(gu)[0, :, 3].any()
    if act == "bfloat16":
        y, s = blr.blr_adapters_forward(a, ends, other, offsets, keep_tape=True)
        assert (num(s)[:, 2] == top).all()
        assert (num(y) == 2.0 ** 108).all() and (num(dx) == 2.0 ** 108).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act,d_in,r", [("float32", 65536, 24), ("float16", 131072, 8), ("bfloat16", 131072, 72)])
def test_gradients_of_an_x_past_the_caches(dev, act, d_in, r):
    """x of over 64 MB, which its gradient reads without keeping it, against the
    formula in 64 bits: 3 products a row and a term for the roundings of ds."""
    import torch
    say(f"adapters, 300 rows of {d_in}, {act}, rank {r}")
    M, d_out, E = 300, 128, 3
    t = getattr(torch, act)
    torch.manual_seed(r)
    ids = torch.randint(-1, E, (M,), device=dev).int()
    x, dy = torch.randn((M, d_in), device=dev).to(t), torch.randn((M, d_out), device=dev).to(t)
    down, up = torch.randn((E, r, d_in), device=dev).to(t), torch.randn((E, d_out, r), device=dev).to(t)
    tape = torch.randn((M, r), device=dev)
    offsets, order, _ = blr.blr_route_sort(ids, E)
    gd, _, none = blr.blr_adapters_backward(x, dy, down, up, offsets, order, None, tape, need_dx=False)
    assert none is None
    for e in range(E):
        at = torch.nonzero(ids == e).flatten()
        dys, xs, B = dy[at].double(), x[at].double(), up[e].double()
        want, mag = (dys @ B).T @ xs, (dys.abs() @ B.abs()).T @ xs.abs()
        ref.within(num(gd[e]), host(want), host(mag), 3 * len(at) + d_out + 4)
