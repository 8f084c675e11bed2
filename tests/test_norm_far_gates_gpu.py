"""Gates at plus and minus infinity: phi and its slope are what they tend to."""
import numpy as np
import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say

# phi and slope at -inf and at +inf: sigmoid, silu
ENDS = {1: ((0.0, 0.0), (1.0, 0.0)), 2: ((0.0, 0.0), (np.inf, 1.0))}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [1, 2])
@pytest.mark.parametrize("span", [1, 2])
def test_infinite_gates(dev, kind, span):
    """out = x + phi(z) f, df = phi(z) dout, dgate = phi'(z) f dout: exact, since
    a product with 0 or 1 is (and with infinity, of the product's sign)."""
    import torch
    g = torch.Generator(device=dev).manual_seed(5)
    M, d = 4, 72
    x, f, dout = (torch.randn((M, d), generator=g, device=dev) for _ in range(3))
    gate = torch.empty((M // span, d), device=dev)
    gate[0], gate[-1] = -float("inf"), float("inf")
    if span == 1:
        gate[1], gate[2] = -float("inf"), float("inf")
    how = dict(gate=gate, gate_kind=kind, span=span)
    say(f"infinite gates, kind {kind}, span {span}")
    out, _, _, _ = blr.blr_norm_forward(x, f, **how)
    _, df, dgate, _, _ = blr.blr_norm_backward(None, dout, None, f, None, None, **how)
    half = M // 2
    for rows, (phi, slope) in zip((slice(0, half), slice(half, M)), ENDS[kind]):
        assert torch.equal(out[rows], x[rows] + phi * f[rows])
        assert torch.equal(df[rows], phi * dout[rows])
        want = slope * f[rows] * dout[rows]
        if span == 1:
            assert torch.equal(dgate[rows], want)
        else:  # a product may enter the sum unrounded: two products' and a sum's half steps
            got = dgate[0 if rows.start == 0 else 1].double()
            assert bool(((got - want.double().sum(0)).abs() <= 2.0 ** -23 * want.double().abs().sum(0)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [1, 2])
def test_a_gate_that_is_not_a_number(dev, kind):
    """NaN in a gate stays NaN, in its own place."""
    import torch
    x, f = torch.ones((3, 64), device=dev), torch.ones((3, 64), device=dev)
    gate = torch.zeros((3, 64), device=dev)
    gate[1, 7] = float("nan")
    say(f"a NaN gate, kind {kind}")
    out, _, _, _ = blr.blr_norm_forward(x, f, gate=gate, gate_kind=kind)
    _, df, dgate, _, _ = blr.blr_norm_backward(None, x, None, f, None, None, gate=gate, gate_kind=kind)
    for t in (out, df, dgate):
        assert int(t.isnan().sum()) == 1 and bool(t[1, 7].isnan())
