"""The gated feed-forward where its projections, or products of them, leave
f32's range."""
import numpy as np
import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say

SILU, GELU = 0, 1
M, D, FF = 3, 128, 256


def weights(dev):
    import torch
    return (torch.zeros((FF, D), dtype=torch.bfloat16, device=dev) for _ in range(2))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [SILU, GELU])
def test_an_infinite_gate(dev, kind):
    """A row whose g overflows to minus infinity: act and its slope are 0 there,
    as at every g far below zero; at plus infinity act is g and its slope 1."""
    import torch
    wg, wu = weights(dev)
    wg[:128], wg[128:] = -1.0, 1.0
    wu[:, 0] = 2.0 ** -100
    x = torch.zeros((M, D), dtype=torch.bfloat16, device=dev)
    x[1] = 2.0 ** 127  # g: the sum of 128 of them
    x[2, 0] = 1.0
    say(f"g of minus and plus infinity, kind {kind}")
    h, _ = blr.blr_gated_forward(x, wg, wu, kind=kind, h_dtype=torch.float32)
    assert not bool(h[0].any()) and not bool(h[1, :128].any())
    assert bool((h[1, 128:] == float("inf")).all())
    assert bool(h[2].isfinite().all())
    wg[:] = -1.0
    dh = torch.ones((M, FF), device=dev)
    dx, dwg, dwu = blr.blr_gated_backward(x, dh, wg, wu, kind=kind, grad_dtype=torch.float32)
    assert not bool(dx[1].any())
    assert bool(dx.isfinite().all()) and bool(dwg.isfinite().all()) and bool(dwu.isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
def test_a_product_past_the_range(dev, kept):
    """dg = dh u act'(g) where dh u alone is past f32's largest value: it is in
    range with a slope of e^-60, and 0 with none."""
    import torch
    wg, wu = weights(dev)
    x = torch.zeros((M, D), dtype=torch.bfloat16, device=dev)
    x[1, 0], x[2, 0] = 2.0 ** 126, 2.0 ** 126
    wu[:, 0] = 1.0  # u = 2^126
    wg[:128, 0], wg[128:, 0] = -60 * 2.0 ** -126, -1024 * 2.0 ** -126  # g = -60, -1024
    wg[:, 1] = 1.0  # column 1 of dx: the sum of dg
    dh = torch.zeros((M, FF), device=dev)
    dh[1, :128] = 1024.0
    dh[2, 128:] = 1024.0
    tape = blr.blr_gated_forward(x, wg, wu, keep=True)[1] if kept else None
    say(f"dh u of 2^136, kept {kept}")
    dx = blr.blr_gated_backward(x, dh, wg, wu, tape, grads=False)[0].double().cpu().numpy()
    s = 1 / (1 + np.exp(60.0))
    dg = 1024.0 * 2.0 ** 126 * (s - 60 * s * (1 - s))
    # roundings to bf16: dg, and dx; those of f32 are lost beside them
    assert np.isfinite(dx).all() and not dx[2].any()
    assert abs(dx[1, 1] - 128 * dg) <= 2.01 * 2.0 ** -8 * abs(128 * dg)
