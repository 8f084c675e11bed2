"""The gated feed-forward where its projections leave f32's range."""
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
