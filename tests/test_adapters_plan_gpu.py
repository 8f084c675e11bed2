"""GPU tests of the adapters on plans whose offsets are extreme."""
from __future__ import annotations

import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["float32", "bfloat16"])
def test_offsets_are_taken_inside_the_plan(dev, act):
    """Offsets outside [0, M] count as its nearer end, and a group whose end
    comes before its start has no rows: the outputs are those of the plan that
    this leaves. The first group's end lies 2^31 and more below its start."""
    import torch
    say(f"adapters with extreme offsets, {act}")
    M, d_in, d_out, r, E = 150, 256, 128, 16, 4
    torch.manual_seed(0)
    rn = lambda *s: torch.randn(s, device=dev).to(getattr(torch, act))  # noqa: E731
    x, dy, down, up = rn(M, d_in), rn(M, d_out), rn(E, r, d_in), rn(E, d_out, r)
    order = torch.randperm(M, device=dev).int()
    scale = torch.rand(E, device=dev)

    def run(*offsets):
        o = torch.tensor(offsets, dtype=torch.int64).to(torch.int32).to(dev)
        y, tape = blr.blr_adapters_forward(x, down, up, o, order, scale, keep_tape=True)
        return (y, tape) + blr.blr_adapters_backward(x, dy, down, up, o, order, scale, tape)

    low, high = -2 ** 31, 2 ** 31 - 1
    want = run(0, 0, 64, 64, M)
    for bad in ([M, low, 64, 64, high], [high, low, 64, 64, M], [high, -1, 64, 64, M + 1], [low, low, 64, 64, high]):
        assert all(torch.equal(a, b) for a, b in zip(run(*bad), want)), bad
