"""Numbers that C's types do not hold are refused by the binding, before its
tensors are looked at (no GPU: ctypes would cut them to their low bits, and a
span of 2^64 + 1 would have a gate of one row read as a gate for every row)."""
import pytest

import binary_rank_linear_amd as blr

E_SHAPE, E_DTYPE = -2, -9


@pytest.mark.parametrize("span", [0, -1, 1 << 63, (1 << 64) + 1, 1 << 200])
def test_span(span):
    import torch
    x = torch.zeros((4, 64))
    for f in (lambda: blr.blr_norm_forward(x, x, gate=x[:1], span=span),
              lambda: blr.blr_norm_backward(x, x, x, x, gate=x[:1], span=span),
              lambda: blr.workspace_norm(4, 64, span)):
        with pytest.raises(blr.BlrError) as e:
            f()
        assert e.value.status == E_SHAPE


@pytest.mark.parametrize("kind", [-1, 3, 1 << 32, (1 << 32) + 1])
def test_kinds(kind):
    import torch
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    for f in (lambda: blr.blr_norm_forward(x, x, gate=x, gate_kind=kind),
              lambda: blr.blr_norm_backward(x, x, x, x, gate=x, gate_kind=kind),
              lambda: blr.blr_gated_forward(x, x, x, kind=kind), lambda: blr.blr_gated_backward(x, x, x, x, kind=kind)):
        with pytest.raises(blr.BlrError) as e:
            f()
        assert e.value.status == E_DTYPE
