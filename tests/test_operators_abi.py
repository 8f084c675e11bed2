"""Refusals of the routing and adapter calls (no GPU: every call fails its
checks before any device work, so its pointers are never followed)."""
import ctypes

import numpy as np
import pytest

import binary_rank_linear_amd as blr

E_NULL, E_SHAPE, E_WS, E_DEV, E_HIP, E_ALIGN, E_DTYPE = -1, -2, -4, -5, -6, -7, -9
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 50
_keep = np.zeros(4096, np.uint8)
P = ctypes.c_void_p((_keep.ctypes.data + 15) // 16 * 16)


def off(n):
    return ctypes.c_void_p(P.value + n)


def sort(pairs=64, E=8, ws_bytes=BIG, **kw):
    a = dict(ids=P, offsets=P, order=P, slot=P, ws=P, **{})
    a.update(kw)
    return blr.load().blr_route_sort(pairs, E, a["ids"], a["offsets"], a["order"], a["slot"], a["ws"], ws_bytes, None)


def gather(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    a = dict(x=P, offsets=P, slot=P, rows=P)
    a.update(kw)
    return blr.load().blr_route_gather(T, k, E, d, dtype, a["x"], a["offsets"], a["slot"], a["rows"], None)


def combine(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    a = dict(x=P, offsets=P, slot=P, weights=P, rows=P)
    a.update(kw)
    return blr.load().blr_route_combine(T, k, E, d, dtype, a["x"], a["offsets"], a["slot"], a["weights"], a["rows"],
                                        0, None)


def combine_backward(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    a = dict(x=P, z=P, offsets=P, slot=P, weights=P, rows=P, dw=P)
    a.update(kw)
    return blr.load().blr_route_combine_backward(T, k, E, d, dtype, a["x"], a["z"], a["offsets"], a["slot"],
                                                 a["weights"], a["rows"], a["dw"], None)


def forward(M=64, d_in=256, d_out=128, r=16, E=4, act=F32, wt=F32, ws_bytes=BIG, **kw):
    a = dict(x=P, down=P, up=P, offsets=P, order=P, scale=P, y=P, tape=P, ws=P)
    a.update(kw)
    return blr.load().blr_adapters_forward(M, d_in, d_out, r, E, act, wt, a["x"], a["down"], a["up"], a["offsets"],
                                           a["order"], a["scale"], a["y"], 0, a["tape"], a["ws"], ws_bytes, None)


def backward(M=64, d_in=256, d_out=128, r=16, E=4, act=F32, wt=F32, ws_bytes=BIG, **kw):
    a = dict(x=P, dy=P, down=P, up=P, offsets=P, order=P, scale=P, tape=P, gd=P, gu=P, dx=P, ws=P)
    a.update(kw)
    return blr.load().blr_adapters_backward(M, d_in, d_out, r, E, act, wt, a["x"], a["dy"], a["down"], a["up"],
                                            a["offsets"], a["order"], a["scale"], a["tape"], a["gd"], a["gu"], 0,
                                            a["dx"], 0, a["ws"], ws_bytes, None)


def test_status_string_of_types():
    assert blr.status_string(E_DTYPE) != "unknown status"


def test_sort_refuses():
    for k in ("ids", "offsets", "order", "slot"):
        assert sort(**{k: None}) == E_NULL, k
        assert sort(**{k: off(2)}) == E_ALIGN, k
    for pairs, E in [(0, 8), (-1, 8), ((1 << 31) - 65536, 8), (1 << 40, 8), (64, 0), (64, -1), (64, 1025)]:
        assert sort(pairs, E) == E_SHAPE
        assert blr.load().blr_route_workspace_bytes(pairs, E) == 0
    assert sort(ws=None) == E_WS
    need = blr.load().blr_route_workspace_bytes(64, 8)
    assert need > 0 and sort(ws_bytes=need - 1) == E_WS
    assert sort(ws=off(4)) == E_ALIGN


@pytest.mark.parametrize("call", [gather, combine, combine_backward])
def test_rows_refuse(call):
    for k in ("x", "offsets", "slot", "rows"):
        assert call(**{k: None}) == E_NULL, k
    for k in ("x", "rows"):
        assert call(**{k: off(8)}) == E_ALIGN, k
    for k in ("offsets", "slot"):
        assert call(**{k: off(2)}) == E_ALIGN, k
    for d in (0, -8, 4, 12, 129, (1 << 20) + 8):
        assert call(d=d) == E_SHAPE, d
    for T, k in [(0, 1), (-1, 1), (1, 0), (1, 1025), (1 << 31, 1), (1 << 62, 4), ((1 << 31) // 512, 1024)]:
        assert call(T=T, k=k) == E_SHAPE, (T, k)
    assert call(E=0) == E_SHAPE and call(E=1025) == E_SHAPE
    for t in (-1, 3):
        assert call(dtype=t) == E_DTYPE


def test_combine_backward_needs_rows_for_weight_gradients():
    assert combine_backward(z=None) == E_NULL
    assert combine_backward(z=off(8)) == E_ALIGN
    assert combine_backward(dw=off(2)) == E_ALIGN
    assert combine(weights=off(2)) == E_ALIGN


@pytest.mark.parametrize("call,needed", [(forward, ("x", "down", "up", "offsets", "y")),
                                         (backward, ("dy", "x", "tape", "down", "up", "offsets", "gd", "gu"))])
def test_adapters_refuse(call, needed):
    for k in needed:
        assert call(**{k: None}) == E_NULL, k
        assert call(**{k: off(4 if k != "offsets" else 2)}) == E_ALIGN, k
    for k in ("order", "scale"):
        assert call(**{k: off(2)}) == E_ALIGN, k
    for bad in [dict(M=0), dict(M=-3), dict(M=1 << 31), dict(d_in=0), dict(d_in=64), dict(d_in=200), dict(d_out=130),
                dict(d_out=1 << 21), dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(E=0), dict(E=1025)]:
        assert call(**bad) == E_SHAPE, bad
    for act, wt in [(F16, F32), (F16, BF16), (BF16, F16), (BF16, F32), (3, F32), (F32, 3), (-1, F32)]:
        assert call(act=act, wt=wt) == E_DTYPE, (act, wt)
    need = blr.load().blr_adapters_workspace_bytes(64, 256, 128, 16, 4)
    assert need > 0
    assert call(ws_bytes=need - 1) == E_WS and call(ws=None) == E_WS
    assert call(ws=off(4)) == E_ALIGN


def test_adapters_backward_needs_an_output():
    assert backward(gd=None, gu=None, dx=None) == E_NULL


def test_accepted_sizes_reach_the_device():
    """On a machine without a GPU the edge sizes fail at the device check, not
    at the sizes'."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    ok = (E_DEV, E_HIP)
    assert sort(pairs=(1 << 31) - 65537, E=1024) in ok
    assert gather(T=1, k=1024, E=1, d=8, dtype=BF16) in ok
    assert combine(weights=None) in ok
    assert combine_backward(z=None, dw=None) in ok
    for act, wt in [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)]:
        assert forward(M=1, d_in=128, d_out=1 << 20, r=8, E=1024, act=act, wt=wt, order=None, scale=None,
                       tape=None) in ok
        assert backward(r=128, act=act, wt=wt, dx=None) in ok
        assert backward(act=act, wt=wt, gd=None, gu=None, x=None, tape=None) in ok


@pytest.mark.parametrize("M,d_in,d_out,r,E", [(1, 128, 128, 8, 1), (8192, 4096, 4096, 16, 8),
                                             (30000, 5120, 17408, 64, 16), (100000, 128, 1 << 20, 128, 1024)])
def test_adapter_workspace_stays_in_proportion(M, d_in, d_out, r, E):
    """The gradients' partials stay below the activations that the call reads,
    and the splits' below 34 copies of s."""
    n = blr.load().blr_adapters_workspace_bytes(M, d_in, d_out, r, E)
    assert 0 < n <= 34 * 4 * M * r + 4 * M * max(d_in, d_out) + 4096


def test_binding_refuses():
    import torch
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        blr.blr_route_sort(torch.zeros(4, dtype=torch.int32), 4)  # not on a GPU
    with pytest.raises(TypeError):
        blr.blr_route_sort([0, 1], 4)
    with pytest.raises(ValueError):
        blr.blr_adapters_forward(x, x, x, x)
