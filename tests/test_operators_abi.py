"""Refusals of the routing and adapter calls (no GPU: every call fails its
checks before any device work, so its pointers are never followed)."""
import ctypes

import pytest

import binary_rank_linear_amd as blr

E_NULL, E_SHAPE, E_WS, E_DEV, E_HIP, E_ALIGN, E_DTYPE, E_OVERLAP = -1, -2, -4, -5, -6, -7, -9, -10
F32, F16, BF16 = 0, 1, 2
BIG = 1 << 50
GAP = 1 << 52  # addresses far enough apart for any size


def at(i, n=0):
    return ctypes.c_void_p((i + 1) * GAP + n)


def call(name, fixed, keys, kw, tail):
    """`name` with the pointers `keys` (in the call's order) standing apart;
    `kw` replaces some: a number is an offset from the place of its own."""
    args = []
    for i, k in enumerate(keys):
        if not isinstance(k, str):
            args.append(k[0])
            continue
        v = kw.get(k, 0)
        args.append(at(i, v) if isinstance(v, int) else v)
    return getattr(blr.load(), name)(*fixed, *args, *tail, None)


def sort(pairs=64, E=8, ws_bytes=BIG, **kw):
    return call("blr_route_sort", (pairs, E), ("ids", "offsets", "order", "slot", "ws"), kw, (ws_bytes,))


def gather(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    return call("blr_route_gather", (T, k, E, d, dtype), ("x", "offsets", "slot", "rows"), kw, ())


def combine(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    return call("blr_route_combine", (T, k, E, d, dtype), ("x", "offsets", "slot", "weights", "rows"), kw, (0,))


def combine_backward(T=4, k=2, E=8, d=128, dtype=F32, **kw):
    return call("blr_route_combine_backward", (T, k, E, d, dtype),
                ("x", "z", "offsets", "slot", "weights", "rows", "dw"), kw, ())


def forward(M=64, d_in=256, d_out=128, r=16, E=4, act=F32, wt=F32, ws_bytes=BIG, **kw):
    return call("blr_adapters_forward", (M, d_in, d_out, r, E, act, wt),
                ("x", "down", "up", "offsets", "order", "scale", "y", (0,), "tape", "ws"), kw, (ws_bytes,))


def backward(M=64, d_in=256, d_out=128, r=16, E=4, act=F32, wt=F32, ws_bytes=BIG, **kw):
    return call("blr_adapters_backward", (M, d_in, d_out, r, E, act, wt),
                ("x", "dy", "down", "up", "offsets", "order", "scale", "tape", "gd", "gu", (0,), "dx", (0,), "ws"), kw,
                (ws_bytes,))


def test_status_string_of_types():
    assert blr.status_string(E_DTYPE) != "unknown status"
    assert blr.status_string(E_OVERLAP) != "unknown status"


def meet(caller, out, other, kw=None):
    """The call with `out` placed on the memory of `other`."""
    return caller(**{**(kw or {}), out: at(0), other: at(0)})


@pytest.mark.parametrize("caller,outs,ins", [
    (sort, ("offsets", "order", "slot"), ("ids",)),
    (gather, ("rows",), ("x", "offsets", "slot")),
    (combine, ("rows",), ("x", "offsets", "slot", "weights")),
    (combine_backward, ("rows", "dw"), ("x", "z", "offsets", "slot", "weights")),
    (forward, ("y", "tape", "ws"), ("x", "down", "up", "offsets", "order", "scale")),
    (backward, ("gd", "gu", "dx", "ws"), ("x", "dy", "down", "up", "offsets", "order", "scale", "tape"))])
def test_outputs_stand_apart(caller, outs, ins):
    for o in outs:
        for other in ins + outs:
            if other != o:
                assert meet(caller, o, other) == E_OVERLAP, (o, other)
    if caller is sort:  # the workspace is one only where it is used
        assert meet(sort, "order", "ws", dict(pairs=8193)) == E_OVERLAP
    # one byte of an input inside the output's end
    assert forward(x=at(20), y=at(20, 64 * 256 * 4 - 16)) == E_OVERLAP


def test_sort_refuses():
    for k in ("ids", "offsets", "order", "slot"):
        assert sort(**{k: None}) == E_NULL, k
        assert sort(**{k: 2}) == E_ALIGN, k
    for pairs, E in [(0, 8), (-1, 8), ((1 << 31) - 65536, 8), (1 << 40, 8), (64, 0), (64, -1), (64, 1025)]:
        assert sort(pairs, E) == E_SHAPE
        assert blr.load().blr_route_workspace_bytes(pairs, E) == 0
    assert sort(pairs=8193, ws=None) == E_WS
    need = blr.load().blr_route_workspace_bytes(8193, 8)
    assert need > 0 and sort(pairs=8193, ws_bytes=need - 1) == E_WS
    assert sort(ws=4) == E_ALIGN


@pytest.mark.parametrize("caller", [gather, combine, combine_backward])
def test_rows_refuse(caller):
    for k in ("x", "offsets", "slot", "rows"):
        assert caller(**{k: None}) == E_NULL, k
    for k in ("x", "rows"):
        assert caller(**{k: 8}) == E_ALIGN, k
    for k in ("offsets", "slot"):
        assert caller(**{k: 2}) == E_ALIGN, k
    for d in (0, -8, 4, 12, 129, (1 << 20) + 8):
        assert caller(d=d) == E_SHAPE, d
    for T, k in [(0, 1), (-1, 1), (1, 0), (1, 1025), (1 << 31, 1), (1 << 62, 4), ((1 << 31) // 512, 1024)]:
        assert caller(T=T, k=k) == E_SHAPE, (T, k)
    assert caller(E=0) == E_SHAPE and caller(E=1025) == E_SHAPE
    for t in (-1, 3):
        assert caller(dtype=t) == E_DTYPE


def test_combine_backward_needs_rows_for_weight_gradients():
    assert combine_backward(z=None) == E_NULL
    assert combine_backward(z=8) == E_ALIGN
    assert combine_backward(dw=2) == E_ALIGN
    assert combine(weights=2) == E_ALIGN


@pytest.mark.parametrize("caller,needed", [(forward, ("x", "down", "up", "offsets", "y")),
                                         (backward, ("dy", "x", "tape", "down", "up", "offsets", "gd", "gu"))])
def test_adapters_refuse(caller, needed):
    for k in needed:
        assert caller(**{k: None}) == E_NULL, k
        assert caller(**{k: 4 if k != "offsets" else 2}) == E_ALIGN, k
    for k in ("order", "scale"):
        assert caller(**{k: 2}) == E_ALIGN, k
    for bad in [dict(M=0), dict(M=-3), dict(M=1 << 31), dict(d_in=0), dict(d_in=64), dict(d_in=200), dict(d_out=130),
                dict(d_out=1 << 21), dict(r=0), dict(r=4), dict(r=12), dict(r=136), dict(E=0), dict(E=1025)]:
        assert caller(**bad) == E_SHAPE, bad
    for act, wt in [(F16, F32), (F16, BF16), (BF16, F16), (BF16, F32), (3, F32), (F32, 3), (-1, F32)]:
        assert caller(act=act, wt=wt) == E_DTYPE, (act, wt)
    need = blr.load().blr_adapters_workspace_bytes(64, 256, 128, 16, 4)
    assert need > 0
    assert caller(ws_bytes=need - 1) == E_WS and caller(ws=None) == E_WS
    assert caller(ws=4) == E_ALIGN


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
    assert sort(pairs=8192, ws=None, ws_bytes=0) in ok
    assert forward(x=at(20), y=at(20, 64 * 256 * 4)) in ok  # end to end
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
    the splits' below 34 copies of s, the transposes take the adapters once, and
    the panels six bytes for each of at most 16 more ranks and E tiles."""
    n = blr.load().blr_adapters_workspace_bytes(M, d_in, d_out, r, E)
    assert 0 < n <= 34 * 4 * M * r + 4 * M * (d_in + d_out) + 4 * E * r * (d_in + d_out) \
        + 2 * 6 * 2 * r * (M + 64 * min(E + 1, M)) + 4096


def test_binding_refuses():
    import torch
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        blr.blr_route_sort(torch.zeros(4, dtype=torch.int32), 4)  # not on a GPU
    with pytest.raises(TypeError):
        blr.blr_route_sort([0, 1], 4)
    with pytest.raises(ValueError):
        blr.blr_adapters_forward(x, x, x, x)
