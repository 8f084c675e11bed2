"""Refusals of the norms', checkpoints' and gated feed-forward's calls (no GPU: every call fails its
checks before any device work, so its pointers are never followed)."""
import ctypes

import pytest

import binary_rank_linear_amd as blr
from test_operators_abi import BF16, BIG, E_ALIGN, E_DEV, E_DTYPE, E_HIP, E_NULL, E_OVERLAP, E_SHAPE, E_WS, F16, F32, at

NO_GPU = (E_DEV, E_HIP)  # what a call that passes every check meets on a machine without a GPU


def f32(v):
    return ctypes.c_float(v)


def call(name, args, keys, kw):
    """`name` with args in order; an entry of `keys` is a pointer's name, which
    stands at an address of its own unless kw places it (a number: that many
    bytes further)."""
    place = {k: i for i, k in enumerate(keys)}
    out = []
    for a in args:
        if isinstance(a, str):
            v = kw.get(a, 0)
            a = at(place[a], v) if isinstance(v, int) else v
        out.append(a)
    assert not set(kw) - set(place), set(kw) - set(place)
    return getattr(blr.load(), name)(*out, None)


def save(M=4, d=64, dtype=F32, **kw):
    return call("blr_checkpoint_save", (M, d, dtype, "x", "q", "b"), ("x", "q", "b"), kw)


def load(M=4, d=64, dtype=F32, **kw):
    return call("blr_checkpoint_load", (M, d, dtype, "q", "b", "x"), ("x", "q", "b"), kw)


FWD = ("x", "f", "w_after", "gate", "w", "out", "n", "stats", "q", "b")
BWD = ("dn", "dout", "out", "out_q", "out_b", "f", "f_q", "f_b", "w_after", "gate", "w", "stats", "dx", "df", "dgate",
       "dw", "dw_after", "ws")
ROWS = dict(out_q=None, out_b=None, f_q=None, f_b=None)  # out and f as rows


def forward(M=4, d=64, xt=F32, ft=F32, nt=F32, norm_f=1, kind=0, span=1, **kw):
    return call("blr_norm_forward", (M, d, xt, ft, nt, "x", "f", norm_f, "w_after", "gate", kind, span, f32(1), f32(1),
                                     "w", f32(1e-6), "out", "n", "stats", "q", "b"), FWD, kw)


def backward(M=4, d=64, xt=F32, ft=F32, nt=F32, has_f=1, norm_f=1, kind=0, span=1, ws_bytes=BIG, **kw):
    kw = {**ROWS, **kw}
    return call("blr_norm_backward",
                (M, d, xt, ft, nt, "dn", "dout", "out", "out_q", "out_b", has_f, "f", "f_q", "f_b", norm_f, "w_after",
                 "gate", kind, span, f32(1), f32(1), "w", "stats", "dx", "df", "dgate", "dw", "dw_after", 0, "ws",
                 ws_bytes), BWD, kw)


@pytest.mark.parametrize("caller,outs", [(save, ("q", "b")), (load, ("x",))])
def test_checkpoint_refuses(caller, outs):
    assert caller() in NO_GPU
    for k in ("x", "q", "b"):
        assert caller(**{k: None}) == E_NULL, k
    for k in ("x", "q"):
        assert caller(**{k: 8}) == E_ALIGN, k
    for dtype in (-1, 3):
        assert caller(dtype=dtype) == E_DTYPE
    for M, d in [(0, 64), (-1, 64), ((1 << 31) - 65536, 64), (4, 0), (4, -32), (4, 16), (4, 48), (4, (1 << 20) + 32)]:
        assert caller(M, d) == E_SHAPE, (M, d)
    for o in outs:
        for other in ("x", "q", "b"):
            if o != other:
                assert caller(**{o: at(0), other: at(0)}) == E_OVERLAP, (o, other)


def test_norm_forward_refuses():
    assert forward() in NO_GPU
    for types in [(F16, F32, F16), (F16, F16, F32), (BF16, F16, BF16), (F32, 3, F32), (-1, F32, F32)]:
        assert forward(xt=types[0], ft=types[1], nt=types[2]) == E_DTYPE, types
    for ft in (F32, F16, BF16):
        for nt in (F32, F16, BF16):
            assert forward(ft=ft, nt=nt) in NO_GPU
    for kind in (-1, 3):
        assert forward(kind=kind) == E_DTYPE
    for M, d, span in [(0, 64, 1), ((1 << 31) - 65536, 64, 1), (4, 0, 1), (4, 4, 1), (4, 68, 1), (4, 16392, 1),
                       (4, 64, 0), (4, 64, -1)]:
        assert forward(M, d, span=span) == E_SHAPE, (M, d, span)
    assert forward(d=40) == E_SHAPE and forward(d=40, q=None, b=None) in NO_GPU  # a checkpoint's blocks are of 32
    for kw in (dict(x=None), dict(f=None), dict(out=None), dict(q=None), dict(b=None),
               dict(f=None, out=None, n=None, stats=None, q=None, b=None)):
        assert forward(**kw) == E_NULL, kw
    assert forward(f=None, out=None) in NO_GPU
    assert forward(span=1 << 62) in NO_GPU
    for k in ("x", "f", "gate", "w_after", "w", "out", "n", "q"):
        assert forward(**{k: 8}) == E_ALIGN, k
    assert forward(stats=2) == E_ALIGN
    outs = ("out", "n", "stats", "q", "b")
    for o in outs:
        for other in FWD:
            if o != other:
                assert forward(**{o: at(0), other: at(0)}) == E_OVERLAP, (o, other)


def test_norm_backward_refuses():
    kept = dict(out=None, f=None, out_q=0, out_b=0, f_q=0, f_b=0)
    assert backward() in NO_GPU and backward(**kept) in NO_GPU
    for types in [(F16, F32, F16), (F16, F16, F32), (BF16, F16, BF16), (F32, 3, F32)]:
        assert backward(xt=types[0], ft=types[1], nt=types[2]) == E_DTYPE, types
    assert backward(kind=3) == E_DTYPE
    for M, d, span in [(0, 64, 1), (4, 12, 1), (4, 16392, 1), (4, 64, 0)]:
        assert backward(M, d, span=span) == E_SHAPE
        assert blr.load().blr_norm_workspace_bytes(M, d, span) == 0
    assert backward(d=40) in NO_GPU and backward(d=40, **kept) == E_SHAPE
    for kw in (dict(dn=None, dout=None), dict(out=None), dict(f=None), dict(stats=None), dict(dn=None),  # dw needs dn
               dict(gate=None), dict(out_q=0, out_b=0), dict(f_q=0, f_b=0), dict(out=None, out_q=0),
               dict(f=None, f_b=0), dict(dx=None, df=None, dgate=None, dw=None, dw_after=None)):
        assert backward(**kw) == E_NULL, kw
    assert backward(has_f=0) == E_NULL  # df, dgate and dw_after cannot be
    assert backward(has_f=0, f=None, df=None, dgate=None, dw_after=None) in NO_GPU
    # without the norm f's values serve dgate and dw_after alone
    assert backward(norm_f=0, f=None) == E_NULL
    assert backward(norm_f=0, f=None, dgate=None, dw_after=None) in NO_GPU
    assert backward(dn=None, out=None, dw=None) in NO_GPU
    for span in (1, 3):
        need = blr.load().blr_norm_workspace_bytes(1000, 64, span)
        assert need > 0 and backward(1000, span=span, ws_bytes=need - 1) == E_WS
        assert backward(1000, span=span, ws_bytes=need) in NO_GPU
    assert backward(ws=None) == E_WS
    for k in set(BWD) - {"stats", "out_b", "f_b", "out_q", "f_q"}:
        assert backward(**{k: 8}) == E_ALIGN, k
    for k in ("out_q", "f_q"):
        assert backward(**{**kept, k: 8}) == E_ALIGN, k
    assert backward(stats=2) == E_ALIGN
    for form in (ROWS, kept):
        there = [k for k in BWD if form.get(k, 0) is not None]
        for o in ("dx", "df", "dgate", "dw", "dw_after", "ws"):
            for other in there:
                if o != other:
                    assert backward(**{**form, o: at(0), other: at(0)}) == E_OVERLAP, (o, other)


GFWD = ("x", "w_gate", "w_up", "h", "tape_q", "tape_b")
GBWD = ("x", "x_q", "x_b", "dh", "w_gate", "w_up", "tape_q", "tape_b", "dx", "dw_gate", "dw_up", "ws")


def gated(M=4, d=128, ff=256, dtype=BF16, ht=BF16, kind=0, **kw):
    return call("blr_gated_forward", (M, d, ff, dtype, ht, "x", "w_gate", "w_up", kind, "h", "tape_q", "tape_b"), GFWD, kw)


def gated_backward(M=4, d=128, ff=256, dtype=BF16, ht=BF16, gt=BF16, kind=0, gscale=1.0, ws_bytes=BIG, **kw):
    kw = {"x_q": None, "x_b": None, **kw}
    return call("blr_gated_backward",
                (M, d, ff, dtype, ht, gt, "x", "x_q", "x_b", "dh", "w_gate", "w_up", kind, "tape_q", "tape_b",
                 f32(gscale), "dx", 0, "dw_gate", "dw_up", 0, "ws", ws_bytes), GBWD, kw)


@pytest.mark.parametrize("caller", [gated, gated_backward])
def test_gated_refuses(caller):
    assert caller() in NO_GPU and caller(tape_q=None, tape_b=None) in NO_GPU
    assert caller(dtype=F16, ht=F32, **({"gt": F16} if caller is gated_backward else {})) in NO_GPU
    for kw in (dict(dtype=F32), dict(dtype=F32, ht=F32), dict(ht=F16), dict(dtype=3), dict(ht=-1), dict(kind=2),
               dict(kind=-1)):
        assert caller(**kw) == E_DTYPE, kw
    for M, d, ff in [(0, 128, 128), ((1 << 31) - 65536, 128, 128), (4, 64, 128), (4, 192, 128), (4, 128, 0),
                     (4, 128, 160), (4, (1 << 20) + 128, 128), (4, 128, (1 << 20) + 128), (1 << 30, 128, 1 << 20),
                     (1 << 30, 1 << 20, 128)]:
        assert caller(M, d, ff) == E_SHAPE, (M, d, ff)
        assert blr.load().blr_gated_workspace_bytes(M, d, ff) == 0
    for k in ("w_gate", "w_up", "tape_q", "tape_b"):
        assert caller(**{k: None}) == E_NULL, k
    for k in ("x", "w_gate", "w_up", "tape_q"):
        assert caller(**{k: 8}) == E_ALIGN, k
    outs = ("h", "tape_q", "tape_b") if caller is gated else ("dx", "dw_gate", "dw_up", "ws")
    there = GFWD if caller is gated else [k for k in GBWD if k not in ("x_q", "x_b")]
    for o in outs:
        for other in there:
            if o != other:
                assert caller(**{o: at(0), other: at(0)}) == E_OVERLAP, (o, other)


def test_gated_forward_refuses():
    for k in ("x", "h"):
        assert gated(**{k: None}) == E_NULL, k
    assert gated(h=8) == E_ALIGN


def test_gated_backward_refuses():
    for gt in (F16, 3):
        assert gated_backward(gt=gt) == E_DTYPE
    for g in (0.0, -1.0, 3.0, float("inf"), float("nan")):
        assert gated_backward(gscale=g) == -3, g
    for kw in (dict(dh=None), dict(x=None), dict(dw_up=None), dict(dx=None, dw_gate=None, dw_up=None),
               dict(x_q=0, x_b=0), dict(x=None, x_q=0), dict(x=None, dw_gate=None, dw_up=None, tape_q=None, tape_b=None)):
        assert gated_backward(**kw) == E_NULL, kw
    for kw in (dict(x=None, x_q=0, x_b=0), dict(x=None, dw_gate=None, dw_up=None), dict(dx=None)):
        assert gated_backward(**kw) in NO_GPU, kw
    for k in ("dh", "dx", "dw_gate", "dw_up", "ws"):
        assert gated_backward(**{k: 8}) == E_ALIGN, k
    need = blr.load().blr_gated_workspace_bytes(1000, 128, 256)
    assert need > 0 and gated_backward(1000, ws_bytes=need - 1) == E_WS and gated_backward(ws=None) == E_WS
    assert gated_backward(1000, ws_bytes=need) in NO_GPU
    for k in ("x_q", "x_b"):
        assert gated_backward(**{**dict(x=None, x_q=0, x_b=0), k: at(0), "dx": at(0)}) == E_OVERLAP, k


def test_binding_refuses():
    """The binding names what is wrong before it asks the library."""
    import torch
    x = torch.zeros((4, 64))
    for f in (lambda: blr.blr_norm_forward(x), lambda: blr.blr_checkpoint_save(x),
              lambda: blr.blr_norm_backward(x, x, x), lambda: blr.blr_gated_forward(x, x, x),
              lambda: blr.blr_gated_backward(x, x, x, x), lambda: blr.blr_checkpoint_load(x, x, torch.float32)):
        with pytest.raises((TypeError, ValueError)):
            f()
