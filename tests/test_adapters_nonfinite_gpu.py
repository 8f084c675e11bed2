"""GPU tests of NaN and infinity in the adapters' 16-bit rows: they reach what
meets them and nothing else."""
from __future__ import annotations

import numpy as np
import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say

TYPES = [("float16", "float16"), ("bfloat16", "bfloat16"), ("float32", "float16")]


def inputs(dev, act, wt, r, rows, seed=0):
    """Rows of adapters 0, 1, 3 and of none in turn, `rows` of each; adapter 2
    has none."""
    import torch
    torch.manual_seed(seed)
    E, d_in, d_out, M = 4, 256, 128, 4 * rows
    rn = lambda t, *s: torch.randn(s, device=dev).to(getattr(torch, t))  # noqa: E731
    v = dict(x=rn(act, M, d_in), dy=rn(act, M, d_out), down=rn(wt, E, r, d_in), up=rn(wt, E, d_out, r))
    ids = torch.tensor([0, 1, 3, -1], device=dev).int().repeat(rows)
    offsets, order, _ = blr.blr_route_sort(ids, E)
    return v, ids, (offsets, order, torch.tensor([0.5, 2.0, 1.0, -1.5], device=dev))


def run(v, plan, tape=None):
    y, s = blr.blr_adapters_forward(v["x"], v["down"], v["up"], *plan, keep_tape=True)
    gd, gu, dx = blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], *plan, s if tape is None else tape)
    return dict(y=y, s=s, gd=gd, gu=gu, dx=dx)


def same(a, b):
    import torch
    return torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("rows", [5, 16, 17, 70])
@pytest.mark.parametrize("r", [8, 16, 24, 72])
@pytest.mark.parametrize("act,wt", TYPES)
def test_bad_values_stay_where_they_are(dev, act, wt, r, rows, bad):
    import torch
    say(f"adapters with {bad}, {act}/{wt}, r={r}, {rows} rows each")
    v, ids, plan = inputs(dev, act, wt, r, rows)
    want = run(v, plan)
    assert all(torch.isfinite(t).all() for t in want.values())
    none, keep = ids < 0, [0, 1, 2]

    # in rows without an adapter and in the adapter without rows: nothing changes
    u = {n: t.clone() for n, t in v.items()}
    u["x"][none], u["dy"][none] = bad, bad
    u["down"][2], u["up"][2] = bad, bad
    tape = want["s"].clone()
    tape[none] = bad
    got = run(u, plan, tape)
    assert all(same(got[n], want[n]) for n in want)

    # in one row of adapter 3: its other rows and the other adapters are the same
    row = int(torch.nonzero(ids == 3)[rows // 2])
    others = torch.arange(len(ids), device=dev) != row
    u = {n: t.clone() for n, t in v.items()}
    u["x"][row, 7] = bad
    got = run(u, plan)
    assert all(same(got[n][others], want[n][others]) for n in ("y", "s")) and same(got["dx"], want["dx"])
    assert same(got["gd"][keep], want["gd"][keep]) and same(got["gu"][keep], want["gu"][keep])
    assert not torch.isfinite(got["s"][row]).any() and not torch.isfinite(got["y"][row]).any()
    assert not torch.isfinite(got["gd"][3, :, 7]).any() and not torch.isfinite(got["gu"][3]).any()
    other_columns = torch.arange(256, device=dev) != 7
    assert same(got["gd"][3][:, other_columns], want["gd"][3][:, other_columns])
    u = {n: t.clone() for n, t in v.items()}
    u["dy"][row, 9] = bad
    got = run(u, plan)
    assert same(got["y"], want["y"]) and same(got["dx"][others], want["dx"][others])
    assert same(got["gd"][keep], want["gd"][keep]) and same(got["gu"][keep], want["gu"][keep])
    assert not torch.isfinite(got["dx"][row]).any() and not torch.isfinite(got["gd"][3]).any()
    assert not torch.isfinite(got["gu"][3, 9]).any()
    assert same(got["gu"][3, torch.arange(128, device=dev) != 9], want["gu"][3, torch.arange(128, device=dev) != 9])

    # in adapter 3 itself: the rows of the others are the same
    fine, hit = ids != 3, ids == 3
    for name, at in (("down", (3, r - 1, 5)), ("up", (3, 11, r - 2))):
        u = {n: t.clone() for n, t in v.items()}
        u[name][at] = bad
        got = run(u, plan)
        assert all(same(got[n][fine], want[n][fine]) for n in ("y", "s", "dx"))
        assert same(got["gd"][keep], want["gd"][keep]) and same(got["gu"][keep], want["gu"][keep])
        if name == "down":
            assert not torch.isfinite(got["s"][hit][:, r - 1]).any() and same(got["s"][:, :r - 1], want["s"][:, :r - 1])
            assert not torch.isfinite(got["y"][hit]).any() and not torch.isfinite(got["dx"][hit][:, 5]).any()
            assert not torch.isfinite(got["gu"][3][:, r - 1]).any()
            assert same(got["gu"][3][:, :r - 1], want["gu"][3][:, :r - 1]) and same(got["gd"], want["gd"])
        else:
            assert same(got["s"], want["s"]) and not torch.isfinite(got["y"][hit][:, 11]).any()
            other = torch.arange(128, device=dev) != 11
            assert same(got["y"][:, other], want["y"][:, other])
            assert not torch.isfinite(got["dx"][hit]).any() and not torch.isfinite(got["gd"][3, r - 2]).any()
            rest = torch.arange(r, device=dev) != r - 2
            assert same(got["gd"][3][rest], want["gd"][3][rest]) and same(got["gu"], want["gu"])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 20])
@pytest.mark.parametrize("act,wt", TYPES + [("float32", "float32")])
def test_an_infinite_scale(dev, act, wt, rows):
    """The rows and the gradients of that adapter are not finite, the others'
    are the same."""
    import torch
    say(f"adapters with an infinite scale, {act}/{wt}, {rows} rows each")
    v, ids, plan = inputs(dev, act, wt, 16, rows)
    want = run(v, plan)
    scale = plan[2].clone()
    scale[1] = float("inf")
    got = run(v, (plan[0], plan[1], scale))
    fine, hit, keep = ids != 1, ids == 1, [0, 2, 3]
    assert same(got["s"], want["s"]) and all(same(got[n][fine], want[n][fine]) for n in ("y", "dx"))
    assert all(same(got[n][keep], want[n][keep]) for n in ("gd", "gu"))
    assert not any(torch.isfinite(t).any() for t in (got["y"][hit], got["dx"][hit], got["gd"][1], got["gu"][1]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_routing_keeps_them_in_their_rows(dev, dtype):
    """Combine and its gradient on 16-bit rows: a bad row reaches its token and
    its weight's gradient; one that is not placed reaches nothing."""
    import torch
    say(f"route with NaN and infinities, {dtype}")
    t = getattr(torch, dtype)
    T, k, E, d = 40, 3, 5, 264
    rng = np.random.default_rng(0)
    ids = torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).to(dev)
    ids[4, 1], ids[9] = 2, -1
    offsets, order, slot = blr.blr_route_sort(ids, E)
    z, dy, w = torch.randn((T * k, d), device=dev).to(t), torch.randn((T, d), device=dev).to(t), torch.rand((T, k), device=dev)
    y = blr.blr_route_combine(z, offsets, slot, w)
    dz, dw = blr.blr_route_combine_backward(dy, z, offsets, slot, w)
    for bad in (float("nan"), float("inf"), float("-inf")):
        zb, wb, yb = z.clone(), w.clone(), dy.clone()
        zb[int(offsets[-1]):], wb[ids < 0] = bad, bad
        yb[9] = bad  # a token none of whose pairs is placed
        assert same(blr.blr_route_combine(zb, offsets, slot, wb), y)
        got = blr.blr_route_combine_backward(yb, zb, offsets, slot, wb)
        assert same(got[0], dz) and same(got[1], dw)
        zb[int(slot[4, 1]), 3] = bad
        got_y = blr.blr_route_combine(zb, offsets, slot, wb)
        at = torch.zeros((T, d), dtype=torch.bool, device=dev)
        at[4, 3] = True
        assert not torch.isfinite(got_y[at]).any() and same(got_y[~at], y[~at])
        got = blr.blr_route_combine_backward(yb, zb, offsets, slot, wb)
        at = torch.zeros((T, k), dtype=torch.bool, device=dev)
        at[4, 1] = True
        assert same(got[0], dz) and not torch.isfinite(got[1][at]).any() and same(got[1][~at], dw[~at])
