"""GPU parity of the low-rank adapters, forward and backward, with their plain
64-bit form: every element within the bound of its sums."""
from __future__ import annotations

import numpy as np
import pytest

import _operators_ref as ref
import binary_rank_linear_amd as blr
import synth
from _gpu_util import host, say, to_dev

TYPES = [("float32", "float32"), ("float32", "float16"), ("float32", "bfloat16"), ("float16", "float16"),
         ("bfloat16", "bfloat16")]


def dt(name):
    import torch
    return getattr(torch, name)


def num(t):
    return host(t.double())


def make(dev, M, d_in, d_out, r, E, act, wt, kind, seed=0):
    """Inputs of a call, with the plan of its rows."""
    import torch
    rng = np.random.default_rng(seed + M + d_in)
    if kind == "tokens":
        ids = rng.integers(0, E, M)
        ids[rng.random(M) < 0.15] = -1
    elif kind == "runs":  # adapters of several tiles and ranges, some without rows
        cuts = np.sort(rng.integers(0, M + 1, max(1, E // 2)))
        of = rng.permutation(np.arange(-1, E))[:cuts.size + 1]
        ids = np.repeat(np.resize(of, cuts.size + 1), np.diff(np.concatenate([[0], cuts, [M]])))
    elif kind == "one":
        ids = np.full(M, E // 2)
    else:
        ids = np.full(M, -1)
    g = torch.Generator(device=dev).manual_seed(seed + 1)

    def normal(shape, sigma, t):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dt(t))

    v = dict(ids=ids.astype(np.int32), x=normal((M, d_in), 1.0, act), down=normal((E, r, d_in), d_in ** -0.5, wt),
             up=normal((E, d_out, r), r ** -0.5, wt), y=normal((M, d_out), 1.0, act), dy=normal((M, d_out), 0.5, act),
             scale=torch.rand(E, generator=g, device=dev) + 0.25)
    v["offsets"], v["order"], _ = blr.blr_route_sort(torch.from_numpy(v["ids"]).to(dev), E)
    return v


def check_forward(v, act, acc, scale=True, order=True):
    M, d_in = v["x"].shape
    r = v["down"].shape[1]
    ids = v["ids"] if order else np.sort(np.where(v["ids"] < 0, v["down"].shape[0], v["ids"]))
    (s, y), (sm, ym) = ref.adapters_forward(num(v["x"]), num(v["down"]), num(v["up"]), ids,
                                            num(v["scale"]) if scale else None)
    y0 = num(v["y"]) if acc else 0.0
    out = v["y"].clone() if acc else None
    got, tape = blr.blr_adapters_forward(v["x"], v["down"], v["up"], v["offsets"], v["order"] if order else None,
                                         v["scale"] if scale else None, y=out, accumulate_y=acc, keep_tape=True)
    # s: d_in products and, with them, the splits' and waves' sums; y: r more, the factor, the addition to y
    ref.within(num(tape), s, sm, d_in + 1)
    ref.within(num(got), y0 + y, np.abs(y0) + ym, d_in + r + 4, act)
    if acc:  # rows without an adapter are not touched
        none = (ids < 0) | (ids >= v["down"].shape[0])
        assert np.array_equal(num(got)[none], y0[none])
    return got, tape


def check_backward(v, act, acc, scale=True):
    import torch
    M, d_in = v["x"].shape
    E, r, _ = v["down"].shape
    d_out = v["up"].shape[1]
    _, tape = blr.blr_adapters_forward(v["x"], v["down"], v["up"], v["offsets"], v["order"], keep_tape=True)
    want, mag = ref.adapters_backward(num(v["x"]), num(v["dy"]), num(v["down"]), num(v["up"]), v["ids"],
                                      num(v["scale"]) if scale else None, num(tape))
    kw = {}
    if acc:
        base = [torch.randn(v["down"].shape, device=tape.device), torch.randn(v["up"].shape, device=tape.device),
                torch.randn_like(v["x"])]
        want = [w + num(b) for w, b in zip(want, base)]
        mag = [m + np.abs(num(b)) for m, b in zip(mag, base)]
        kw = dict(zip(("grad_down", "grad_up", "dx"), base), accumulate_grads=True, accumulate_dx=True)
    got = blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], v["offsets"], v["order"],
                                    v["scale"] if scale else None, tape, **kw)
    most = int(np.bincount(v["ids"][v["ids"] >= 0], minlength=1).max())
    terms = (d_out + most + 4, most + 4, d_out + r + 4)
    for g, w, m, n, name, t in zip(got, want, mag, terms, ("grad_down", "grad_up", "dx"), ("float32", "float32", act)):
        try:
            ref.within(num(g), w, m, n, t)
        except AssertionError as e:
            raise AssertionError(f"{name}: {e}") from None
    return got, tape


SHAPES = [(1, 128, 128, 8, 1, "one"), (3, 256, 128, 16, 4, "tokens"), (64, 128, 256, 8, 2, "one"),
          (65, 384, 256, 24, 3, "tokens"), (130, 256, 640, 40, 5, "tokens"), (300, 512, 384, 64, 7, "runs"),
          (200, 256, 256, 128, 3, "runs"), (257, 128, 128, 32, 200, "tokens"), (17, 1280, 128, 16, 1024, "tokens"),
          (1500, 256, 384, 16, 4, "runs"), (1100, 128, 256, 72, 2, "one"), (90, 128, 128, 8, 3, "none")]


@pytest.mark.gpu
@pytest.mark.parametrize("act,wt", TYPES)
@pytest.mark.parametrize("M,d_in,d_out,r,E,kind", SHAPES)
def test_forward(dev, M, d_in, d_out, r, E, kind, act, wt):
    say(f"adapters forward M={M} {d_in}->{d_out} r={r} E={E} {kind} {act}/{wt}")
    v = make(dev, M, d_in, d_out, r, E, act, wt, kind)
    check_forward(v, act, acc=True)
    check_forward(v, act, acc=False, scale=False)
    check_forward(v, act, acc=True, order=False)


@pytest.mark.gpu
@pytest.mark.parametrize("act,wt", TYPES)
@pytest.mark.parametrize("M,d_in,d_out,r,E,kind", SHAPES)
def test_backward(dev, M, d_in, d_out, r, E, kind, act, wt):
    import torch
    say(f"adapters backward M={M} {d_in}->{d_out} r={r} E={E} {kind} {act}/{wt}")
    v = make(dev, M, d_in, d_out, r, E, act, wt, kind)
    got, tape = check_backward(v, act, acc=False)
    check_backward(v, act, acc=True, scale=False)
    # each half alone: the same bits
    plan = (v["offsets"], v["order"], v["scale"])
    gd, gu, none = blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], *plan, tape, need_dx=False)
    assert none is None and torch.equal(gd, got[0]) and torch.equal(gu, got[1])
    a, b, dx = blr.blr_adapters_backward(None, v["dy"], v["down"], v["up"], *plan, grads=False)
    assert a is None and b is None and torch.equal(dx, got[2])


@pytest.mark.gpu
def test_gradients_against_differences(dev):
    """y is linear in x, down and up, so (L(p + v) - L(p - v)) / 2 is the
    gradient along v exactly. L = sum dy.y of f32 outputs, each off by at most
    its bound: the two sides differ by at most sum |dy| times that, plus the
    gradients' own bounds times |v|."""
    import torch
    say("adapters gradients against differences")
    M, d_in, d_out, r, E = 150, 256, 128, 16, 4
    v = make(dev, M, d_in, d_out, r, E, "float32", "float32", "tokens")
    (gd, gu, dx), _ = check_backward(v, "float32", acc=False)

    def loss(**kw):
        u = {**v, **kw}
        y, _ = blr.blr_adapters_forward(u["x"], u["down"], u["up"], v["offsets"], v["order"], v["scale"])
        _, (_, ym) = ref.adapters_forward(num(u["x"]), num(u["down"]), num(u["up"]), v["ids"], num(v["scale"]))
        dy = num(v["dy"])
        n = d_in + r + 4
        return (dy * num(y)).sum(), (np.abs(dy) * ym).sum() * n * ref.U * 1.01

    for name, g in (("x", dx), ("down", gd), ("up", gu)):
        step = torch.randn_like(v[name])
        hi, e1 = loss(**{name: v[name] + step})
        lo, e2 = loss(**{name: v[name] - step})
        # p + v and p - v are themselves rounded to f32, half a step of each element
        moved = ((np.abs(num(v[name])) + np.abs(num(step))) * np.abs(num(g))).sum() * ref.U
        own = (np.abs(num(g)) * np.abs(num(step))).sum() * (d_in + d_out + r + M + 8) * ref.U * 40
        assert abs((hi - lo) / 2 - (num(g) * num(step)).sum()) <= (e1 + e2) / 2 + moved + own, name


@pytest.mark.gpu
def test_nothing_leaks_between_rows(dev):
    """NaN and infinity in rows without an adapter, in adapters without rows
    and in other rows' adapters stay where they are."""
    import torch
    say("adapters with NaN and infinities")
    M, d_in, d_out, r, E = 100, 256, 128, 24, 5
    v = make(dev, M, d_in, d_out, r, E, "float32", "float32", "tokens")
    ids = v["ids"]
    ids[ids == 2] = 1  # adapter 2 has no rows
    v["offsets"], v["order"], _ = blr.blr_route_sort(torch.from_numpy(ids).to(dev), E)
    y, tape = check_forward(v, "float32", acc=False)
    (gd, gu, dx), _ = check_backward(v, "float32", acc=False)
    none = torch.from_numpy(ids < 0).to(dev)
    x, dy, down, up = (v[n].clone() for n in ("x", "dy", "down", "up"))
    bad = 3
    x[none] = float("nan")
    dy[none] = float("inf")
    down[2] = float("nan")
    up[2] = float("inf")
    down[bad, 1, 5] = float("nan")
    up[bad, 7, 2] = float("inf")
    plan = (v["offsets"], v["order"], v["scale"])
    y2, tape2 = blr.blr_adapters_forward(x, down, up, *plan, keep_tape=True)
    tape_in = tape.clone()
    tape_in[none] = float("nan")
    gd2, gu2, dx2 = blr.blr_adapters_backward(x, dy, down, up, *plan, tape_in)
    fine = torch.from_numpy(ids != bad).to(dev)
    assert torch.equal(y2[fine], y[fine]) and torch.equal(tape2[fine], tape[fine]) and torch.equal(dx2[fine], dx[fine])
    keep = [e for e in range(E) if e != bad]
    assert torch.equal(gd2[keep], gd[keep]) and torch.equal(gu2, gu)  # grad_up reads neither down nor up
    hit = ~fine
    assert torch.isnan(tape2[hit][:, 1]).all() and torch.isfinite(tape2[hit][:, 0]).all()
    # only the column with the infinite weight is not finite (its rank's s is), besides the NaN rank's
    assert torch.isnan(y2[hit]).all()


@pytest.mark.gpu
def test_an_infinite_row_stays_infinite(dev):
    import torch
    say("adapters with an infinite element")
    x = torch.zeros((2, 128), device=dev)
    x[0, 3] = float("inf")
    x[1, 3] = 1.0
    down, up = torch.ones((1, 8, 128), device=dev), torch.ones((1, 128, 8), device=dev)
    down[0, :, 4:] = 0  # 0 . 0, not 0 . inf
    offsets = torch.tensor([0, 2], dtype=torch.int32, device=dev)
    y, tape = blr.blr_adapters_forward(x, down, up, offsets, keep_tape=True)
    assert torch.isposinf(tape[0]).all() and torch.isposinf(y[0]).all()
    assert (tape[1] == 1).all() and (y[1] == 8).all()


@pytest.mark.gpu
def test_writes_stay_inside(dev):
    import torch
    say("adapters outputs between guards")
    M, d_in, d_out, r, E, guard = 700, 256, 384, 24, 3, 4096
    v = make(dev, M, d_in, d_out, r, E, "float32", "float32", "one")
    need = blr.workspace_adapters(M, d_in, d_out, r, E).numel()

    def between(shape, dtype=torch.float32):
        n = int(np.prod(shape))
        whole = torch.full((n + 2 * guard,), 7, dtype=dtype, device=dev)
        return whole, whole[guard:guard + n].view(shape)

    buf = dict(y=between((M, d_out)), tape=between((M, r)), gd=between((E, r, d_in)), gu=between((E, d_out, r)),
               dx=between((M, d_in)), ws=between((need,), torch.uint8))
    plan = (v["offsets"], v["order"], v["scale"])
    out = {n: t for n, (_, t) in buf.items()}
    blr.blr_adapters_forward(v["x"], v["down"], v["up"], *plan, y=out["y"], tape_s=out["tape"], ws=out["ws"])
    blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], *plan, out["tape"], grad_down=out["gd"],
                              grad_up=out["gu"], dx=out["dx"], ws=out["ws"])
    torch.cuda.synchronize()
    for name, (whole, _) in buf.items():
        assert (whole[:guard] == 7).all() and (whole[-guard:] == 7).all(), name


@pytest.mark.gpu
def test_rows_past_32_bit_offsets(dev):
    """x and dx of over 2^32 bytes and 2^31 elements; three rows have an adapter."""
    import torch
    say("adapters with 17000 rows of 131072")
    M, d, r = 17000, 131072, 8
    ids = np.full(M, -1, np.int32)
    at = [0, 16390, M - 1]
    ids[at] = 0
    x = torch.zeros((M, d), dtype=torch.bfloat16, device=dev)
    torch.manual_seed(0)
    x[at] = torch.randn((3, d), device=dev).to(torch.bfloat16)
    down = (torch.randn((1, r, d), device=dev) / 256).to(torch.bfloat16)
    up = torch.randn((1, 128, r), device=dev).to(torch.bfloat16)
    dy = torch.randn((M, 128), device=dev).to(torch.bfloat16)
    offsets, order, _ = blr.blr_route_sort(torch.from_numpy(ids).to(dev), 1)
    y, tape = blr.blr_adapters_forward(x, down, up, offsets, order, keep_tape=True)
    xs, A, B = num(x[at]), num(down), num(up)
    one = np.zeros(3, np.int32)
    (s, yw), (sm, ym) = ref.adapters_forward(xs, A, B, one, None)
    ref.within(num(tape[at]), s, sm, d)
    ref.within(num(y[at]), yw, ym, d + r + 2, "bfloat16")
    assert int((y != 0).any(1).sum()) == 3
    gd, gu, dx = blr.blr_adapters_backward(x, dy, down, up, offsets, order, None, tape)
    want, mag = ref.adapters_backward(xs, num(dy[at]), A, B, one, None, num(tape[at]))
    ref.within(num(gd), want[0], mag[0], 140)
    ref.within(num(gu), want[1], mag[1], 8)
    ref.within(num(dx[at]), want[2], mag[2], 140, "bfloat16")
    dx[at] = 0
    assert not dx.any()


@pytest.mark.gpu
@pytest.mark.parametrize("act,r", [("float32", 24), ("float16", 16), ("bfloat16", 72)])
def test_gradients_of_a_dy_past_the_caches(dev, act, r):
    """dy of over 256 MB, which ds reads without keeping it; 90 rows over two
    adapters (a tile of 64 rows, and shorter ones) have one."""
    import torch
    say(f"adapters with 2100 rows of 131072, {act}, rank {r}")
    M, d_in, d_out, E = 2100, 128, 131072, 2
    t = getattr(torch, act)
    torch.manual_seed(r)
    ids = np.full(M, -1, np.int32)
    at = np.sort(np.random.default_rng(r).choice(M, 90, replace=False))
    ids[at] = np.arange(90) % 7 == 0
    x = torch.randn((M, d_in), device=dev).to(t)
    dy = torch.full((M, d_out), float("nan"), dtype=t, device=dev)
    dy[at] = torch.randn((90, d_out), device=dev).to(t)
    down = torch.randn((E, r, d_in), device=dev).to(t)
    up = (torch.randn((E, d_out, r), device=dev) / 256).to(t)
    scale = torch.tensor([0.5, -3.0], device=dev)
    tape = torch.randn((M, r), device=dev)
    offsets, order, _ = blr.blr_route_sort(torch.from_numpy(ids).to(dev), E)
    gd, gu, dx = blr.blr_adapters_backward(x, dy, down, up, offsets, order, scale, tape)
    want, mag = ref.adapters_backward(num(x[at]), num(dy[at]), num(down), num(up), ids[at], num(scale), num(tape[at]))
    ref.within(num(gd), want[0], mag[0], d_out + 94)
    ref.within(num(gu), want[1], mag[1], 94)
    ref.within(num(dx[at]), want[2], mag[2], d_out + r + 4, act)
    dx[at] = 0
    assert not dx.any()


@pytest.mark.gpu
def test_long_ranges(dev):
    """Rows enough for several ranges of the greatest length (4096) in the
    gradients; their sums against 64 bits on the GPU, in runs of columns."""
    import torch
    say("adapters gradients of 9000 rows of 131072")
    M, d_in, d_out, r = 9000, 128, 131072, 8
    torch.manual_seed(1)
    ids = torch.zeros(M, dtype=torch.int32, device=dev)
    ids[::9] = -1
    offsets, order, _ = blr.blr_route_sort(ids, 1)
    x = torch.randn((M, d_in), device=dev).to(torch.bfloat16)
    dy = torch.randn((M, d_out), device=dev).to(torch.bfloat16)
    down = torch.randn((1, r, d_in), device=dev).to(torch.bfloat16)
    up = (torch.randn((1, d_out, r), device=dev) / 256).to(torch.bfloat16)
    tape = torch.randn((M, r), device=dev)
    gd, gu, dx = blr.blr_adapters_backward(x, dy, down, up, offsets, order, None, tape)
    on = ids >= 0
    s, ds = tape[on].double(), torch.zeros((int(on.sum()), r), dtype=torch.float64, device=dev)
    dm = torch.zeros_like(ds)
    for c in range(0, d_out, 16384):
        part, w = dy[on, c:c + 16384].double(), up[0, c:c + 16384].double()
        ref.within(host(gu[0, c:c + 16384].double()), host(part.T @ s), host(part.abs().T @ s.abs()), M)
        ds += part @ w
        dm += part.abs() @ w.abs()
    xs = x[on].double()
    ref.within(num(gd[0]), host(ds.T @ xs), host(dm.T @ xs.abs()), d_out + M)
    ref.within(num(dx[on]), host(ds @ down[0].double()), host(dm @ down[0].double().abs()), d_out + r, "bfloat16")
    assert not dx[~on].any()


@pytest.mark.gpu
@pytest.mark.parametrize("act,wt", [("float32", "bfloat16"), ("bfloat16", "bfloat16")])
def test_many_adapters_with_several_ranges(dev, act, wt):
    """Adapters of several ranges on both sides of the 64th, in shuffled rows,
    among many of a few rows or none."""
    import torch
    say(f"adapters: 200 of them, three with several ranges, {act}/{wt}")
    M, E = 2500, 200
    v = make(dev, M, 128, 256, 24, E, act, wt, "none")
    rng = np.random.default_rng(3)
    ids = rng.permutation(np.concatenate([np.full(900, 3), np.full(700, 70), np.full(600, 150),
                                          rng.integers(-20, E, 300)]))
    v["ids"] = np.where(ids < 0, -1, ids).astype(np.int32)
    v["offsets"], v["order"], _ = blr.blr_route_sort(torch.from_numpy(v["ids"]).to(dev), E)
    check_forward(v, act, acc=True)
    check_backward(v, act, acc=True)
    check_backward(v, act, acc=False)


@pytest.mark.gpu
@pytest.mark.parametrize("cnt", [1, 15, 16, 17, 63, 64, 65, 128, 507, 508, 512, 513, 769])
@pytest.mark.parametrize("act", ["float32", "float16", "bfloat16"])
def test_row_counts_at_tile_edges(dev, cnt, act):
    """One adapter with a number of rows on each side of the kernels' tiles and
    ranges, beside others with one row and none."""
    say(f"adapters with {cnt} rows of one adapter, {act}")
    M, E = cnt + 5, 4
    v = make(dev, M, 128, 256, 16, E, act, act, "none", seed=cnt)
    import torch
    ids = np.full(M, 2, np.int32)
    ids[[0, M - 1]] = 0
    ids[[1, 2, M // 2 + 1]] = -1
    v["ids"] = ids
    v["offsets"], v["order"], _ = blr.blr_route_sort(torch.from_numpy(ids).to(dev), E)
    check_forward(v, act, acc=True)
    check_backward(v, act, acc=False)


@pytest.mark.gpu
def test_plans_out_of_order_do_no_harm(dev):
    """Offsets that do not ascend or point outside, and rows outside [0, M):
    refused by nothing on the host, and the kernels' own limits keep every
    access inside; the outputs' guards are left as they were."""
    import torch
    say("adapters with malformed plans")
    M, d_in, d_out, r, E, guard = 600, 256, 256, 16, 6, 1024
    v = make(dev, M, d_in, d_out, r, E, "float32", "float32", "tokens")
    tape = torch.randn((M, r), device=dev)

    def between(shape):
        n = int(np.prod(shape))
        whole = torch.full((n + 2 * guard,), 7.0, device=dev)
        return whole, whole[guard:guard + n].view(shape)

    for bad in ([0, M, 0, M, 0, M, 0], [-5, 9, M + 100, 3, 2 ** 31 - 1, -2 ** 31, 7], [M] * 7, [2 ** 31 - 1] * 7):
        offsets = torch.tensor(bad, dtype=torch.int64).to(torch.int32).to(dev)
        order = v["order"].clone()
        order[::7] = -1
        order[1::7] = M
        buf = dict(y=between((M, d_out)), t=between((M, r)), gd=between((E, r, d_in)), gu=between((E, d_out, r)),
                   dx=between((M, d_in)))
        out = {n: t for n, (_, t) in buf.items()}
        blr.blr_adapters_forward(v["x"], v["down"], v["up"], offsets, order, v["scale"], y=out["y"], tape_s=out["t"])
        blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], offsets, order, v["scale"], tape,
                                  grad_down=out["gd"], grad_up=out["gu"], dx=out["dx"])
        torch.cuda.synchronize()
        for name, (whole, _) in buf.items():
            assert (whole[:guard] == 7).all() and (whole[-guard:] == 7).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["float32", "bfloat16"])
def test_positions_without_a_row_add_nothing(dev, act):
    """A plan's position whose row is outside [0, M) is left out of every
    gradient, whatever the rows that the plan does name hold."""
    import torch
    say(f"adapters, positions without a row, {act}")
    M, d_in, d_out, r, E = 150, 256, 128, 16, 3
    v = make(dev, M, d_in, d_out, r, E, act, act, "tokens")
    v["ids"][0] = 0  # row 0 is another adapter's than the positions that lose theirs
    offsets, order, _ = blr.blr_route_sort(torch.from_numpy(v["ids"]).to(dev), E)
    first, end = int(offsets[1]), int(offsets[3])
    assert end - first > 4
    lost = [first, first + 3, end - 1]
    rows = order[lost].long()
    order[lost] = torch.tensor([-1, M, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    tape = torch.randn((M, r), device=dev)

    def run():
        y, _ = blr.blr_adapters_forward(v["x"], v["down"], v["up"], offsets, order, v["scale"],
                                        y=torch.full((M, d_out), 7.0, dtype=v["x"].dtype, device=dev))
        return (y,) + blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], offsets, order, v["scale"], tape,
                                                dx=torch.full_like(v["x"], 7.0))

    y, gd, gu, dx = run()
    assert (y[rows] == 7).all() and (dx[rows] == 7).all()  # a row that no position names is not written
    kept = v["ids"].copy()
    kept[rows.cpu().numpy()] = -1
    want, mag = ref.adapters_backward(num(v["x"]), num(v["dy"]), num(v["down"]), num(v["up"]), kept, num(v["scale"]),
                                      num(tape))
    ref.within(num(gd), want[0], mag[0], d_out + M + 4)
    ref.within(num(gu), want[1], mag[1], M + 4)
    v["x"][0] = float("nan")
    v["dy"][0] = float("inf")
    tape[0] = float("nan")
    y2, gd2, gu2, dx2 = run()
    assert torch.equal(gd2[1:], gd[1:]) and torch.equal(gu2[1:], gu[1:])
    assert torch.equal(y2[1:], y[1:]) and torch.equal(dx2[1:], dx[1:])


@pytest.mark.gpu
def test_reruns_streams_and_graphs(dev):
    """The same bits on a rerun, on another stream, and from two captured
    graphs (each with a workspace of its own) replayed in turn on new inputs
    with eager calls between."""
    import torch
    say("adapters reruns, side stream, two graphs")
    M, d_in, d_out, r, E = 900, 256, 384, 16, 5
    v = make(dev, M, d_in, d_out, r, E, "float32", "float16", "runs")
    plan = (v["offsets"], v["order"], v["scale"])

    def run(ws=None, stream=None):
        y, tape = blr.blr_adapters_forward(v["x"], v["down"], v["up"], *plan, keep_tape=True, ws=ws, stream=stream)
        return (y, tape) + blr.blr_adapters_backward(v["x"], v["dy"], v["down"], v["up"], *plan, tape, ws=ws,
                                                     stream=stream)

    eager = run()
    assert all(torch.equal(a, b) for a, b in zip(run(), eager))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    graphs = []
    for _ in range(2):
        ws = blr.workspace_adapters(M, d_in, d_out, r, E, dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(ws)
        graphs.append((g, out, ws))
    for step in range(3):
        v["x"].normal_()
        v["dy"].normal_()
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = run()
        for _, out, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_beside_a_layer(dev):
    """As it is used: one `blr` layer that all tokens share, and a mixture of
    adapters beside it, two weighted choices a token: sort, gather, adapters
    on the sorted rows, combine onto the layer's y; then the gradients back to
    x and to the choices' weights."""
    import torch
    say("blr layer with routed adapters")
    T, k, E, d_in, d_out, r = 203, 2, 6, 256, 384, 16
    lay = to_dev(synth.custom(T, d_in, d_out, 128, seed=12), dev)
    v = make(dev, T, d_in, d_out, r, E, "float32", "float32", "tokens")
    v["x"] = lay["x"]
    rng = np.random.default_rng(2)
    ids = rng.integers(-1, E, (T, k)).astype(np.int32)
    w = torch.rand((T, k), device=dev)
    y, _, _ = blr.blr_forward(lay["x"], lay["bits_u"], lay["bits_v"], lay["h"], lay["l"], lay["g"])
    base = num(y)
    offsets, order, slot = blr.blr_route_sort(torch.from_numpy(ids).to(dev), E)
    xs = blr.blr_route_gather(v["x"], offsets, slot)
    ys, tape = blr.blr_adapters_forward(xs, v["down"], v["up"], offsets, None, v["scale"], keep_tape=True)
    blr.blr_route_combine(ys, offsets, slot, w, y=y, accumulate_y=True)
    dys, dw = blr.blr_route_combine_backward(v["dy"], ys, offsets, slot, w)
    gd, gu, dxs = blr.blr_adapters_backward(xs, dys, v["down"], v["up"], offsets, None, v["scale"], tape)
    dx = blr.blr_route_combine(dxs, offsets, slot)

    x, A, B, c, dy, wn = (num(t) for t in (v["x"], v["down"], v["up"], v["scale"], v["dy"], w))
    want_y, want_dx, want_dw = base.copy(), np.zeros(x.shape), np.zeros(wn.shape)
    ym, dxm, dwm = np.abs(base), np.zeros(x.shape), np.zeros(wn.shape)
    want_gd, want_gu, gdm, gum = (np.zeros(a.shape) for a in (A, B, A, B))
    for j in range(k):
        (s, yj), (sm, yjm) = ref.adapters_forward(x, A, B, ids[:, j], c)
        wj = wn[:, j][:, None]
        want_y += wj * yj
        ym += wj * yjm
        want_dw[:, j], dwm[:, j] = (dy * yj).sum(1), (np.abs(dy) * yjm).sum(1)
        (a, b, dxj), (am, bm, dxjm) = ref.adapters_backward(x, wj * dy, A, B, ids[:, j], c, s)
        # the tape's own error, through |s| -> its sum of absolute terms
        _, (_, bm, _) = ref.adapters_backward(np.abs(x), np.abs(wj * dy), np.abs(A), np.abs(B), ids[:, j], c, sm)
        want_dx, dxm = want_dx + dxj, dxm + dxjm
        want_gd, gdm, want_gu, gum = want_gd + a, gdm + am, want_gu + b, gum + bm
    n = d_in + d_out + r + T * k + 16
    for got, want, mag in ((y, want_y, ym), (dx, want_dx, dxm), (dw, want_dw, dwm), (gd, want_gd, gdm),
                           (gu, want_gu, gum)):
        ref.within(num(got), want, mag, n)


@pytest.mark.gpu
def test_binding_refuses(dev):
    import torch
    say("adapters refusals")
    v = make(dev, 8, 128, 256, 8, 3, "float32", "float32", "tokens")
    x, dy, down, up, o, order, c = (v[n] for n in ("x", "dy", "down", "up", "offsets", "order", "scale"))
    tape = torch.zeros((8, 8), device=dev)
    fwd, bwd = blr.blr_adapters_forward, blr.blr_adapters_backward
    for bad in [lambda: fwd(x.double(), down, up, o), lambda: fwd(x, down, up.half(), o),
                lambda: fwd(x, down, up, o.long()), lambda: fwd(x, down, up, o, order.long()),
                lambda: fwd(x, down, up, o, order, c.half()), lambda: bwd(None, dy, down, up, o, order, c, tape),
                lambda: bwd(x, dy, down, up, o, order, c)]:
        with pytest.raises(TypeError):
            bad()
    for bad in [lambda: fwd(x[:, :64], down, up, o), lambda: fwd(x, down, up[:2], o), lambda: fwd(x, down, up, o[:2]),
                lambda: fwd(x, down, up, o, order[:4]), lambda: fwd(x, down, up, o, order, c[:1]),
                lambda: fwd(x, down, up, o, accumulate_y=True), lambda: fwd(x[0], down, up, o),
                lambda: fwd(dy, up, up, o), lambda: fwd(x.cpu(), down, up, o),
                lambda: fwd(torch.zeros((128, 8), device=dev).t(), down, up, o),
                lambda: bwd(x, dy, down, up, o, order, c, tape, accumulate_grads=True),
                lambda: bwd(x, dy, down, up, o, order, c, tape, grads=False, grad_down=torch.zeros_like(down)),
                lambda: bwd(x, dy, down, up, o, order, c, tape, need_dx=False, dx=torch.zeros_like(x))]:
        with pytest.raises(ValueError):
            bad()
    for bad in [lambda: bwd(x, dy, down, up, o, order, c, tape, dx=x),
                lambda: fwd(x.half(), down, up, o), lambda: fwd(x.half(), down.bfloat16(), up.bfloat16(), o),
                lambda: fwd(x, down[:, :4].contiguous(), up[:, :, :4].contiguous(), o),
                lambda: fwd(x, down, up, o, ws=torch.empty(64, dtype=torch.uint8, device=dev)),
                lambda: bwd(x, dy, down, up, o, order, c, tape, grads=False, need_dx=False)]:
        with pytest.raises(blr.BlrError):
            bad()
