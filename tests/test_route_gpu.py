"""GPU parity of the token routing with its plain 64-bit form: the sort equal,
rows equal, weighted sums and gradients within the bound of their sums."""
from __future__ import annotations

import numpy as np
import pytest

import _operators_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import host, say

DTYPES = ["float32", "float16", "bfloat16"]


def dt(name):
    import torch
    return getattr(torch, name)


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def make_ids(shape, E, kind, seed):
    rng = np.random.default_rng(seed)
    n = int(np.prod(shape))
    if kind == "uniform":
        ids = rng.integers(0, E, n)
    elif kind == "one":
        ids = np.full(n, E - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    elif kind == "wild":  # half of them no expert: negative, E, and the type's ends
        ids = np.where(rng.random(n) < 0.5, rng.integers(0, E, n),
                       rng.choice([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1], n))
    else:  # skewed, in runs
        ids = np.repeat(rng.integers(0, E, n), 1 + rng.integers(0, 40, n))[:n]
    return ids.astype(np.int32).reshape(shape)


def check_sort(ids, E, dev, **kw):
    import torch
    got = blr.blr_route_sort(put(ids, dev), E, **kw)
    torch.cuda.synchronize()
    for g, want, name in zip(got, ref.sort(ids, E), ("offsets", "order", "slot")):
        assert g.shape == want.shape and np.array_equal(host(g), want), name
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 1000, 1025, 8191, 8192, 8193, 12289, 70001])
@pytest.mark.parametrize("E", [1, 2, 7, 63, 64, 65, 512, 1023, 1024])
def test_sort(dev, n, E):
    say(f"route_sort pairs={n} E={E}")
    for kind in ("uniform", "one", "none", "wild", "runs"):
        check_sort(make_ids((n,), E, kind, n + E), E, dev)


@pytest.mark.gpu
def test_sort_many_pairs(dev):
    """More pairs than 256 ranges of the least length hold."""
    say("route_sort 300001 x 5 pairs")
    for kind in ("uniform", "wild"):
        check_sort(make_ids((300001, 5), 61, kind, 3), 61, dev)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,d,none", [(1, 1, 1, 8, 0), (1, 3, 5, 128, 0.5), (5, 2, 3, 24, 0), (67, 4, 9, 136, 0.2),
                                          (300, 2, 16, 1024, 0.1), (130, 8, 128, 2056, 0), (33, 5, 8, 4104, 0.3),
                                          (9, 13, 64, 520, 0.1), (40, 2, 4, 256, 1.0)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows(dev, T, k, E, d, none, dtype):
    """sort, gather, combine and its gradient as they are used together."""
    import torch
    say(f"route rows T={T} k={k} E={E} d={d} none={none} {dtype}")
    rng = np.random.default_rng(T * 31 + d)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < none] = -1
    offsets, order, slot = check_sort(ids, E, dev)
    o, s = host(offsets), host(slot)
    torch.manual_seed(d)
    x, y0, dy = (torch.randn((T, d), device=dev).to(dt(dtype)) for _ in range(3))
    z = torch.randn((T * k, d), device=dev).to(dt(dtype))
    w = torch.randn((T, k), device=dev)
    num = lambda t: host(t.double())  # noqa: E731

    rows = blr.blr_route_gather(x, offsets, slot)
    assert np.array_equal(num(rows), ref.gather(num(x), o, s))

    # what is not placed must not be read: NaN there changes nothing
    zn, wn = z.clone(), w.clone()
    zn[int(o[-1]):] = float("nan")
    wn[put(ids, dev) < 0] = float("nan")
    y = blr.blr_route_combine(zn, offsets, slot, wn)
    want, mag = ref.combine(num(z), o, s, host(w))
    ref.within(num(y), want, mag, k + 1, dtype)
    ones = blr.blr_route_combine(zn, offsets, slot)
    want1, mag1 = ref.combine(num(z), o, s)
    ref.within(num(ones), want1, mag1, k, dtype)
    added = y0.clone()
    assert blr.blr_route_combine(zn, offsets, slot, wn, y=added, accumulate_y=True) is added
    ref.within(num(added), num(y0) + want, mag + np.abs(num(y0)), k + 2, dtype)

    dz, dw = blr.blr_route_combine_backward(dy, zn, offsets, slot, wn)
    want, want_w, mag = ref.combine_backward(num(dy), num(z), o, s, host(w))
    ref.within(num(dz), want, np.abs(want), 1, dtype)
    ref.within(num(dw), want_w, mag, d)
    dz1, dw1 = blr.blr_route_combine_backward(dy, None, offsets, slot)
    assert dw1 is None
    assert np.array_equal(num(dz1), ref.combine_backward(num(dy), None, o, s)[0])
    # again: the same bits
    again = blr.blr_route_combine_backward(dy, zn, offsets, slot, wn)
    assert torch.equal(again[0], dz) and torch.equal(again[1], dw)


@pytest.mark.gpu
def test_infinities_stay_in_their_tokens(dev):
    import torch
    say("route combine with infinities")
    ids = np.array([[0, 1], [1, 2], [2, 0]], np.int32)
    offsets, _, slot = check_sort(ids, 3, dev)
    z = torch.ones((6, 64), device=dev)
    z[int(slot[1, 0])] = float("inf")
    z[int(slot[2, 1])] = float("nan")
    y = host(blr.blr_route_combine(z, offsets, slot))
    assert (y[0] == 2).all() and np.isposinf(y[1]).all() and np.isnan(y[2]).all()


@pytest.mark.gpu
def test_writes_stay_inside(dev):
    """Outputs inside a larger buffer: what lies around them is left as it was."""
    import torch
    say("route outputs between guards")
    T, k, E, d = 37, 3, 5, 72
    ids = make_ids((T, k), E, "wild", 4)
    guard = 1024

    def between(shape, dtype):
        n = int(np.prod(shape))
        whole = torch.full((n + 2 * guard,), 7, dtype=dtype, device=dev)
        return whole, whole[guard:guard + n].view(shape)

    buf = {n: between(s, torch.int32) for n, s in (("offsets", (E + 1,)), ("order", (T * k,)), ("slot", (T, k)))}
    plan = check_sort(ids, E, dev, **{n: v for n, (_, v) in buf.items()})
    x = torch.randn((T, d), device=dev)
    z, w = torch.randn((T * k, d), device=dev), torch.rand((T, k), device=dev)
    buf.update(rows=between((T * k, d), torch.float32), y=between((T, d), torch.float32),
               dz=between((T * k, d), torch.float32), dw=between((T, k), torch.float32))
    blr.blr_route_gather(x, plan[0], plan[2], rows=buf["rows"][1])
    blr.blr_route_combine(z, plan[0], plan[2], w, y=buf["y"][1])
    blr.blr_route_combine_backward(x, z, plan[0], plan[2], w, dz=buf["dz"][1], dw=buf["dw"][1])
    torch.cuda.synchronize()
    for name, (whole, _) in buf.items():
        assert (whole[:guard] == 7).all() and (whole[-guard:] == 7).all(), name


@pytest.mark.gpu
def test_rows_past_32_bit_offsets(dev):
    """Row arrays of over 2^32 bytes and 2^31 elements."""
    import torch
    say("route rows of 40000 x 65536 bf16")
    T, d, E = 40000, 65536, 3
    ids = make_ids((T, 1), E, "uniform", 8)
    offsets, order, slot = check_sort(ids, E, dev)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device=dev)
    x += torch.arange(T, device=dev)[:, None] % 251
    rows = blr.blr_route_gather(x, offsets, slot)
    want = (order % 251).to(torch.bfloat16)
    assert torch.equal(rows[:, 0], want) and torch.equal(rows[:, -1], want) and torch.equal(rows[:, d // 2 + 3], want)
    del x
    y = blr.blr_route_combine(rows, offsets, slot)
    want = (torch.arange(T, device=dev) % 251).to(torch.bfloat16)
    assert torch.equal(y[:, 0], want) and torch.equal(y[:, -1], want)
    del rows
    dz, _ = blr.blr_route_combine_backward(y, None, offsets, slot)
    assert torch.equal(dz[:, -1], (order % 251).to(torch.bfloat16))


@pytest.mark.gpu
def test_other_stream_and_graph(dev):
    """On a stream of its own, then captured and replayed on new inputs with
    other work between the replays."""
    import torch
    say("route on a side stream and in a graph")
    T, k, E, d = 333, 4, 17, 384
    side = torch.cuda.Stream()
    ids = put(make_ids((T, k), E, "uniform", 1), dev)
    x, w = torch.randn((T, d), device=dev), torch.rand((T, k), device=dev)
    ws = blr.workspace_route(T * k, E, dev)

    def run(stream=None):
        offsets, order, slot = blr.blr_route_sort(ids, E, ws=ws, stream=stream)
        rows = blr.blr_route_gather(x, offsets, slot, stream=stream)
        y = blr.blr_route_combine(rows, offsets, slot, w, stream=stream)
        dz, dw = blr.blr_route_combine_backward(x, rows, offsets, slot, w, stream=stream)
        return offsets, order, slot, rows, y, dz, dw

    eager = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for step in range(4):
        ids.copy_(put(make_ids((T, k), E, "wild", 20 + step), dev))
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(run(), kept))


@pytest.mark.gpu
def test_binding_refuses(dev):
    import torch
    say("route refusals")
    ids = torch.zeros((4, 2), dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        blr.blr_route_sort(ids.long(), 4)
    with pytest.raises(blr.BlrError):
        blr.blr_route_sort(ids, 1025)
    with pytest.raises(blr.BlrError):
        blr.blr_route_sort(ids[:0], 4)
    with pytest.raises(ValueError):
        blr.blr_route_sort(ids.t(), 4)
    with pytest.raises(blr.BlrError):
        blr.blr_route_sort(ids, 4, slot=ids)
    with pytest.raises(blr.BlrError):
        blr.blr_route_sort(ids.repeat(2000, 1), 4, ws=torch.empty(16, dtype=torch.uint8, device=dev))
    offsets, order, slot = blr.blr_route_sort(ids, 4)
    x = torch.zeros((4, 64), device=dev)
    with pytest.raises(TypeError):
        blr.blr_route_gather(x.double(), offsets, slot)
    with pytest.raises(ValueError):
        blr.blr_route_gather(x[:3], offsets, slot)
    with pytest.raises(ValueError):
        blr.blr_route_gather(torch.zeros((4, 128), device=dev)[:, ::2], offsets, slot)
    with pytest.raises(blr.BlrError):
        blr.blr_route_gather(torch.zeros((4, 12), device=dev), offsets, slot)
    z = torch.zeros((8, 64), device=dev)
    with pytest.raises(ValueError):
        blr.blr_route_combine(z, offsets, slot, accumulate_y=True)
    with pytest.raises(blr.BlrError):
        blr.blr_route_combine(z, offsets, slot, y=z[:4])
    with pytest.raises(TypeError):
        blr.blr_route_combine(z, offsets, slot, torch.zeros((4, 2), dtype=torch.float16, device=dev))
    with pytest.raises(TypeError):
        blr.blr_route_combine_backward(x, None, offsets, slot, torch.zeros((4, 2), device=dev))
    with pytest.raises(ValueError):
        blr.blr_route_combine_backward(x, z, offsets, slot, dw=torch.zeros((4, 2), device=dev))
