"""The norms around a block against their formulas in 64 bits."""
import numpy as np
import pytest

import _block_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import say
from _operators_ref import within

# Roundings on the longest way of a value through a row's sums: at most 16
# products and additions in a thread, 6 additions along the wave, 16 over the
# waves, twice (a mean inside a mean), the root and the division (3), the gate
# (exp within 2 units, sum, quotient, products: 8) and the products around them.
ROW = 110
F32, F16, BF16 = "float32", "float16", "bfloat16"
TYPES = [(F32, F32, F32), (F32, F32, BF16), (F32, BF16, F16), (F32, F16, F32), (F16, F16, F16), (BF16, BF16, BF16)]


def dt(name):
    import torch
    return getattr(torch, name)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def case(dev, M, d, types, *, f=True, norm_f=True, after=True, gate=None, span=1, kind=0, w=True, seed=0, skip=0.75,
         scale=0.5):
    import torch
    g = torch.Generator(device=dev).manual_seed(seed + 1000 * M + d)

    def normal(shape, t, sigma=1.0):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dt(t))

    xt, ft, nt = types
    v = dict(x=normal((M, d), xt, 2.0), dn=normal((M, d), nt), dout=normal((M, d), xt),
             w=normal((d,), F32) if w else None, f=None, w_after=None, gate=None)
    if f:
        v["f"] = normal((M, d), ft)
        v["w_after"] = normal((d,), F32) if after else None
        if gate:
            v["gate"] = normal((-(-M // span), d), ft, 2.0)
    v["how"] = dict(w_after=v["w_after"], gate=v["gate"], gate_kind=kind, span=span, norm_f=f and norm_f, skip=skip,
                    scale=scale)
    v["c"] = dict(w=f64(v["w"]), w_after=f64(v["w_after"]), gate=f64(v["gate"]), kind=kind, span=span,
                  norm_f=f and norm_f, skip=float(np.float32(skip)), scale=float(np.float32(scale)),
                  eps=float(np.float32(1e-6)), has_f=f)
    return v


def check_forward(v, types, keep):
    out, n, stats, kept = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=dt(types[2]), keep=keep, **v["how"])
    c = v["c"]
    stream = f64(v["x"])
    if c["has_f"]:
        want, mag, rf = ref.norm_after(stream, f64(v["f"]), c)
        within(f64(out), want, mag, ROW, types[0])
        stream = f64(out)  # what follows is of the rows as they are stored
        if c["norm_f"]:
            within(f64(stats[1]), rf, rf, ROW)
        else:
            assert not stats[1].any()
    else:
        assert out is None and not stats[1].any()
    want, r = ref.norm_before(stream, c["w"], c["eps"])
    within(f64(stats[0]), r, r, ROW)
    within(f64(n), want, np.abs(want), ROW, types[2])
    if keep:
        q, b = ref.pack(stream, types[0])
        assert np.array_equal(kept[0].cpu().numpy(), q) and np.array_equal(kept[1].cpu().numpy(), b)
    return out if c["has_f"] else v["x"], stats, kept


def check_backward(v, types, out, stats, M, *, dn=True, dout=True, f=None, **more):
    """f: what stands for it in the call (rows, a checkpoint)."""
    c = v["c"]
    f = v["f"] if f is None else f

    def rows(t):
        if t is None or not isinstance(t, tuple):
            return f64(t)
        return ref.unpack(t[0].cpu().numpy(), t[1].cpu().numpy())

    got = blr.blr_norm_backward(v["dn"] if dn else None, v["dout"] if dout else None, out, f, v["w"], stats,
                                x_dtype=dt(types[0]), f_dtype=dt(types[1]) if c["has_f"] else None, **v["how"], **more)
    want = ref.norm_backward(f64(v["dn"]) if dn else None, f64(v["dout"]) if dout else None, rows(out), rows(f),
                             f64(stats), c)
    names = ("dx", "df", "dgate", "dw", "dw_after")
    for name, g in zip(names, got):
        if g is None:
            assert name not in want or (name == "dw_after" and c["w_after"] is None) or \
                (name == "dw" and c["w"] is None), name
            continue
        t = {"dx": types[0], "df": types[1], "dgate": types[1] if c["span"] == 1 else F32}.get(name, F32)
        # sums over rows: their additions too
        terms = ROW + (M if name in ("dw", "dw_after") else c["span"] if name == "dgate" else 0)
        value, mag = want[name]
        say(f"  {name} {t}")
        within(f64(g), value, mag, terms, t)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,d", [(1, 128), (5, 8), (67, 520), (3, 4096), (2, 8200), (3, 6152), (2, 8192), (131, 1096)])
def test_sandwich(dev, types, M, d):
    say(f"norm {types} {M}x{d}")
    v = case(dev, M, d, types, gate=True, kind=2)
    out, stats, _ = check_forward(v, types, False)
    check_backward(v, types, out, stats, M)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("M,span", [(1, 1), (1, 7), (37, 1), (37, 2), (37, 10), (37, 37), (37, 100), (2100, 1000),
                                    (2100, 3), (5000, 5000)])
def test_gates(dev, kind, M, span):
    types = (F32, BF16, BF16)
    say(f"gate {kind} M={M} span={span}")
    v = case(dev, M, 256, types, gate=True, kind=kind, span=span)
    out, stats, _ = check_forward(v, types, False)
    check_backward(v, types, out, stats, M)


@pytest.mark.gpu
@pytest.mark.parametrize("types", [(F32, F32, BF16), (BF16, BF16, BF16), (F16, F16, F16)])
@pytest.mark.parametrize("M,d", [(1, 32), (37, 736), (6, 4096), (3, 5120), (2, 16384)])
def test_checkpoints(dev, types, M, d):
    """The forward keeps the stream in 8 bits; the backward reads both rows so."""
    say(f"norm kept {types} {M}x{d}")
    v = case(dev, M, d, types, gate=True, kind=1)
    _, stats, kept = check_forward(v, types, True)
    check_backward(v, types, kept, stats, M, f=blr.blr_checkpoint_save(v["f"]))
    v = case(dev, M, d, types, f=False)
    x, stats, kept = check_forward(v, types, True)
    check_backward(v, types, kept, stats, M)


@pytest.mark.gpu
@pytest.mark.parametrize("norm_f,after,w", [(False, False, True), (False, True, False), (True, False, True),
                                            (True, True, False)])
def test_without(dev, norm_f, after, w):
    """Parts left out: the norm of f, the weights, one of the two gradients."""
    types, M, d = (F32, F16, F16), 45, 640
    say(f"norm_f={norm_f} after={after} w={w}")
    v = case(dev, M, d, types, norm_f=norm_f, after=after, w=w)
    out, stats, _ = check_forward(v, types, False)
    check_backward(v, types, out, stats, M)
    check_backward(v, types, out, stats, M, dout=False)
    check_backward(v, types, None, stats, M, dn=False)
    if not norm_f:  # f's values take no part in dx and df
        got = blr.blr_norm_backward(v["dn"], v["dout"], out, None, v["w"], stats, has_f=True, f_dtype=dt(F16),
                                    grads=False, **v["how"])
        want = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
        assert all(bool((a == b).all()) for a, b in zip(got[:2], want[:2])) and got[2:] == (None,) * 3


@pytest.mark.gpu
def test_accumulates(dev):
    import torch
    types, M, d, span = (F32, F32, F32), 700, 384, 300
    v = case(dev, M, d, types, gate=True, span=span)
    out, stats, _ = check_forward(v, types, False)
    first = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
    sums = [t.clone() for t in first[2:]]
    say("gradients added to what is there")
    again = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, dgate=sums[0], dw=sums[1],
                                  dw_after=sums[2], accumulate_grads=True, **v["how"])
    for a, b in zip(first[:2], again[:2]):
        assert torch.equal(a, b)
    for a, b in zip(first[2:], again[2:]):
        assert torch.equal(a * 2, b)  # doubling is exact


@pytest.mark.gpu
def test_against_differences(dev):
    """Every gradient against central differences of the forward in 64 bits."""
    types, M, d = (F32, F32, F32), 6, 32
    v = case(dev, M, d, types, gate=True, kind=2, span=4)
    out, _, stats, _ = [*blr.blr_norm_forward(v["x"], v["f"], v["w"], **v["how"])[:1], None,
                        *blr.blr_norm_forward(v["x"], v["f"], v["w"], **v["how"])[2:]]
    got = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
    c, base = v["c"], dict(x=f64(v["x"]), f=f64(v["f"]))
    base.update({k: c[k] for k in ("gate", "w", "w_after")})
    dn, dout = f64(v["dn"]), f64(v["dout"])

    def loss(at):
        cc = {**c, **{k: at[k] for k in ("gate", "w", "w_after")}}
        o = ref.norm_after(at["x"], at["f"], cc)[0]
        return (dout * o).sum() + (dn * ref.norm_before(o, at["w"], c["eps"])[0]).sum()

    rng = np.random.default_rng(0)
    for name, g in zip(("x", "f", "gate", "w", "w_after"), got):
        g = f64(g)
        way = rng.standard_normal(base[name].shape)
        h = 1e-5
        diff = (loss({**base, name: base[name] + h * way}) - loss({**base, name: base[name] - h * way})) / (2 * h)
        # the f32 gradient's own roundings (ROW of 2^-24 each on sums of about
        # 20 terms of size one), and h^2 of the third derivative
        assert abs(diff - (g * way).sum()) <= 1e-4 * np.abs(g * way).sum(), name


@pytest.mark.gpu
def test_rows_apart(dev):
    """A row that is not finite leaves the others' results as they were, and
    spoils its own; rows of zeros stay finite."""
    import torch
    types, M, d = (F32, F32, BF16), 9, 1024
    v = case(dev, M, d, types)
    clean = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=torch.bfloat16, keep=True, **v["how"])
    v["x"][4, 100], v["x"][6] = float("nan"), 0.0
    v["f"][6] = 0.0
    say("a NaN in row 4, zeros in row 6")
    got = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=torch.bfloat16, keep=True, **v["how"])
    others = [i for i in range(M) if i not in (4, 6)]
    for a, b in zip(clean[:2], got[:2]):
        assert torch.equal(a[others], b[others])
        assert bool(b[4].isnan().any()) and not b[6].any()
    assert torch.equal(clean[2][:, others], got[2][:, others]) and bool(got[2][:, 6].isfinite().all())
    assert torch.equal(clean[3][0][others], got[3][0][others])
    assert int((got[3][1][4] == 255).sum()) == 1
    dx, df, _, _, _ = blr.blr_norm_backward(v["dn"], v["dout"], got[3], v["f"], v["w"], got[2], **v["how"])
    assert bool(dx[others].isfinite().all()) and bool(df[others].isfinite().all()) and bool(dx[6].isfinite().all())
    assert bool(dx[4].isnan().any())


@pytest.mark.gpu
def test_reruns_and_other_stream(dev):
    import torch
    types, M, d = (F32, BF16, BF16), 1500, 512
    v = case(dev, M, d, types, gate=True, span=128, kind=1)
    one = blr.blr_norm_forward(v["x"], v["f"], v["w"], keep=True, **v["how"])
    back = blr.blr_norm_backward(v["dn"], v["dout"], one[3], v["f"], v["w"], one[2], **v["how"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    say("the same on another stream")
    two = blr.blr_norm_forward(v["x"], v["f"], v["w"], keep=True, stream=s, **v["how"])
    back2 = blr.blr_norm_backward(v["dn"], v["dout"], two[3], v["f"], v["w"], two[2], stream=s, **v["how"])
    s.synchronize()
    for a, b in zip([*one[:3], *one[3], *back], [*two[:3], *two[3], *back2]):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured(dev):
    """Forward and backward replayed from one graph, eager work between."""
    import torch
    types, M, d = (F32, F32, BF16), 600, 1024
    v = case(dev, M, d, types, gate=True, span=64)
    ws = blr.workspace_norm(M, d, 64)
    out = torch.empty_like(v["x"])
    n = torch.empty((M, d), dtype=torch.bfloat16, device=dev)
    stats = torch.empty((2, M), device=dev)
    grads = [torch.empty_like(v["x"]), torch.empty_like(v["f"]), torch.empty(v["gate"].shape, device=dev),
             torch.empty(d, device=dev), torch.empty(d, device=dev)]

    def step():
        blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=n.dtype, out=out, n=n, stats=stats, **v["how"])
        blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, dx=grads[0], df=grads[1],
                              dgate=grads[2], dw=grads[3], dw_after=grads[4], ws=ws, **v["how"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    say("capture")
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        v["x"].copy_(torch.randn_like(v["x"]))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in [out, n, stats, *grads]]
        for t in [out, n, stats, *grads]:
            t.fill_(7.0)
        say(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [out, n, stats, *grads]))


@pytest.mark.gpu
@pytest.mark.parametrize("d,M", [(8, (1 << 22) + 4099), (520, (1 << 20) + 1027)])
def test_more_rows_than_a_grid_is_wide(dev, d, M):
    """Rows in the grid's second line: every row has the result that it has
    alone."""
    import torch
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((M, d), generator=g, device=dev).bfloat16()
    w = torch.randn(d, generator=g, device=dev)
    say(f"{M} rows of {d}")
    _, n, stats, _ = blr.blr_norm_forward(x, None, w)
    at = torch.cat([torch.arange(0, 700, device=dev), torch.arange(M - 6000, M, device=dev),
                    torch.randint(0, M, (20000,), generator=g, device=dev)])
    _, alone, s1, _ = blr.blr_norm_forward(x[at], None, w)
    assert torch.equal(n[at], alone) and torch.equal(stats[0][at], s1[0])
    want, r = ref.norm_before(f64(x[at]), f64(w), float(np.float32(1e-6)))
    within(f64(alone), want, np.abs(want), ROW, BF16)
    within(f64(stats[0]), 1 / np.sqrt((x.float() ** 2).mean(1).double().cpu().numpy() + float(np.float32(1e-6))),
           f64(stats[0]), 2 * ROW)


@pytest.mark.gpu
def test_parts_alone(dev):
    """Each output by itself has the bits that it has among the others."""
    import torch
    types, M, d = (F32, BF16, F16), 77, 512
    v = case(dev, M, d, types, gate=True, span=9, kind=1)
    out, n, stats, kept = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=torch.float16, keep=True, **v["how"])
    say("forward: out alone, the checkpoint with it, n without statistics")
    o = blr.blr_norm_forward(v["x"], v["f"], v["w"], need_n=False, need_stats=False, **v["how"])
    assert torch.equal(o[0], out) and o[1:] == (None, None, None)
    o = blr.blr_norm_forward(v["x"], v["f"], need_n=False, need_stats=False, keep=True, **v["how"])
    assert torch.equal(o[0], out) and all(torch.equal(a, b) for a, b in zip(o[3], kept))
    o = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=torch.float16, need_stats=False, **v["how"])
    assert torch.equal(o[1], n) and o[2] is None
    whole = blr.blr_norm_backward(v["dn"], v["dout"], kept, v["f"], v["w"], stats, **v["how"])
    say("backward: rows alone, the weights' gradients alone, dn alone from a checkpoint")
    got = blr.blr_norm_backward(v["dn"], v["dout"], kept, v["f"], v["w"], stats, grads=False, **v["how"])
    assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1]) and got[2:] == (None, None, None)
    got = blr.blr_norm_backward(v["dn"], v["dout"], kept, v["f"], v["w"], stats, need_dx=False, need_df=False, **v["how"])
    assert got[:2] == (None, None) and all(torch.equal(a, b) for a, b in zip(got[2:], whole[2:]))
    check_backward(v, types, kept, stats, M, dout=False)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,high,low", [(1, (1.0, 0.0), (0.0, 0.0)), (2, (np.inf, 1.0), (0.0, 0.0))])
def test_gates_far_out(dev, kind, high, low):
    """Gates at the ends: sigmoid 0 and 1, silu z and 0, and their slopes."""
    import torch
    v = case(dev, 4, 64, (F32, F32, F32), norm_f=False, after=False, gate=True, kind=kind)
    v["gate"][0], v["gate"][1], v["gate"][2] = 1e4, -1e4, 3e38
    v["f"].fill_(1.0)
    how = {**v["how"], "skip": 0.0, "scale": 1.0}
    out, _, stats, _ = blr.blr_norm_forward(v["x"], v["f"], None, **how)
    far = {1: (1.0, 0.0, 1.0), 2: (1e4, 0.0, 3e38)}[kind]
    for i, want in enumerate(far):
        assert torch.equal(out[i], torch.full_like(out[i], want)), i
    _, _, dz, _, _ = blr.blr_norm_backward(None, v["dout"], None, v["f"], None, None, **how)
    for i, slope in enumerate((high[1], low[1], high[1])):
        assert torch.equal(dz[i], v["dout"][i] * slope), i


@pytest.mark.gpu
def test_past_32_bits(dev):
    """More than 2^32 values: the far rows have the results that they have alone."""
    import torch
    d = 4096
    M = (1 << 32) // d + 37
    g = torch.Generator(device=dev).manual_seed(4)
    tail = [torch.randn((50, d), generator=g, device=dev).bfloat16() for _ in range(4)]

    def rows(t):
        big = torch.ones((M, d), dtype=torch.bfloat16, device=dev)
        big[-50:] = t
        return big

    w = torch.randn(d, generator=g, device=dev)
    how = dict(norm_f=True, w_after=w, skip=0.5, scale=2.0)
    say(f"norm {M}x{d}")
    x, f, dn, dout = (rows(t) for t in tail)
    out, n, stats, kept = blr.blr_norm_forward(x, f, w, keep=True, **how)
    o1, n1, s1, k1 = blr.blr_norm_forward(tail[0], tail[1], w, keep=True, **how)
    assert torch.equal(out[-50:], o1) and torch.equal(n[-50:], n1) and torch.equal(stats[:, -50:], s1)
    assert torch.equal(kept[0][-50:], k1[0]) and torch.equal(kept[1][-50:], k1[1])
    dx, df, _, _, _ = blr.blr_norm_backward(dn, dout, kept, f, w, stats, **how)
    dx1, df1, _, _, _ = blr.blr_norm_backward(tail[2], tail[3], k1, tail[1], w, s1, **how)
    assert torch.equal(dx[-50:], dx1) and torch.equal(df[-50:], df1)
