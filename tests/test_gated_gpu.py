"""The gated feed-forward against its formulas in 64 bits."""
import numpy as np
import pytest

import _block_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import say
from _operators_ref import HALF, U, within

F32, F16, BF16 = "float32", "float16", "bfloat16"
SILU, GELU = 0, 1
# roundings of act and its slope around g: the exponential (4), the inverse (3)
# and the products and sums around them
ACT = 24


def dt(name):
    import torch
    return getattr(torch, name)


def f64(t):
    return t.detach().cpu().double().numpy()


def case(dev, M, d, ff, t, ht=None, seed=0, sigma=1.0, dh_sigma=1.0):
    import torch
    g = torch.Generator(device=dev).manual_seed(seed + M + d + ff)

    def normal(shape, s, name):
        return (torch.randn(shape, generator=g, device=dev) * s).to(dt(name))

    return dict(x=normal((M, d), sigma, t), w_gate=normal((ff, d), d ** -0.5, t), w_up=normal((ff, d), d ** -0.5, t),
                dh=normal((M, ff), dh_sigma, ht or t))


def check_forward(v, kind, ht, keep=False):
    """h against the formula; g and u are sums of d exact products."""
    h, tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, h_dtype=dt(ht), keep=keep)
    x, wg, wu = f64(v["x"]), f64(v["w_gate"]), f64(v["w_up"])
    d = x.shape[1]
    (g, u), (mg, mu) = (x @ wg.T, x @ wu.T), (np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T)
    a, slope, ma, _ = ref.act(kind, g)
    # h = act(g) u: an error e of g moves act by at most 1.13 e (silu's and
    # gelu's slopes lie within +- 1.13)
    mag = 1.13 * mg * np.abs(u) + np.abs(a) * mu + ma * np.abs(u) + 1.13 * mg * mu * d * U
    within(f64(h), a * u, mag, d + ACT, ht)
    if keep:
        for i, (val, m) in enumerate(((g, mg), (u, mu))):
            q, b = tape[0][i].cpu().numpy(), tape[1][i].cpu().numpy()
            # the sums' error, then half a step; a block's step is its largest value's
            got = ref.unpack(q, b)
            step = np.ldexp(1.0, np.repeat(b.astype(int), 32, axis=1) - 133)
            assert (np.abs(got - val) <= 0.5 * step + (d + 2) * U * m).all()
            # and the step is the one of the block's largest, up to that error
            top = np.abs(val).reshape(len(val), -1, 32).max(2)
            err = ((d + 2) * U * m).reshape(len(val), -1, 32).max(2)
            s = np.ldexp(1.0, b.astype(int) - 133)
            assert (top + err >= 63.75 * s).all() and (top - err <= 127.5 * s).all()
    return h, tape


def check_backward(v, kind, tape, *, gt=None, gscale=1.0, x=None, **more):
    got = blr.blr_gated_backward(v["x"] if x is None else x, v["dh"], v["w_gate"], v["w_up"], tape, kind=kind,
                                 gscale=gscale, grad_dtype=None if gt is None else dt(gt), **more)
    t = str(v["w_gate"].dtype).split(".")[1]
    xv, dh, wg, wu = f64(v["x"]) if x is None else None, f64(v["dh"]), f64(v["w_gate"]), f64(v["w_up"])
    if isinstance(x, tuple):
        import torch
        xv = f64(blr.blr_checkpoint_load(*x, dt(t)))
    M, ff = dh.shape
    d = wg.shape[1]
    if tape is None:
        g, u = xv @ wg.T, xv @ wu.T
        mg, mu = np.abs(xv) @ np.abs(wg).T, np.abs(xv) @ np.abs(wu).T
        eg, eu = (d + 2) * U * mg, (d + 2) * U * mu
    else:
        g, u = (ref.unpack(tape[0][i].cpu().numpy(), tape[1][i].cpu().numpy()) for i in (0, 1))
        eg = eu = np.zeros_like(g)
    a, slope, ma, ms = ref.act(kind, g)
    dg, du = dh * u * slope, dh * a
    # errors of dg and du: those of g and u (slopes of act within 1.13, of its
    # slope within 1), the arithmetic, and the one rounding to 16 bits under
    # gscale, whose subnormals are absolute
    tiny = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[t] / gscale
    e_dg = np.abs(dh) * (np.abs(u) * eg + (np.abs(slope) + eg) * eu + ACT * U * ms * np.abs(u))
    e_du = np.abs(dh) * (1.13 * eg + ACT * U * ma)
    e_dg, e_du = ((1 + HALF[t]) * e + HALF[t] * np.abs(val) + tiny for e, val in ((e_dg, dg), (e_du, du)))
    want = {"dx": (dg @ wg + du @ wu, e_dg @ np.abs(wg) + e_du @ np.abs(wu),
                   np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu), 2 * ff, t)}
    if xv is not None:
        want["dw_gate"] = (dg.T @ xv, e_dg.T @ np.abs(xv), np.abs(dg).T @ np.abs(xv), M, gt or t)
        want["dw_up"] = (du.T @ xv, e_du.T @ np.abs(xv), np.abs(du).T @ np.abs(xv), M, gt or t)
    for name, out in zip(("dx", "dw_gate", "dw_up"), got):
        if out is None:
            continue
        value, err, mag, terms, ot = want[name]
        say(f"  {name} {ot}")
        # the errors of the factors enter as a part of the bound, the rest is
        # the sum's (`within` multiplies its third argument by terms U)
        n = (terms + 4) * U
        within(f64(out), value, (mag + err) + err * (1 + HALF[ot]) / n, terms + 4, ot)
    return got


SHAPES = [(1, 128, 128), (2, 256, 384), (16, 128, 640), (17, 384, 256), (63, 256, 128), (64, 640, 512), (65, 128, 256),
          (127, 256, 256), (129, 384, 128), (300, 512, 640), (257, 128, 384)]


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,d,ff", SHAPES)
def test_forward(dev, t, M, d, ff):
    for kind in (SILU, GELU):
        for ht in (t, F32):
            say(f"gated {t} -> {ht} kind={kind} {M}x{d}x{ff}")
            check_forward(case(dev, M, d, ff, t), kind, ht, keep=True)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,d,ff", SHAPES)
def test_backward(dev, t, M, d, ff):
    for kind, ht, gt, kept in ((SILU, t, t, True), (GELU, F32, F32, False), (GELU, t, F32, True), (SILU, F32, t, False)):
        say(f"gated backward {t} dh={ht} grads={gt} kind={kind} tape={kept} {M}x{d}x{ff}")
        v = case(dev, M, d, ff, t, ht, dh_sigma=1e-2)
        tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, keep=True)[1] if kept else None
        check_backward(v, kind, tape, gt=gt, gscale=64.0 if t == F16 else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,ff", [(200, 256, 5504), (130, 128, 8192), (700, 256, 4224)])
def test_middle_tiles(dev, M, d, ff):
    """Rows between the smallest tiles' and the largest's."""
    v = case(dev, M, d, ff, BF16, dh_sigma=1e-2)
    say(f"gated {M}x{d}x{ff}")
    _, tape = check_forward(v, GELU, BF16, keep=True)
    check_backward(v, GELU, None)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M,d,ff", [(2100, 1024, 2176), (4200, 2176, 1024)])
def test_large_tiles(dev, t, M, d, ff):
    """Shapes whose contractions take the tiles of 256, ragged in rows and in
    columns; rows are checked at the tiles' edges and everywhere by the sums."""
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    say(f"gated {t} {M}x{d}x{ff}")
    _, tape = check_forward(v, SILU, t, keep=True)
    check_backward(v, SILU, tape, gscale=64.0 if t == F16 else 1.0)
    check_backward(v, SILU, None, gscale=64.0 if t == F16 else 1.0)


@pytest.mark.gpu
def test_x_from_its_checkpoint(dev):
    import torch
    M, d, ff, t = 200, 256, 384, BF16
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    kept = blr.blr_checkpoint_save(v["x"])
    tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], keep=True)[1]
    for tp in (None, tape):
        say(f"x in 8 bits, projections {'again' if tp is None else 'kept'}")
        check_backward(v, SILU, tp, x=kept)
    say("dx alone, from the tape, without x")
    dx = blr.blr_gated_backward(None, v["dh"], v["w_gate"], v["w_up"], tape, grads=False)[0]
    both = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape)
    assert torch.equal(dx, both[0])
    alone = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape, need_dx=False)
    assert alone[0] is None and torch.equal(alone[1], both[1]) and torch.equal(alone[2], both[2])


@pytest.mark.gpu
def test_small_gradients_in_f16(dev):
    """dh of 1e-6: without a scale dg and du are subnormal in f16, under 2^14
    they keep their 11 bits."""
    v = case(dev, 130, 256, 256, F16, F32, dh_sigma=1e-6)
    say("dh of 1e-6 in f16, gscale 2^14")
    check_backward(v, SILU, None, gt=F32, gscale=2.0 ** 14)


@pytest.mark.gpu
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("ff", [256, 2176])
def test_accumulates(dev, gt, ff):
    """Also where dx's contraction, over 2 ff, is made in several splits."""
    M, d, t = 150, 384, BF16
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    say(f"gradients added to what is there, {gt}")
    one = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], grad_dtype=dt(gt))
    exact = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], grad_dtype=dt(F32))
    two = [o.clone() for o in one]
    blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], dx=two[0], accumulate_dx=True, dw_gate=two[1],
                           dw_up=two[2], accumulate_grads=True)
    for i in (1, 2):  # the f32 product added to the stored value, rounded once
        want = f64(one[i]) + f64(exact[i])
        within(f64(two[i]), want, np.abs(f64(one[i])) + np.abs(f64(exact[i])), 2, gt)
    # dx: the second product is the first's before its rounding
    want = 2 * f64(one[0])
    assert (np.abs(f64(two[0]) - want) <= HALF[t] * np.abs(f64(one[0])) + HALF[t] * 1.01 * np.abs(want) + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [SILU, GELU])
def test_far_out(dev, kind):
    """Projections of any size: act and slope stay what they tend to; a row
    that is not finite spoils no other."""
    import torch
    M, d, ff, t = 70, 128, 128, BF16
    v = case(dev, M, d, ff, t)
    clean = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, keep=True)
    v["x"][3] *= 1e4
    v["x"][5] *= -1e18
    say(f"rows of 1e4 and 1e18, kind {kind}")
    h, tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, h_dtype=torch.float32, keep=True)
    x, wg, wu = f64(v["x"]), f64(v["w_gate"]), f64(v["w_up"])
    g, u = x @ wg.T, x @ wu.T
    a = ref.act(kind, g)[0]
    big = np.abs(a[3] * u[3]) > 0
    assert (np.abs(f64(h)[3] - a[3] * u[3])[big] <= 1e-3 * (np.abs(x[3]) @ np.abs(wu).T * np.maximum(np.abs(a[3]), 1))[big]).all()
    assert bool(h[5].isfinite().all())  # 1e36 at most
    for tp in (tape, None):
        dx, dwg, dwu = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tp, kind=kind)
        assert bool(dx[3].isfinite().all()) and bool(dx[5].isfinite().all()) and bool(dwu.isfinite().all())
    v["x"][9, 7] = float("nan")
    h2, tape2 = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, keep=True)
    others = [i for i in range(M) if i not in (3, 5, 9)]
    assert torch.equal(h2[others], clean[0][others]) and bool(h2[9].isnan().all())
    assert bool((tape2[1][:, 9] == 255).all())
    dx = blr.blr_gated_backward(None, v["dh"], v["w_gate"], v["w_up"], tape2, kind=kind, grads=False)[0]
    assert bool(dx[others].isfinite().all()) and bool(dx[9].isnan().all())


@pytest.mark.gpu
def test_gradients_against_differences(dev):
    """dx and the weights' gradients against differences of the formula."""
    M, d, ff, t = 5, 128, 128, BF16
    for kind in (SILU, GELU):
        v = case(dev, M, d, ff, t, F32)
        got = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], kind=kind, grad_dtype=dt(F32))
        base = {k: f64(v[k]) for k in ("x", "w_gate", "w_up")}
        dh = f64(v["dh"])

        def loss(at):
            g, u = at["x"] @ at["w_gate"].T, at["x"] @ at["w_up"].T
            return (dh * ref.act(kind, g)[0] * u).sum()

        rng = np.random.default_rng(1)
        for name, g in zip(("x", "w_gate", "w_up"), got):
            way = rng.standard_normal(base[name].shape)
            s = 1e-5
            diff = (loss({**base, name: base[name] + s * way}) - loss({**base, name: base[name] - s * way})) / (2 * s)
            # dg and du are of bf16: each is off by at most 2^-8 of itself, dx once more
            assert abs(diff - (f64(g) * way).sum()) <= 2.0 ** -7 * (np.abs(f64(g)) * np.abs(way)).sum(), (kind, name)


@pytest.mark.gpu
def test_reruns_streams_and_rows_behind(dev):
    """The same bits again, on another stream too, and nothing written behind
    the last row."""
    import torch
    M, d, ff, t = 333, 512, 640, F16
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    room = torch.full((M + 40, ff), 7.0, dtype=dt(t), device=dev)
    h, tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], h=room[:M], keep=True)
    back = torch.full((M + 40, d), 7.0, dtype=dt(t), device=dev)
    one = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape, dx=back[:M], gscale=16.0)
    torch.cuda.synchronize()
    assert bool((room[M:] == 7).all()) and bool((back[M:] == 7).all())
    s = torch.cuda.Stream()
    say("again, on another stream")
    h2, tape2 = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], keep=True, stream=s)
    two = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape2, gscale=16.0, stream=s)
    s.synchronize()
    for a, b in zip([h, *tape, *one], [h2, *tape2, *two]):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 300])
def test_captured(dev, M):
    """Forward and backward replayed from a graph, with eager work between."""
    import torch
    d, ff, t = 256, 384, BF16
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    h = torch.empty((M, ff), dtype=dt(t), device=dev)
    tape = (torch.empty((2, M, ff), dtype=torch.int8, device=dev), torch.empty((2, M, ff // 32), dtype=torch.uint8, device=dev))
    out = [torch.empty((M, d), dtype=dt(t), device=dev), *(torch.empty((ff, d), dtype=dt(t), device=dev) for _ in "gu")]
    ws = blr.workspace_gated(M, d, ff)

    def step():
        blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], h=h, tape=tape)
        blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape, dx=out[0], dw_gate=out[1], dw_up=out[2],
                               ws=ws)

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
        v["x"].copy_(torch.randn_like(v["x"].float()).to(v["x"].dtype))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in [h, *tape, *out]]
        for o in [h, *tape, *out]:
            o.zero_()
        say(f"replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [h, *tape, *out]))


@pytest.mark.gpu
def test_past_32_bits(dev):
    """More than 2^32 values of h: the far rows against the formula, and nothing
    of the rows before them, which are zero, in the weights' gradients."""
    import torch
    d, ff, t = 128, 16384, BF16
    M = (1 << 32) // ff + 91
    v = case(dev, 60, d, ff, t, dh_sigma=1e-2)
    x = torch.zeros((M, d), dtype=dt(t), device=dev)
    dh = torch.zeros((M, ff), dtype=dt(t), device=dev)
    x[-60:], dh[-60:] = v["x"], v["dh"]
    say(f"gated {M}x{d}x{ff}")
    h, tape = blr.blr_gated_forward(x, v["w_gate"], v["w_up"], keep=True)
    h1, tape1 = check_forward(v, SILU, t, keep=True)
    assert not bool(h[:-60].any())
    got, one = h[-60:].double(), h1.double()
    assert bool(((got - one).abs() <= 2 * HALF[t] * one.abs() + 1e-6).all())  # a sum's order may round it the other way
    q, b = tape[0][:, -60:], tape[1][:, -60:]
    assert int((b != tape1[1]).sum()) <= 4 and int((q.int() - tape1[0].int()).abs().max()) <= 64
    say("backward")
    dx, dwg, dwu = blr.blr_gated_backward(x, dh, v["w_gate"], v["w_up"], tape)
    dx1, dwg1, dwu1 = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], (q.contiguous(), b.contiguous()))
    assert not bool(dx[:-60].any())
    for a, c in ((dx[-60:], dx1), (dwg, dwg1), (dwu, dwu1)):
        a, c = a.double(), c.double()
        assert bool(((a - c).abs() <= 2 * HALF[t] * c.abs() + 1e-5 * c.abs().max()).all())
