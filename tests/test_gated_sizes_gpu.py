"""The gated feed-forward's gradients in the tiles of 256, in every type and
added to what is there; projections of any size; f16 past its range; the tape
past 2^32 values."""
import numpy as np
import pytest

import _block_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import say
from _operators_ref import HALF
from test_gated_gpu import BF16, F16, F32, GELU, SILU, case, check_backward, check_forward, dt, f64


def tiles(m, n, b):
    return -(-m // b) * -(-n // b)


def takes_256(m, n):
    """The rule: a round of one tile of 256 on every CU takes 1.6 of one of two
    tiles of 128."""
    return 8 * -(-tiles(m, n, 256) // 256) <= 5 * -(-tiles(m, n, 128) // 512)


def check_added(v, one, **how):
    """Gradients of the same call added to `one`: f32 is doubled exactly, 16 bits
    to within the two roundings."""
    import torch
    two = [o.clone() for o in one]
    blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], dx=two[0], accumulate_dx=True, dw_gate=two[1],
                           dw_up=two[2], accumulate_grads=True, **how)
    for a, b in zip(one, two):
        if a.dtype == torch.float32:
            assert torch.equal(a * 2, b)
        else:  # the stored value is the product rounded, and the sum is rounded again
            t = str(a.dtype).split(".")[1]
            want, half = 2 * f64(a), HALF[t]
            tiny = 2.0 ** -24 if t == F16 else 2.0 ** -133
            assert (np.abs(f64(b) - want) <= half * np.abs(f64(a)) + half * 1.01 * np.abs(want) + tiny).all()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("M", [1, 64, 100, 321])
def test_weights_gradients_in_large_tiles(dev, t, M):
    """Contractions of one to six steps, the last one short, columns that end
    inside a tile."""
    d, ff = 3968, 2048
    assert takes_256(2 * ff, d) and d % 256
    for gt in (F32, t):
        v = case(dev, M, d, ff, t, dh_sigma=1e-2)
        say(f"weights' gradients {t} -> {gt} {M}x{d}x{ff}")
        g = 64.0 if t == F16 else 1.0
        one = check_backward(v, SILU, None, gt=gt, gscale=g)
        check_added(v, one, kind=SILU, gscale=g)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [F16, BF16])
def test_dx_in_large_tiles(dev, t):
    M, d, ff = 4200, 2176, 256
    assert takes_256(M, d) and M % 256 and d % 256
    v = case(dev, M, d, ff, t, dh_sigma=1e-2)
    say(f"dx {t} {M}x{d}x{ff}")
    g = 64.0 if t == F16 else 1.0
    one = check_backward(v, GELU, None, gt=F32, gscale=g)
    check_added(v, one, kind=GELU, gscale=g)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [SILU, GELU])
@pytest.mark.parametrize("kept", [False, True])
def test_gradients_of_far_rows(dev, kind, kept):
    """Rows of 1e4 and 1e18: every gradient is finite and that of the formula.
    dg and du are off by a half step of bf16, results once more, and what f32
    loses in sums of 128 products is far below: 2^-6 in all, in the 2-norm."""
    M, d, ff, t = 70, 128, 128, BF16
    v = case(dev, M, d, ff, t)
    v["x"][3] *= 1e4
    v["x"][5] *= -1e18
    tape = blr.blr_gated_forward(v["x"], v["w_gate"], v["w_up"], kind=kind, keep=True)[1] if kept else None
    say(f"gradients of rows of 1e4 and 1e18, kind {kind} kept {kept}")
    got = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], tape, kind=kind)
    x, dh, wg, wu = (f64(v[k]) for k in ("x", "dh", "w_gate", "w_up"))
    g, u = (x @ wg.T, x @ wu.T) if tape is None else \
        (ref.unpack(tape[0][i].cpu().numpy(), tape[1][i].cpu().numpy()) for i in (0, 1))
    a, slope, _, _ = ref.act(kind, g)
    dg, du = dh * u * slope, dh * a
    for name, o, want in zip(("dx", "dw_gate", "dw_up"), got, (dg @ wg + du @ wu, dg.T @ x, du.T @ x)):
        o = f64(o)
        assert np.isfinite(o).all(), name
        assert np.linalg.norm(o - want) <= 2.0 ** -6 * np.linalg.norm(want), name
    # the rows between them, on their own
    for i in (0, 3, 5, 69):
        want = dg[i] @ wg + du[i] @ wu
        assert np.linalg.norm(f64(got[0])[i] - want) <= 2.0 ** -6 * np.linalg.norm(want), i


@pytest.mark.gpu
def test_f16_past_its_range(dev):
    """dg or du times gscale past f16's largest value is infinite: it spoils its
    own row of dx, and the weights' gradients, which shows that gscale is too
    large; under a smaller one all are right."""
    import torch
    M, d, ff = 40, 128, 256
    v = case(dev, M, d, ff, F16, F32, dh_sigma=1e-2)
    v["dh"][3] *= 1e5  # to about 3000, and dg and du to about 10^4
    say("f16 under gscale 2^8")
    dx, dwg, dwu = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], gscale=256.0)
    others = [i for i in range(M) if i != 3]
    assert not bool(dx[3].isfinite().any()) and bool(dx[others].isfinite().all())
    assert not bool(dwg.isfinite().all()) and not bool(dwu.isfinite().all())
    say("f16 under gscale 2^-2")
    # in f32, which holds the gradients
    got = check_backward(v, SILU, None, gt=F32, gscale=0.25, need_dx=False)
    assert got[0] is None and bool(got[1].isfinite().all()) and bool(got[2].isfinite().all())
    dx2 = blr.blr_gated_backward(v["x"], v["dh"], v["w_gate"], v["w_up"], gscale=0.25, grads=False)[0]
    assert bool(dx2.isfinite().all())


@pytest.mark.gpu
def test_tape_past_32_bits(dev):
    """More than 2^32 values: the far rows' bytes are those of the rows alone. A
    sum's order may move a value over a rounding's border, by one step, or a
    block's largest over its own, which doubles or halves the step."""
    import torch
    d, ff, t = 128, 16384, BF16
    M = (1 << 32) // ff + 91
    v = case(dev, 60, d, ff, t)
    x = torch.zeros((M, d), dtype=dt(t), device=dev)
    x[-60:] = v["x"]
    say(f"tape {M}x{d}x{ff}")
    q, b = blr.blr_gated_forward(x, v["w_gate"], v["w_up"], keep=True)[1]
    assert not bool(q[:, :-60].any()) and not bool(b[:, :-60].any())
    _, (q1, b1) = check_forward(v, SILU, t, keep=True)
    q, b = q[:, -60:].cpu().numpy().astype(int), b[:, -60:].cpu().numpy().astype(int)
    q1, b1 = q1.cpu().numpy().astype(int), b1.cpu().numpy().astype(int)
    same = np.repeat(b == b1, 32, axis=-1)
    assert np.abs(q - q1)[same].max() <= 1 and (q != q1)[same].mean() <= 1e-3
    assert (b != b1).sum() <= 4
    step = np.ldexp(1.0, np.repeat(np.maximum(b, b1), 32, axis=-1) - 133)
    assert (np.abs(ref.unpack(q, b) - ref.unpack(q1, b1)) <= step).all()
