"""The norms' backward where a team of waves takes several rows: sums kept over
rows, gates that begin, end or go on within its range, and the sums of ranges."""
import pytest

import binary_rank_linear_amd as blr
from _gpu_util import say
from test_norm_gpu import BF16, F16, F32, case, check_backward, check_forward, dt

CUS, MAX_WAVES = 256, 16


def per_range(M, d):
    """Rows of a range: those of M over all teams that are on the chip at once,
    16 waves to a CU, a team's rows 512 columns a wave (1024 past 8192)."""
    waves = -(-d // (512 if d <= 8192 else 1024))
    return -(-M // (CUS * (MAX_WAVES // waves)))


# (rows, columns, rows of a gate or 0 without one, rows of a range at least)
SHAPES = [(1100, 8192, 1, 5), (1100, 8192, 2, 5), (1100, 8192, 3, 5), (1100, 8192, 7, 5), (1100, 8192, 300, 5),
          (1100, 8192, 5, 5), (1100, 8192, 1100, 5), (1100, 8192, 0, 5), (2100, 4096, 0, 5), (2100, 4096, 1, 5),
          (2100, 4096, 2, 5), (2100, 4096, 64, 5), (700, 8200, 1, 3), (700, 8200, 2, 3), (700, 8200, 0, 3),
          (1024, 6144, 2, 4), (1025, 6152, 3, 5), (13000, 256, 2, 4), (13000, 256, 0, 4), (13001, 256, 3, 4),
          (13001, 520, 6000, 7), (16385, 8, 4, 5), (9000, 1032, 5, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,span,per", SHAPES)
def test_several_rows_to_a_range(dev, M, d, span, per):
    assert per_range(M, d) >= per
    for types in ((F32, BF16, F32), (F16, F16, F16)) if d < 4096 else ((F32, F32, BF16),):
        say(f"norm backward {types} {M}x{d} span={span}")
        v = case(dev, M, d, types, gate=span > 0, kind=2, span=max(span, 1))
        out, stats, _ = check_forward(v, types, False)
        check_backward(v, types, out, stats, M)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,span", [(1100, 8192, 3), (2100, 4096, 2), (13000, 256, 2), (700, 8200, 2), (5, 256, 3),
                                      (1100, 8192, 300)])
def test_added_to_what_is_there(dev, M, d, span):
    """Gates written whole from one range, and joined from several: either adds."""
    import torch
    types = (F32, F32, F32)
    v = case(dev, M, d, types, gate=True, span=span, kind=1)
    out, stats, _ = check_forward(v, types, False)
    say(f"added to what is there {M}x{d} span={span}")
    first = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
    sums = [t.clone() for t in first[2:]]
    blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, dgate=sums[0], dw=sums[1], dw_after=sums[2],
                          accumulate_grads=True, **v["how"])
    for a, b in zip(first[2:], sums):
        assert torch.equal(a * 2, b)  # doubling is exact
    v["dout"].zero_(), v["dn"].zero_()
    blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, dgate=sums[0], dw=sums[1], dw_after=sums[2],
                          accumulate_grads=True, **v["how"])
    for a, b in zip(first[2:], sums):
        assert torch.equal(a * 2, b)  # gradients of zero add nothing


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,span", [(1100, 8192, 3), (2100, 4096, 0), (13000, 256, 2)])
def test_from_checkpoints(dev, M, d, span):
    """Both rows in 8 bits, several rows to a range."""
    types = (F32, BF16, BF16)
    v = case(dev, M, d, types, gate=span > 0, kind=1, span=max(span, 1))
    say(f"from checkpoints {M}x{d} span={span}")
    _, stats, kept = blr.blr_norm_forward(v["x"], v["f"], v["w"], n_dtype=dt(BF16), keep=True, **v["how"])[1:]
    check_backward(v, types, kept, stats, M, f=blr.blr_checkpoint_save(v["f"]))


@pytest.mark.gpu
def test_rows_of_a_range_do_not_touch(dev):
    """A row that is not finite in the middle of a range: the rows after it have
    the bits that they have without it."""
    import torch
    M, d, types = 2100, 4096, (F32, F32, F32)
    for gate in (False, True):
        v = case(dev, M, d, types, gate=gate, kind=2)
        out, _, stats, _ = blr.blr_norm_forward(v["x"], v["f"], v["w"], **v["how"])
        clean = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
        bad = torch.arange(2, M, 5, device=dev)
        v["dn"][bad, 17] = float("nan")
        v["dout"][bad, 4000] = float("inf")
        say(f"rows that are not finite, gate {gate}")
        got = blr.blr_norm_backward(v["dn"], v["dout"], out, v["f"], v["w"], stats, **v["how"])
        good = torch.ones(M, dtype=torch.bool, device=dev)
        good[bad] = False
        for a, b in zip(clean[:3], got[:3]):
            if a is not None:
                assert torch.equal(a[good], b[good])
        assert bool(got[0][bad].isnan().any(1).all())
