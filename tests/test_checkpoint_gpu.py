"""Rows kept in 8 bits against their definition: every q and b equal, loads
exact (they are one power of two times a whole number of 8 bits)."""
import numpy as np
import pytest

import _block_ref as ref
import binary_rank_linear_amd as blr
from _gpu_util import say


def torch_dtype(name):
    import torch
    return getattr(torch, name)


def as_f64(t):
    return t.detach().cpu().double().numpy()


def edge_rows(dtype):
    """Blocks at every border: zeros, subnormals, values just under and over a
    power of two and under 127.5 steps, ties, the type's largest, one value
    that is not finite."""
    import torch
    t = torch_dtype(dtype)
    fi = torch.finfo(t)
    rng = np.random.default_rng(5)
    rows = [np.zeros(32), rng.standard_normal(32), np.full(32, -1.0)]
    for top in (1.0, 2.0 - 2.0 ** -7, 2.0 - 2.0 ** -6, 1.9921875, 1.99, 127.0, 127.5, 128.0, 2.0 ** -14, 2.0 ** -20):
        r = rng.uniform(-1, 1, 32) * top
        r[7] = -top
        rows.append(r)
    tie = (np.arange(32) - 16.0) + 0.5  # half steps of the block whose largest is 127
    tie[0] = 127.0
    rows.append(tie)
    for v in (fi.max, fi.max / 2, fi.tiny, fi.tiny / 4, fi.smallest_normal * fi.eps):
        r = rng.uniform(-1, 1, 32) * v
        r[31] = v
        rows.append(r)
    for v in (np.inf, -np.inf, np.nan):
        r = rng.standard_normal(32)
        r[rng.integers(32)] = v
        rows.append(r)
    return torch.from_numpy(np.stack(rows)).to(t)


def check(x, dtype):
    import torch
    q, b = blr.blr_checkpoint_save(x)
    back = blr.blr_checkpoint_load(q, b, x.dtype)
    torch.cuda.synchronize()
    want_q, want_b = ref.pack(as_f64(x), dtype)
    assert np.array_equal(b.cpu().numpy(), want_b)
    assert np.array_equal(q.cpu().numpy(), want_q)
    values = ref.unpack(want_q, want_b)
    assert np.array_equal(as_f64(back), values, equal_nan=True)
    fine = np.repeat(want_b, 32, axis=1) < ref.MOST[dtype]
    half = np.ldexp(0.5, np.repeat(want_b.astype(int), 32, axis=1) - 133)
    assert (np.abs(values - as_f64(x))[fine] <= half[fine]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_borders(dev, dtype):
    x = edge_rows(dtype).to(dev)
    say(f"checkpoint borders {dtype}")
    check(x, dtype)                              # a block a row
    check(x.reshape(1, -1).contiguous(), dtype)  # all in one row


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("M,d", [(1, 32), (3, 96), (67, 1056), (5, 4096)])
def test_rows(dev, dtype, M, d):
    import torch
    g = torch.Generator(device=dev).manual_seed(M + d)
    x = (torch.randn((M, 1), generator=g, device=dev).mul(3).exp() * torch.randn((M, d), generator=g, device=dev))
    say(f"checkpoint {dtype} {M}x{d}")
    check(x.clamp(-6e4, 6e4).to(torch_dtype(dtype)), dtype)


@pytest.mark.gpu
def test_other_type_on_load(dev):
    """A checkpoint of f32 rows read as 16 bits: one rounding to nearest."""
    import torch
    x = edge_rows("float32").to(dev)
    q, b = blr.blr_checkpoint_save(x)
    full = blr.blr_checkpoint_load(q, b, torch.float32)
    for t in (torch.float16, torch.bfloat16):
        say(f"f32 checkpoint read as {t}")
        got = blr.blr_checkpoint_load(q, b, t)
        assert torch.equal(torch.nan_to_num(got.float(), 7.0, 1e38, -1e38),
                           torch.nan_to_num(full.to(t).float(), 7.0, 1e38, -1e38))


@pytest.mark.gpu
def test_past_32_bits(dev):
    """More than 2^32 values: the far end is addressed right."""
    import torch
    M, d = (1 << 32) // 4096 + 3, 4096
    x = torch.zeros((M, d), dtype=torch.bfloat16, device=dev)
    x[-3:] = torch.randn((3, d), device=dev).bfloat16()
    say(f"checkpoint {M}x{d}")
    q, b = blr.blr_checkpoint_save(x)
    want_q, want_b = ref.pack(as_f64(x[-3:]), "bfloat16")
    assert np.array_equal(q[-3:].cpu().numpy(), want_q) and np.array_equal(b[-3:].cpu().numpy(), want_b)
    assert not bool(q[:-3].any())
    back = blr.blr_checkpoint_load(q, b, torch.bfloat16)
    assert np.array_equal(as_f64(back[-3:]), ref.unpack(want_q, want_b))
