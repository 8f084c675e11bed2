"""The adapters' workspaces: a forward needs its own, not the backward's."""
import ctypes

import pytest

import binary_rank_linear_amd as blr
from test_operators_abi import BIG, E_DEV, E_HIP, E_OVERLAP, E_WS, at, backward, forward

MIB = 1 << 20


def sizes(*args):
    lib = blr.load()
    return lib.blr_adapters_forward_workspace_bytes(*args), lib.blr_adapters_workspace_bytes(*args)


@pytest.mark.parametrize("M", [1, 64, 700, 8192, 100000])
@pytest.mark.parametrize("r", [8, 64, 128])
def test_forward_needs_no_room_for_the_adapters(M, r):
    """At most 32 partials of s, or a megabyte, however many adapters there
    are and however wide; never more than both calls need."""
    for d_in, d_out in [(128, 128), (4096, 12288), (128, 1 << 20), (1 << 20, 128)]:
        for E in (1, 32, 1024):
            own, both = sizes(M, d_in, d_out, r, E)
            assert 0 < own <= max(32 * 4 * M * r + 256, MIB) and own <= both, (d_in, d_out, E)
    assert sizes(1, 4096, 12288, 64, 1024)[0] <= MIB  # 4 GB with the backward's


def test_invalid_sizes_have_none():
    for bad in [(0, 128, 128, 8, 1), (1, 64, 128, 8, 1), (1, 128, 128, 4, 1), (1, 128, 128, 8, 1025)]:
        assert sizes(*bad) == (0, 0)


@pytest.mark.parametrize("M,d_in,d_out,r,E", [(64, 256, 128, 16, 4), (64, 4096, 4096, 16, 1024),
                                             (8192, 4096, 12288, 64, 8)])
def test_each_call_checks_its_own(M, d_in, d_out, r, E):
    import torch
    own, both = sizes(M, d_in, d_out, r, E)
    size = dict(M=M, d_in=d_in, d_out=d_out, r=r, E=E)
    assert forward(ws_bytes=own - 1, **size) == E_WS
    assert backward(ws_bytes=both - 1, **size) == E_WS
    # y beside the workspace's end, and on it
    y = ctypes.c_void_p(at(20).value + own)
    assert forward(ws=at(20), ws_bytes=BIG, y=ctypes.c_void_p(y.value - 16), **size) == E_OVERLAP
    if not torch.cuda.is_available():  # what passes the checks ends at the device's
        assert forward(ws=at(20), ws_bytes=own, y=y, **size) in (E_DEV, E_HIP)
        assert backward(ws_bytes=both, **size) in (E_DEV, E_HIP)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d_in,d_out,r,E", [(1, 256, 384, 16, 1024), (700, 2048, 128, 24, 3), (3000, 4096, 256, 64, 5)])
def test_forward_in_its_own_workspace(dev, M, d_in, d_out, r, E):
    """The least that it accepts, between guards, gives the bits of the larger
    one; without a workspace the call takes no more than that and its y."""
    import torch
    from _gpu_util import say
    say(f"adapters forward in its own workspace M={M} {d_in}->{d_out} r={r} E={E}")
    torch.manual_seed(M)
    x, down, up = (torch.randn(s, device=dev) for s in ((M, d_in), (E, r, d_in), (E, d_out, r)))
    offsets, order, _ = blr.blr_route_sort(torch.randint(0, E, (M,), device=dev).int(), E)
    want = blr.blr_adapters_forward(x, down, up, offsets, order, keep_tape=True,
                                    ws=blr.workspace_adapters(M, d_in, d_out, r, E, dev))
    need = blr.workspace_adapters(M, d_in, d_out, r, E, dev, forward=True).numel()
    assert need == sizes(M, d_in, d_out, r, E)[0]
    whole = torch.full((need + 8192,), 7, dtype=torch.uint8, device=dev)
    got = blr.blr_adapters_forward(x, down, up, offsets, order, keep_tape=True, ws=whole[4096:4096 + need])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (whole[:4096] == 7).all() and (whole[-4096:] == 7).all()
    with pytest.raises(blr.BlrError):
        blr.blr_adapters_forward(x, down, up, offsets, order, ws=whole[:need - 16])
    del got, whole
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    # what was asked for, not the blocks that it came in, whose remainders the allocator may leave undivided
    asked = lambda when: torch.cuda.memory_stats()[f"requested_bytes.all.{when}"]  # noqa: E731
    before = asked("current")
    y, _ = blr.blr_adapters_forward(x, down, up, offsets, order)
    assert asked("peak") - before <= need + y.numel() * 4
    assert torch.equal(y, want[0])
