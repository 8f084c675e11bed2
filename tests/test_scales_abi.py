"""Scales and sizes at the ends of their ranges are refused before any device
work (no GPU: a call that passes its checks fails for want of one)."""
import ctypes

import binary_rank_linear_amd as blr
from test_abi import E_SCALE, bwd, ptrs  # noqa: F401  (ptrs: a fixture)
from test_block_abi import FWD, NO_GPU, call, gated_backward
from test_operators_abi import F32

# the least power of two whose inverse f32 holds is 2^-127; 2^-149 is f32's least
SMALLEST, TOO_SMALL = 2.0 ** -127, (2.0 ** -128, 2.0 ** -140, 2.0 ** -149)


def plane(scale, ptrs):
    return blr.load().blr_plane_linear(128, 256, 256, ptrs["x"], ptrs["bu"], ptrs["y"], ctypes.c_float(scale), None)


def test_a_scale_without_an_inverse(ptrs):  # noqa: F811
    """The products are divided by the scale: with 2^-128 or less the inverse is
    infinite, and results would be infinite or NaN."""
    lib = blr.load()
    for s in TOO_SMALL:
        assert gated_backward(gscale=s) == E_SCALE, s
        assert bwd(lib, 128, 256, 256, 128, ptrs, gscale=s) == E_SCALE, s
        assert plane(s, ptrs) == E_SCALE, s
    for s in (SMALLEST, 2.0 ** -126, 1.0, 2.0 ** 127):
        assert gated_backward(gscale=s) in NO_GPU, s
        assert bwd(lib, 128, 256, 256, 128, ptrs, gscale=s) in NO_GPU, s
        assert plane(s, ptrs) in NO_GPU, s


def test_eps():
    """1 / sqrt(mean + eps) has no value for an eps below zero or NaN, and only
    zero for an infinite one."""
    def norm(eps):
        return call("blr_norm_forward", (4, 64, F32, F32, F32, "x", None, 0, None, None, 0, 1, ctypes.c_float(1),
                                         ctypes.c_float(1), "w", ctypes.c_float(eps), None, "n", "stats", None, None),
                    FWD, {})

    for eps in (-1e-6, -1.0, float("nan"), float("inf"), float("-inf")):
        assert norm(eps) == E_SCALE, eps
    for eps in (0.0, -0.0, 1e-45, 1e-6, 1.0):
        assert norm(eps) in NO_GPU, eps
