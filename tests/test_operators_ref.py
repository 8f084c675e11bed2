"""The plain 64-bit forms that the routing and adapter tests use, against
finite differences and hand-worked values (no GPU)."""
import numpy as np
import pytest

import _operators_ref as ref


def test_sort_by_hand():
    offsets, order, slot = ref.sort(np.array([[2, 0], [-1, 2], [0, 9]], np.int32), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 4, 0, 3, 2, 5]
    assert slot.tolist() == [[2, 0], [4, 3], [1, 5]]


def loss(x, A, B, ids, c, dy):
    (_, y), _ = ref.adapters_forward(x, A, B, ids, c)
    return float((dy * y).sum())


def test_adapter_gradients_against_differences():
    """The loss is linear in each of x, A and B, so central differences are
    exact for any step, up to 64-bit rounding."""
    rng = np.random.default_rng(5)
    M, d_in, d_out, r, E = 7, 6, 5, 3, 4
    x, dy = rng.standard_normal((M, d_in)), rng.standard_normal((M, d_out))
    A, B = rng.standard_normal((E, r, d_in)), rng.standard_normal((E, d_out, r))
    c = rng.uniform(0.5, 2.0, E)
    ids = np.array([0, 2, 0, -1, 2, 3, 0])
    (s, _), _ = ref.adapters_forward(x, A, B, ids, c)
    (gA, gB, dx), _ = ref.adapters_backward(x, dy, A, B, ids, c, s)
    for arr, g in ((x, dx), (A, gA), (B, gB)):
        v = rng.standard_normal(arr.shape)
        keep = arr.copy()
        arr += v
        up = loss(x, A, B, ids, c, dy)
        arr -= 2 * v
        down = loss(x, A, B, ids, c, dy)
        arr[...] = keep
        assert (up - down) / 2 == pytest.approx(float((g * v).sum()), rel=1e-10)
    assert not gA[1].any() and not gB[1].any() and not dx[3].any()


def test_combine_gradients_against_differences():
    rng = np.random.default_rng(6)
    T, k, E, d = 5, 3, 4, 6
    ids = rng.integers(-1, E, (T, k))
    offsets, _, slot = ref.sort(ids, E)
    z, w, dy = rng.standard_normal((T * k, d)), rng.standard_normal((T, k)), rng.standard_normal((T, d))
    dz, dw, _ = ref.combine_backward(dy, z, offsets, slot, w)
    f = lambda z, w: float((dy * ref.combine(z, offsets, slot, w)[0]).sum())  # noqa: E731
    vz, vw = rng.standard_normal(z.shape), rng.standard_normal(w.shape)
    assert (f(z + vz, w) - f(z - vz, w)) / 2 == pytest.approx(float((dz * vz).sum()), rel=1e-10)
    assert (f(z, w + vw) - f(z, w - vw)) / 2 == pytest.approx(float((dw * vw).sum()), rel=1e-10)
    # the gather's gradient is the combine with weights of one
    g = rng.standard_normal((T * k, d))
    x, v = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    diff = ((ref.gather(x + v, offsets, slot) - ref.gather(x - v, offsets, slot)) * g).sum() / 2
    assert diff == pytest.approx(float((ref.combine(g, offsets, slot)[0] * v).sum()), rel=1e-10)


def test_the_bound_sees_a_wrong_element():
    want = np.array([1.0, -2.0])
    ref.within(want * (1 + 2.0 ** -25), want, np.abs(want), 4)
    with pytest.raises(AssertionError):
        ref.within(want + np.array([0, 1e-4]), want, np.abs(want), 4)
    with pytest.raises(AssertionError):
        ref.within(np.array([np.nan, -2.0]), want, np.abs(want), 4)
