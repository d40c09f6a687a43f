"""Pins of the norm + rotation oracle (oracle/norm_rope.py), CPU only."""

import numpy as np
import pytest

from oracle import norm_rope as on


def _rows(T, R, seed):
    ang = np.random.default_rng(seed).uniform(0, 6.28, (T, R // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1)


def test_hand_values():
    """A quarter turn of one pair, with the other features left alone."""
    row = np.array([0.0, 1.0])                   # R = 2: cos, sin
    x = np.array([[[3.0, 4.0, 5.0, 6.0]]])
    for inter in (False, True):
        y, _ = on.forward(x, None, [row], 4, inter, 0.0)
        assert np.allclose(y, [[[-4.0, 3.0, 5.0, 6.0]]])
    row = np.array([0.0, 1.0, 1.0, 0.0])         # angle 0: quarter turn, angle 1: none
    assert np.allclose(on.forward(x, None, [row], 4, False, 0.0)[0], [[[-5.0, 4.0, 3.0, 6.0]]])
    assert np.allclose(on.forward(x, None, [row], 4, True, 0.0)[0], [[[-4.0, 3.0, 5.0, 6.0]]])
    # mean(x^2) = 21.5
    n, _ = on.forward(x, np.array([1.0, 2.0, 1.0, 1.0]), None, 4, False, 3.5)
    assert np.allclose(n, np.array([[[3.0, 8.0, 5.0, 6.0]]]) / 5.0)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(inter):
    """<R_p q, R_k k> depends on p - k alone."""
    D, R = 16, 8
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, D)), rng.normal(size=(1, 1, D))
    freq = 0.7 ** np.arange(R // 2)
    row = lambda p: np.concatenate([np.cos(p * freq), np.sin(p * freq)])  # noqa: E731
    turn = lambda x, p: on.forward(x, None, [row(p)], D, inter, 0.0)[0].ravel()  # noqa: E731
    assert np.isclose(turn(q, 9) @ turn(k, 4), turn(q, 105) @ turn(k, 100))
    assert np.isclose(np.linalg.norm(turn(q, 9)), np.linalg.norm(q))
    assert not np.isclose(turn(q, 9) @ turn(k, 4), turn(q, 9) @ turn(k, 5))


@pytest.mark.parametrize("inter,norm,rotate", [(False, True, True), (True, True, True),
                                               (False, False, True), (False, True, False)])
def test_gradients_are_the_differences(inter, norm, rotate):
    """Central differences of a scalar of the forward, step 1e-6: truncation
    about 1e-12 and rounding about 1e-10 of values of order one."""
    T, H, D, R, eps = 2, 2, 8, 4, 1e-3
    rng = np.random.default_rng(3)
    x, c = rng.normal(size=(T, H, D)), rng.normal(size=(T, H, D))
    w = rng.normal(size=D) if norm else None
    rows = _rows(T, R, 5) if rotate else None
    f = lambda x, w: (on.forward(x, w, rows, D, inter, eps)[0] * c).sum()  # noqa: E731
    dx, dw, dx_size, dw_size = on.backward(c, x, w, rows, D, inter, eps)
    step = 1e-6
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        assert abs((f(a, w) - f(b, w)) / (2 * step) - dx[i]) < 1e-8
    assert np.all(np.abs(dx) <= dx_size * (1 + 1e-12))
    if norm:
        for i in range(D):
            a, b = w.copy(), w.copy()
            a[i] += step
            b[i] -= step
            assert abs((f(x, a) - f(x, b)) / (2 * step) - dw[i]) < 1e-8
        assert np.all(np.abs(dw) <= dw_size * (1 + 1e-12))
