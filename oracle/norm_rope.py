"""Oracle for the norm + rotation of query and key heads.  TEST INFRASTRUCTURE ONLY.

Plain float64, written from the definition (``include/cpattn.h``): for a head
row ``x`` with weight ``w``, ``n = x / sqrt(mean(x^2) + eps) * w`` (``n = x``
without a weight), then each of the first ``R`` features' pairs ``(a, b)`` turned
by its angle: ``y_a = n_a cos - n_b sin``, ``y_b = n_b cos + n_a sin``.  The
gradient goes through the rotation's matrix, built entry by entry, and through
the norm's Jacobian, so that it shares no formula with the kernel.

Every function also returns magnitudes that bound the rounding of a float32
evaluation (sums of absolute values where the result has sums).
"""

from __future__ import annotations

import numpy as np


def pairs(R, interleaved):
    """The (a, b) feature indices of each angle."""
    j = np.arange(R // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)


def rotation_matrix(row, D, interleaved):
    """The D x D matrix of one position; ``row`` is its R cosines and sines."""
    R = len(row)
    m = np.eye(D)
    a, b = pairs(R, interleaved)
    for j in range(R // 2):
        c, s = row[j], row[R // 2 + j]
        m[a[j], a[j]] = c
        m[a[j], b[j]] = -s
        m[b[j], b[j]] = c
        m[b[j], a[j]] = s
    return m


def forward(x, w, row_of, D, interleaved, eps):
    """``x [T, H, D]``; ``row_of[t]`` the table row of token t (None: no rotation).
    Returns ``(y, size)``, ``size`` bounding the absolute terms of each y."""
    x = np.asarray(x, dtype=np.float64)
    n = x
    if w is not None:
        n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if row_of is None:
        return n, np.abs(n)
    y, size = np.empty_like(n), np.empty_like(n)
    for t in range(x.shape[0]):
        m = rotation_matrix(np.asarray(row_of[t], np.float64), D, interleaved)
        y[t] = n[t] @ m.T
        size[t] = np.abs(n[t]) @ np.abs(m).T
    return y, size


def backward(dy, x, w, row_of, D, interleaved, eps):
    """Returns ``(dx, dw, dx_size, dw_size)``; ``dw`` is None without a weight."""
    dy = np.asarray(dy, dtype=np.float64)
    g, g_size = dy.copy(), np.abs(dy)
    if row_of is not None:
        for t in range(dy.shape[0]):
            m = rotation_matrix(np.asarray(row_of[t], np.float64), D, interleaved)
            g[t] = dy[t] @ m
            g_size[t] = np.abs(dy[t]) @ np.abs(m)
    if w is None:
        return g, None, g_size, None
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    dw_size = (g_size * np.abs(x) * r).sum((0, 1))
    # d n_i / d x_j = w_i (r delta_ij - r^3 x_i x_j / D)
    dx = np.empty_like(x)
    dx_size = np.empty_like(x)
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            v, rr = x[t, h], r[t, h, 0]
            jac = (np.eye(D) * rr - rr ** 3 * np.outer(v, v) / D) * w[:, None]
            dx[t, h] = g[t, h] @ jac
            dx_size[t, h] = g_size[t, h] @ ((np.eye(D) * rr + rr ** 3 * np.abs(np.outer(v, v)) / D)
                                            * np.abs(w)[:, None])
    return dx, dw, dx_size, dw_size
