"""Oracle for the 4-bit paged KV cache.  TEST INFRASTRUCTURE ONLY.

Plain float64 from the definition (``include/cpattn.h``): a cached feature is c s u,
c a 4-bit float, s the 8-bit float of its group of 16 features, u the cache's power
of two.  Both are found as the nearest of all values there are, by distance, halves to
the even code; the bytes' places are worked out one byte at a time.  Shares no code
with the CUDA path.
"""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3(byte):
    """The value of an 8-bit float: sign, four bits of exponent (bias 7), three of
    mantissa; no infinities, the all-ones pattern is NaN."""
    byte = int(byte)
    e, m = (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return float("nan")
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if byte >> 7 else v


E4M3 = np.array([e4m3(b) for b in range(256)])


def nearest(x, values):
    """Index of the nearest of ``values`` (increasing, even and odd codes in turn) to
    each x >= 0; halves to the even index."""
    x = np.asarray(x, dtype=np.float64)
    d = np.abs(x[..., None] - values)
    best = d.min(-1, keepdims=True)
    even = np.arange(len(values)) % 2 == 0
    # Of (at most two) equally near, the even one.
    return np.argmax((d == best) * (1 + even), -1)


def quantise(x, unit=1.0):
    """Codes ``[..., D]`` (0 .. 15) and scale bytes ``[..., D / 16]`` of rows
    ``[..., D]``."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 16)) / unit
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    scale = nearest(np.clip(np.abs(g).max(-1) / 6, 2.0 ** -9, 448.0), E4M3[:127])
    code = nearest(np.minimum(np.abs(g) / E4M3[scale][..., None], 6.0), GRID)
    code = code + 8 * ((g < 0) & (code > 0))
    code = np.where(bad[..., None], 0, code)
    return (code.reshape(x.shape).astype(np.uint8),
            np.where(bad, 0x7F, scale).astype(np.uint8))


def values(code, scale, unit=1.0):
    """What codes and scale bytes stand for, ``[..., D]`` float64."""
    code = np.asarray(code)
    v = np.where(code > 7, -1.0, 1.0) * GRID[code & 7]
    s = E4M3[np.asarray(scale)] * unit
    return (v.reshape(code.shape[:-1] + (-1, 16)) * s[..., None]).reshape(code.shape)


def code_place(r, f, D):
    """Byte (of a page of one head) and half (0 low, 1 high) of feature f of token r."""
    tile, r = divmod(r, 16)
    j, i = divmod(f, 16)
    return tile * 9 * D + 128 * j + 16 * ((r // 2) ^ (128 * j // D)) + 8 * (r % 2) + i // 2, i % 2


def scale_place(r, j, D):
    tile, r = divmod(r, 16)
    return tile * 9 * D + 8 * D + 16 * j + r


def write(cache, page, head, row, code, scale):
    """Put one token's codes ``[D]`` and scales into ``cache`` (uint8, as the library's)."""
    D = len(code)
    block = cache[page, head].reshape(-1)
    for f in range(D):
        at, high = code_place(row, f, D)
        keep = int(block[at]) & (0x0F if high else 0xF0)
        block[at] = keep | (int(code[f]) << (4 * high))
    for j in range(D // 16):
        block[scale_place(row, j, D)] = scale[j]


def unpack(cache, D, unit=1.0):
    """A whole cache ``[pages, heads, size, 9 D / 16]`` as values ``[pages, size,
    heads, D]``, the bf16 cache's layout."""
    pages, heads, size, _ = cache.shape
    flat = np.asarray(cache).reshape(pages, heads, -1)
    at = np.array([[code_place(r, f, D) for f in range(D)] for r in range(size)])
    byte = flat[:, :, at[..., 0]]
    code = np.where(at[..., 1] == 1, byte >> 4, byte & 15)
    s_at = np.array([[scale_place(r, j, D) for j in range(D // 16)] for r in range(size)])
    return values(code, flat[:, :, s_at], unit).transpose(0, 2, 1, 3)
