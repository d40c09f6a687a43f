"""Attention of many rows over a paged cache whose scores rise along it.

After a row's first key tile the tile kernel computes p against the reference that
the row has, and takes a tile again with its own maximum (scaling O and l, which
are in tensor memory) when the tile's sum of p exceeds 2^16 or is not finite.
Here keys grow by blocks of 128, so that later tiles exceed the first's maximum by
20, 60 and over 128 powers of two (p is infinite then), in rising and falling
order, while every third token's queries are so small that its rows never do.
Tolerances as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from test_gpu_norm_rope import f64
from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu

GROWTH = [1, 1, 8, 0.5, 20, 8, 50, 1, 60, 60]  # of the keys of one tile after the other


def _rise(x):
    """Scales the cached keys by their position, the queries by their token."""
    for b, n in enumerate(x.kv):
        for at in range(0, n, 16):  # a page holds at least 16 keys of one tile
            page, row = x.table[b, at // x.size], at % x.size
            x.kc[page, row:row + 16] *= GROWTH[at // 128 % len(GROWTH)]
    for b in range(len(x.new)):
        x.q[x.cu[b]:x.cu[b + 1]:3] *= 2.0 ** -8


def _exceeding(x, causal):
    """How many powers of two a row's later tiles (of 128 keys from the cache's
    start) exceed its first by, the largest of each row: [tokens, heads]."""
    out = []
    for b, n in enumerate(x.kv):
        rows = np.concatenate([f64(x.kc[p]) for p in x.table[b, :-(-n // x.size)]])[:n]
        q = f64(x.q[x.cu[b]:x.cu[b + 1]])
        s = np.einsum("thd,khd->thk", q, np.repeat(rows, x.H // x.Hk, 1)) * x.scale / np.log(2)
        if causal:
            last = n - len(q) + np.arange(len(q))
            s[np.broadcast_to(np.arange(n) > last[:, None, None], s.shape)] = -np.inf
        top = np.stack([s[..., i:i + 128].max(-1) for i in range(0, n, 128)], -1)
        out.append((top[..., 1:] - top[..., :1]).max(-1))
    return np.concatenate(out)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv,H,Hk,size,split", [
    ([40], [1280], 2, 2, 16, False),              # one Q tile
    ([200], [1300], 1, 1, 64, False),             # two
    ([50, 37], [1000, 1290], 4, 1, 32, False),    # two and one, four heads to a token
    ([140, 300], [700, 1500], 3, 3, 128, False),  # a block that starts inside a sequence
    ([60], [6000], 1, 1, 256, True),              # pieces of four key tiles
    ([150], [5100], 2, 1, 16, True),
])
def test_rising_scores(cp, new, kv, H, Hk, size, split, D, causal):  # noqa: F811
    x = Batch(new, kv, H, Hk, D, size, seed=51)
    _rise(x)
    over = _exceeding(x, causal)
    large = np.ones(len(over), dtype=bool)
    for b in range(len(new)):
        large[x.cu[b]:x.cu[b + 1]:3] = False
    assert (over[large] > 16).mean() > 0.9 and (over[large] > 128).mean() > 0.2
    assert (over[~large] < 8).all()
    ws = cp.alloc_paged_workspace(x.T, len(kv), H, Hk, D, max(new))
    out, lse = cp.paged_attn(*x.on_gpu(), causal=causal, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    items = int(ws[:8].view(torch.int32)[1])
    assert items > 4 if split else items <= 4 * len(new)
    x.check(out, lse, causal)
