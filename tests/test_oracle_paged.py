"""Pins of the paged-cache oracle (oracle/paged.py), CPU only."""

import numpy as np

from oracle import attention as oa
from oracle import decode as odc
from oracle import paged as op


def _paged(lengths, Hk, D, size, seed):
    """A contiguous cache and the same rows in shuffled pages."""
    rng = np.random.default_rng(seed)
    k, v = (rng.normal(size=(sum(lengths), Hk, D)) for _ in range(2))
    counts = [-(-n // size) for n in lengths]
    pages = sum(counts) + 3
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(counts + [1])), -1)
    kc, vc = (rng.normal(size=(pages, size, Hk, D)) for _ in range(2))
    row = used = 0
    for b, n in enumerate(lengths):
        table[b, :counts[b]] = order[used:used + counts[b]]
        used += counts[b]
        for p in range(n):
            kc[table[b, p // size], p % size] = k[row + p]
            vc[table[b, p // size], p % size] = v[row + p]
        row += n
    return k, v, kc, vc, table


def test_one_new_token_is_the_decode():
    """Grouped heads with one new token a sequence against the packed decode
    oracle on repeated heads."""
    lengths, Hk, G, D = [7, 1, 30], 2, 3, 8
    k, v, kc, vc, table = _paged(lengths, Hk, D, 4, seed=1)
    q = np.random.default_rng(2).normal(size=(3, Hk * G, D))
    cu = np.concatenate([[0], np.cumsum(lengths)])
    ref_o, ref_l = odc.decode_attention(q, np.repeat(k, G, 1), np.repeat(v, G, 1), cu, 0.4)
    o, lse, size, span = op.attention(q, kc, vc, table, [0, 1, 2, 3], lengths, 0.4)
    assert np.allclose(o, ref_o, atol=1e-13) and np.allclose(lse, ref_l, atol=1e-13)
    assert np.all(np.abs(o) <= size + 1e-15) and np.all(span > 0)


def test_new_tokens_are_the_last_rows_of_full_attention():
    lengths, new, H, D = [12, 5, 9], [4, 5, 0], 2, 4
    k, v, kc, vc, table = _paged(lengths, H, D, 4, seed=3)
    cu_kv = np.concatenate([[0], np.cumsum(lengths)])
    cu = np.concatenate([[0], np.cumsum(new)])
    qfull = np.random.default_rng(4).normal(size=k.shape)
    rows = np.concatenate([np.arange(cu_kv[b + 1] - n, cu_kv[b + 1]) for b, n in enumerate(new)])
    for causal in (True, False):
        ref_o, ref_l = oa.full_attention(qfull, k, v, cu_kv, 0.5, causal=causal)
        o, lse, _, _ = op.attention(qfull[rows], kc, vc, table, cu, lengths, 0.5, causal)
        assert np.allclose(o, ref_o[rows], atol=1e-13)
        assert np.allclose(lse, ref_l[rows], atol=1e-13)


def test_rows_without_keys_and_places():
    """A cache shorter than its new tokens: the first rows see nothing and have
    no place; rows behind the last sequence stay NaN."""
    k, v, kc, vc, table = _paged([2], 1, 4, 4, seed=5)
    q = np.ones((6, 1, 4))
    o, lse, _, _ = op.attention(q, kc, vc, table, [0, 5], [2], 1.0)
    assert np.all(o[:3] == 0) and np.all(np.isneginf(lse[:3, 0]))
    assert np.allclose(o[3, 0], v[0, 0]) and np.isfinite(lse[4, 0]) and np.isnan(o[5]).all()
    assert op.places([0, 5], [2], table, 4) == [(3, 0, 0, table[0, 0], 0), (4, 0, 1, table[0, 0], 1)]
