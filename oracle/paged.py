"""Oracle for the paged KV cache.  TEST INFRASTRUCTURE ONLY.

Plain float64, token by token, from the definition (``include/cpattn.h``):
token ``p`` of sequence ``b`` is row ``p % page_size`` of page
``page_table[b, p // page_size]``; new token ``i`` of ``q_len`` stands at
position ``kv_len - q_len + i``; query head ``h`` reads KV head
``h // (H // Hk)``.  Shares no code with the CUDA path.
"""

from __future__ import annotations

import numpy as np


def places(cu, kv_lens, page_table, page_size):
    """``[(token, sequence, position, page, row)]`` of every new token that has a
    place (a position below zero has none)."""
    out = []
    for b in range(len(kv_lens)):
        q_len = int(cu[b + 1]) - int(cu[b])
        for i in range(q_len):
            p = int(kv_lens[b]) - q_len + i
            if p >= 0:
                out.append((int(cu[b]) + i, b, p, int(page_table[b][p // page_size]),
                            p % page_size))
    return out


def gather(cache, page_table_row, kv_len):
    """A sequence's ``kv_len`` cached rows, ``[kv_len, Hk, D]`` float64."""
    size = cache.shape[1]
    rows = [cache[int(page_table_row[p // size]), p % size] for p in range(int(kv_len))]
    return np.asarray(rows, dtype=np.float64).reshape((int(kv_len),) + cache.shape[2:])


def attention(q, k_cache, v_cache, page_table, cu, kv_lens, scale, causal=True):
    """Returns ``(O [T, H, D], LSE [T, H], size [T, H, D], span [T, H])``: ``size``
    is sum p |v| / sum p and ``span`` the largest visible scale * sum |q_i k_i|,
    which bound a float32 evaluation's rounding.  Rows behind the last sequence
    are NaN."""
    q = np.asarray(q, dtype=np.float64)
    T, H, D = q.shape
    group = H // k_cache.shape[2]
    out, size = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan)
    lse, span = np.full((T, H), np.nan), np.full((T, H), np.nan)
    for b in range(len(kv_lens)):
        n, t0 = int(kv_lens[b]), int(cu[b])
        q_len = int(cu[b + 1]) - t0
        if q_len == 0:
            continue
        k, v = gather(k_cache, page_table[b], n), gather(v_cache, page_table[b], n)
        for i in range(q_len):
            seen = min(max(n - q_len + i + 1, 0), n) if causal else n
            for h in range(H):
                kh, vh = k[:seen, h // group], v[:seen, h // group]
                if seen == 0:
                    out[t0 + i, h] = size[t0 + i, h] = 0.0
                    lse[t0 + i, h], span[t0 + i, h] = -np.inf, 0.0
                    continue
                s = scale * (kh @ q[t0 + i, h])
                top = s.max()
                p = np.exp(s - top)
                out[t0 + i, h] = p @ vh / p.sum()
                size[t0 + i, h] = p @ np.abs(vh) / p.sum()
                lse[t0 + i, h] = top + np.log(p.sum())
                span[t0 + i, h] = scale * (np.abs(kh) @ np.abs(q[t0 + i, h])).max()
    return out, lse, size, span
