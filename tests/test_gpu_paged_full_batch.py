"""Attention over the paged cache of more sequences than a warp plans (32), few
rows each and caches long enough to be split: a schedule kernel lists the splits;
up to 16 rows a KV head are joined by the split that arrives last, up to 32 by the
merge kernel.  Tolerances as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


def _lengths(n, most_new, lo, hi, seed, longest=()):
    """Ragged lengths, some sequences without new tokens, one without a cache."""
    rng = np.random.default_rng(seed)
    new = [int(x) for x in rng.integers(1, most_new + 1, n)]
    kv = [int(x) for x in np.exp(rng.uniform(np.log(lo), np.log(hi), n))]
    kv = [max(a, b) for a, b in zip(new, kv)]
    new[3] = new[n - 2] = 0
    kv[5], new[7] = 0, most_new
    for i, x in enumerate(longest):
        kv[9 + 4 * i] = x
    return new, kv


# sequences, most new tokens, cache lengths, the longest ones, H, Hk, D, page size
CASES = [
    (33, 1, 20, 300, [10000], 4, 1, 128, 16),         # more splits than the join has in flight
    (33, 1, 20, 300, [9000, 64, 65, 4096], 1, 1, 64, 64),
    (64, 1, 200, 6000, [], 10, 2, 64, 32),
    (100, 1, 100, 3000, [7000], 16, 1, 128, 64),
    (70, 4, 100, 4000, [6001], 4, 4, 64, 16),
    (40, 1, 300, 5000, [], 17, 1, 64, 16),            # 17 rows
    (36, 4, 20, 500, [9000, 3000], 8, 1, 128, 32),    # 32
    (50, 4, 100, 4000, [], 16, 2, 128, 128),
    (34, 2, 100, 8000, [], 32, 2, 64, 256),
]


@pytest.mark.parametrize("n,most,lo,hi,longest,H,Hk,D,size", CASES)
def test_split_caches(cp, n, most, lo, hi, longest, H, Hk, D, size):  # noqa: F811
    new, kv = _lengths(n, most, lo, hi, n + H, longest)
    x = Batch(new, kv, H, Hk, D, size, seed=41, pad=2)
    args = x.on_gpu()
    ws = cp.alloc_paged_workspace(x.T, n, H, Hk, D, most)
    out = torch.full((x.T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.T, H), 7.0, device="cuda")
    cp.paged_attn(*args, out=out, lse=lse, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    # The list's length, behind the error word: some items are split.
    assert int(ws[:8].view(torch.int32)[1]) > sum(a > 0 for a in new)
    x.check(out, lse)
    assert (out[x.cu[-1]:] == 7).all() and (lse[x.cu[-1]:] == 7).all()
    # On the same workspace (its counters have to start again), also captured.
    again = cp.paged_attn(*args, workspace=ws, **x.bounds())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = cp.paged_attn(*args, workspace=ws, **x.bounds())
    for _ in range(3):
        graph.replay()
    rows = int(x.cu[-1])
    for got in (again, cap):
        assert torch.equal(got[0][:rows], out[:rows]) and torch.equal(got[1][:rows], lse[:rows])
    x_all = cp.paged_attn(*args, causal=False, workspace=ws, **x.bounds())
    x.check(*x_all, causal=False)


@pytest.mark.parametrize("most,H,Hk,D", [(1, 4, 1, 128), (4, 8, 1, 64), (1, 10, 2, 64)])
def test_a_bad_page_in_a_split(cp, most, H, Hk, D):  # noqa: F811
    """Its keys and values count as zeros; the other sequences keep their bits."""
    new, kv = _lengths(36, most, 50, 900, 3, [7000])
    x = Batch(new, kv, H, Hk, D, 32, seed=43, spoil=False)
    q, kc, vc, t, cu, kvl = x.on_gpu()
    ws = cp.alloc_paged_workspace(x.T, len(kv), H, Hk, D, most)
    good = cp.paged_attn(q, kc, vc, t, cu, kvl, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    assert int(ws[:8].view(torch.int32)[1]) > sum(a > 0 for a in new)
    at = 4500 // 32
    page = int(t[9, at])
    zeroed = [c.clone() for c in (kc, vc)]
    for c in zeroed:
        c[page] = 0
    want = cp.paged_attn(q, *zeroed, t, cu, kvl, **x.bounds())
    mine = slice(int(x.cu[9]), int(x.cu[10]))
    for number in (-1, kc.shape[0], 2 ** 31 - 1):
        bad = t.clone()
        bad[9, at] = number
        got = cp.paged_attn(q, kc, vc, bad, cu, kvl, workspace=ws, **x.bounds())
        assert cp.poll_error(ws) == cp.ERR_INVALID_ARG
        for g, w, ok in zip(got, want, good):
            assert torch.equal(g, w) and not torch.equal(g[mine], ok[mine])
        got = cp.paged_attn(q, kc, vc, t, cu, kvl, workspace=ws, **x.bounds())
        assert cp.poll_error(ws) == cp.OK
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


def test_one_workspace_while_sequences_finish(cp):  # noqa: F811
    """Made for the first step of 34 sequences of up to 40 new tokens, used by every
    later and smaller one."""
    H, Hk, D = 8, 2, 64
    x = Batch([1] * 34, [40 + 61 * i for i in range(34)], H, Hk, D, 16, seed=47)
    q, kc, vc, t, cu, kv = x.on_gpu()
    ws = cp.alloc_paged_workspace(34 * 40, 34, H, Hk, D, 40)
    for n in (34, 33, 32, 31, 7, 1):
        for bound in (40, 8, 4, 1):
            args = (q[:n], kc, vc, t[:n], cu[:n + 1], kv[:n])
            bounds = dict(max_seqlen=bound, max_kv_len=max(x.kv))
            got = cp.paged_attn(*args, workspace=ws, **bounds)
            assert cp.poll_error(ws) == cp.OK
            want = cp.paged_attn(*args, **bounds)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
