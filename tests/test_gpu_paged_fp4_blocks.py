"""The 4-bit attention of 33 to 64 rows of a KV head: several blocks of a sequence over the
codes, by the schedule kernel's list.  Up to 48 rows they are blocks of 16, whose splits the
last CTA joins; above, blocks of 32, which the merge kernel joins.  Batch and tolerance:
test_gpu_paged_fp4.py."""

import pytest
import torch

from test_gpu_paged_fp4 import MANY, Batch4, cp  # noqa: F401

pytestmark = pytest.mark.gpu

# New tokens, cached ones with them, heads, KV heads, page size: with causality a block of
# rows ends at a key of its own.
FEW = ([10, 1, 7, 3, 0, 10, 2], [3001, 1500, 2222, 5, 40, 61, 1])
EVEN = ([9] * 3, [4000, 4017, 130])
MANY_SEQS = ([10, 1] * 20, [6000 if b % 9 == 0 else 30 + 37 * b for b in range(40)])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch,H,Hk,size,rows", [
    (FEW, 8, 2, 16, 16),             # 40 rows: three blocks of 16 beside single ones
    (EVEN, 10, 2, 64, 16),           # 45: tokens that two blocks share
    (EVEN, 4, 1, 256, 16),           # 36, the third block of four
    (MANY_SEQS, 8, 2, 32, 16),       # more CTAs than a round: splits of at least 24 units
    (FEW, 10, 2, 128, 32),           # 50: two blocks of 32 and the merge kernel
    (EVEN, 7, 1, 16, 32),            # 63, tokens that two blocks share
    (([4, 2, 1], [2500, 1700, 9]), 32, 2, 32, 32),       # 64
    (MANY_SEQS, 12, 2, 64, 32),
])
def test_several_blocks_of_a_sequence(cp, batch, H, Hk, D, size, rows, causal):  # noqa: F811
    new, kv = batch
    most = max(new) * H // Hk
    assert 32 < most <= MANY and (rows == 16) == (most <= 48)
    x = Batch4(new, kv, H, Hk, D, size, seed=81, pad=2)
    args = x.on_gpu()
    ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), H, Hk, D, max(new), max(kv))
    ws.random_(0, 256)
    out, lse = cp.paged_attn_fp4(*args, causal=causal, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse, causal)
    again = cp.paged_attn_fp4(*args, causal=causal, workspace=ws, **x.bounds())
    n = int(x.cu[-1])
    assert torch.equal(again[0][:n], out[:n]) and torch.equal(again[1][:n], lse[:n])
