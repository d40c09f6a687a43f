"""Tensors without elements in the norm + rotation and paged-cache calls: their
address is null, which in the C ABI stands for a tensor that is not given."""

import pytest
import torch

from test_gpu_norm_rope import normal, table
from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_table_without_positions_is_no_missing_table(cp):  # noqa: F811
    """A rotation was asked for and no position has angles: refused, and nothing
    written."""
    x = Batch([2, 1], [40, 20], 4, 2, 64, 16, seed=19)
    _, kc, vc, t, cu, kv = x.on_gpu()
    q, k = normal(3, 4, 64, seed=2).cuda(), normal(3, 2, 64, seed=1).cuda()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    before = kc.clone()
    out = torch.full_like(q, 7.0)
    refused = (ValueError, cp.CpattnError)
    for empty in (table(8, 64)[:0].cuda(), torch.empty(8, 0, device="cuda")):
        for kw in (dict(), dict(q_weight=w, k_weight=w)):
            with pytest.raises(refused):
                cp.qk_norm_rope(q, k, pos, empty, q_out=out, **kw)
            with pytest.raises(refused):
                cp.qk_norm_rope_bwd(q, k, q, k, pos, empty, dq=out, **kw)
            with pytest.raises(refused):
                cp.paged_append(k, k, kc, vc, t, cu, kv, rope_table=empty, q=q, q_out=out, **kw)
        with pytest.raises(refused):
            cp.paged_append(k, k, kc, vc, t, cu, kv, rope_table=empty)
    assert (out == 7).all() and torch.equal(kc.nan_to_num(9), before.nan_to_num(9))


@pytest.mark.parametrize("norm", [True, False])
def test_append_of_no_tokens_with_queries(cp, norm):  # noqa: F811
    """A step in which no sequence has a new token."""
    x = Batch([0, 0], [5, 20], 4, 2, 64, 16, seed=12)
    _, kc, vc, t, cu, kv = x.on_gpu()
    qkv = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda") if norm else None
    before = kc.clone(), vc.clone()
    q = cp.paged_append(qkv[:, 4:6], qkv[:, 6:], kc, vc, t, cu, kv, rope_table=table(32, 64).cuda(),
                        k_weight=w, q=qkv[:, :4], q_weight=w)
    assert q.shape == (0, 4, 64)
    for a, b in zip((kc, vc), before):
        assert torch.equal(a.nan_to_num(9), b.nan_to_num(9))
