"""How many heads a lane group takes is chosen by the batch's size and heads; the
bits of a token do not depend on it: a large batch against the same tokens in
batches of 64 (runs of two heads)."""

import pytest
import torch

from test_gpu_norm_rope import cp, table  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(3, 1), (4, 4), (5, 5), (12, 4), (8, 8), (2, 1)])
def test_equal_bits_in_every_run(cp, H, Hk, D):  # noqa: F811
    T = 24064 * 128 // D
    g = torch.Generator(device="cuda").manual_seed(H * D)
    qkv = torch.randn(T, H + 2 * Hk, D, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k = qkv[:, :H], qkv[:, H:H + Hk]
    pos = torch.randint(0, 999, (T,), generator=g, device="cuda", dtype=torch.int32)
    tab = table(1000, D).cuda()
    w = torch.randn(D, generator=g, device="cuda", dtype=torch.bfloat16)
    kw = dict(q_weight=w, k_weight=w)
    whole = cp.qk_norm_rope(q, k, pos, tab, **kw)
    for a in range(0, T, T // 16 + 1):
        b = min(a + 64, T)
        part = cp.qk_norm_rope(q[a:b], k[a:b], pos[a:b], tab, **kw)
        for x, y in zip(part, whole):
            assert torch.equal(x, y[a:b])
