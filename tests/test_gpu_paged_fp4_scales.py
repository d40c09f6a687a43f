"""The 4-bit attention under a softmax scale that is no normal float, with a k_scale that
makes their product one: the product keeps its 24 bits (a factor in between would leave it
three or four).  Batch and tolerance: test_gpu_paged_fp4.py."""

import pytest

from test_gpu_paged_fp4 import Batch4, cp  # noqa: F401

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,kv,bound", [([1, 2], [40, 300], 300), ([1, 2], [40, 300], 30000),
                                          ([3, 1], [40, 300], 30000), ([1] * 40, [50] * 40, 30000),
                                          ([30, 9], [70, 300], 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_small_softmax_scale_and_a_large_unit(cp, new, kv, bound, D):  # noqa: F811
    x = Batch4(new, kv, 8, 2, D, 16, seed=71, units=(2.0 ** 32, 0.5))
    x.q = (x.q.double() * 2.0 ** 146 / 7).to(torch.bfloat16)
    x.scale = 7 * 2.0 ** -149    # that times log2(e) has four bits: 10 instead of 10.099
    ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), 8, 2, D, max(new), bound)
    out, lse = cp.paged_attn_fp4(*x.on_gpu(), max_seqlen=max(new), max_kv_len=bound,
                                 k_scale=2.0 ** 32, v_scale=0.5, softmax_scale=x.scale, workspace=ws)
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse)
