"""What attention of up to 16 rows a KV head over the paged cache (the decoding
step) keeps of its probabilities.

As in test_gpu_paged.py a score is off by at most D * 2^-24 * span, and the
exponential, the weights of splits and the sums add 2^-18: e = D 2^-24 span +
2^-18.  P meets V as a bf16 value and a bf16 remainder: the value is off by
half a step, 2^-8 of p, and the remainder (taken exactly in fp32) by 2^-8 of
that, so P is off by 2^-16.  O is rounded once to bf16, half a step.  So
|dO| <= 2^-8 |O| + (2^-16 + 2 e) size with size = sum p |v| / sum p: where the
values cancel, O is far more accurate than a P of one bf16 value allows (which
leaves up to 2^-8 size)."""

import numpy as np
import pytest

from oracle import paged as op
from test_gpu_norm_rope import check, f64
from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv,H,Hk", [
    ([1, 1, 1], [300, 40, 1000], 32, 8),                     # 4 rows a KV head
    ([2, 1], [300, 1900], 16, 4),                            # 8 and 4
    ([1, 3], [500, 77], 20, 4),                              # 5 and 15
    ([1], [2000], 16, 1),
    ([1] * 40, [60 + 9 * i for i in range(40)], 8, 2),       # more sequences than a warp plans
    ([2] * 34, [60 + 11 * i for i in range(34)], 16, 2),
])
def test_probabilities_of_a_decoding_step(cp, new, kv, H, Hk, D):  # noqa: F811
    x = Batch(new, kv, H, Hk, D, 16, seed=23)
    out, lse = cp.paged_attn(*x.on_gpu(), **x.bounds())
    x.check(out, lse)
    ref, _, size, span = op.attention(f64(x.q), f64(x.kc), f64(x.vc), x.table, x.cu, x.kv,
                                      x.scale)
    e = D * 2.0 ** -24 * span + 2.0 ** -18
    check(out, ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + 2 * e[..., None]) * size, "O")
