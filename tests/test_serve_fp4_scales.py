"""Which softmax scales the 4-bit attention takes, on the host: softmax_scale * k_scale has
to be a normal float, whatever softmax_scale alone is.  (A call that is not refused for them
gets as far as its workspace's size.)"""

import pytest

from test_serve_refusals import INVALID, SMALL, call, cp, mem  # noqa: F401
from test_serve_refusals_fp4 import attend

MOST = 3.4028234663852886e38     # the largest float
LEAST = 2.0 ** -149              # the smallest
NORMAL = 2.0 ** -126             # the smallest normal one


@pytest.mark.parametrize("scale,unit,want", [
    (MOST, 2.0 ** -32, SMALL), (MOST / 2, 0.5, SMALL), (2.0 ** -100, 2.0 ** 32, SMALL),
    (LEAST, 2.0 ** 32, SMALL), (NORMAL, 1.0, SMALL), (0.9 * NORMAL, 2.0, SMALL),
    (MOST, 1.0, INVALID), (MOST / 2, 2.0, INVALID), (0.9 * NORMAL, 1.0, INVALID),
    (NORMAL, 0.5, INVALID), (LEAST, 2.0 ** 22, INVALID), (LEAST / 4, 2.0 ** 32, INVALID)])
def test_scales(cp, mem, scale, unit, want):  # noqa: F811
    assert call(cp._lib.cpattn_paged_attn_fp4, attend(mem), scale=scale, ku=unit, ws_bytes=0) == want
