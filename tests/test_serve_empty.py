"""Calls without new tokens: an array of no elements may have a null address.
Nothing is enqueued, so no GPU is needed."""

import pytest

from test_serve_refusals import INVALID, append, call, cp, mem  # noqa: F401


@pytest.mark.parametrize("weights", [True, False])
def test_append_of_no_tokens_with_queries(cp, mem, weights):  # noqa: F811
    """As PyTorch gives it: queries [0, H, D], their output, k and v are null."""
    w = {} if weights else dict(wq=None, wk=None)
    none = dict(T=0, q=None, qo=None, k=None, v=None, **w)
    assert call(cp._lib.cpattn_paged_append, append(mem), **none) == 0
    assert call(cp._lib.cpattn_paged_append, append(mem), **{**none, "H": -1}) == INVALID
    assert call(cp._lib.cpattn_paged_append, append(mem), **{**none, "T": 4}) == INVALID
    if weights:  # both weights or neither
        assert call(cp._lib.cpattn_paged_append, append(mem), **{**none, "wk": None}) == INVALID
