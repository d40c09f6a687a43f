"""The host's bounds choose the kernel that lists the work of tiles: few blocks are
listed in the lanes of a warp, more by a block of threads.  Both cut the same lists
at the same places, so that the same lengths give the same bits."""

import pytest
import torch

from test_gpu_norm_rope import normal
from test_gpu_paged import cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,units", [
    # Key tiles of each cache.  The uncut time is estimated at 38 by the exact sizes
    # of the items and at 36 by the lower edges of 128 ranges of sizes (50 and 48), and
    # a list is cut above 37.6 (49.0).
    (16, [10, 21, 22, 19, 19, 19, 4, 19, 23, 25, 23, 26]),
    (8, [30, 3, 27, 39, 39, 35, 10, 30, 1, 34, 30, 39, 32, 43, 25, 2, 28, 27, 16, 38, 11, 26, 26,
         30, 28, 30]),
    (16, [3, 70, 9, 9, 9]),  # well above
    (4, [12] * 30),          # well below
])
@pytest.mark.parametrize("D", [64, 128])
def test_equal_lengths_equal_bits(cp, heads, units, D):  # noqa: F811
    size, new, n = 64, 40, len(units)
    kv = [128 * u - 5 for u in units]
    pages = -(-max(kv) // size)
    kc = normal(pages + n, size, heads, D, seed=1).cuda()
    vc = normal(pages + n, size, heads, D, seed=2).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[b + p for p in range(pages)] for b in range(n)])  # shared pages
    q = normal(new * n + 256 * 40, heads, D, seed=3).cuda()
    cu, kvl = i32([new * b for b in range(n + 1)]), i32(kv)
    got = []
    for rows, bound in ((new * n, new), (q.shape[0], 2000)):
        ws = cp.alloc_paged_workspace(rows, n, heads, heads, D, bound)
        out, lse = cp.paged_attn(q[:rows], kc, vc, table, cu, kvl, max_seqlen=bound,
                                 max_kv_len=max(kv), workspace=ws)
        assert cp.poll_error(ws) == cp.OK
        got.append((int(ws[:8].view(torch.int32)[1]), out[:new * n], lse[:new * n]))
    assert got[0][0] == got[1][0]
    assert torch.equal(got[0][1], got[1][1]) and torch.equal(got[0][2], got[1][2])
