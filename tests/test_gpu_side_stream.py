"""Calls on a stream that is not current: what a call makes is of that stream's
memory, so that no pending work of the current stream still writes there, and
is kept from that stream while the current one reads it."""

import pytest
import torch

from test_gpu_norm_rope import normal, table
from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(cp, stream):  # noqa: F811
    """Calls that make their outputs and workspaces, as functions."""
    x = Batch([1, 2, 1], [700, 20, 333], 8, 2, 128, 16, seed=15, spoil=False)
    q, kc, vc, t, cu, kv = x.on_gpu()
    k = normal(4, 2, 128, seed=1).cuda()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos, tab = torch.arange(4, dtype=torch.int32, device="cuda"), table(800, 128).cuda()
    kw = dict(q_weight=w, k_weight=w, stream=stream)
    return [
        lambda: cp.paged_attn(q, kc, vc, t, cu, kv, stream=stream, **x.bounds()),
        lambda: cp.qk_norm_rope(q, k, pos, tab, **kw),
        lambda: cp.qk_norm_rope_bwd(q, k, q, k, pos, tab, **kw),
        lambda: [cp.paged_append(k, k, kc, vc, t, cu, kv, q=q, rope_table=tab, **kw)],
    ]


def test_pending_work_of_the_current_stream(cp):  # noqa: F811
    """Blocks of every size that the calls make are freed on the current stream
    while a fill of them is still to come there; the calls on another stream are
    done before that fill, and keep their results."""
    want = [f() for f in _calls(cp, None)]
    s = torch.cuda.Stream()
    calls = _calls(cp, s)
    sizes = {o.numel() * o.element_size() for r in want for o in r}
    sizes |= {cp.paged_workspace_size(4, 3, 8, 2, 128, 2)}
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sorted(sizes) * 12]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    for b in blocks:
        b.fill_(0x7f)
    del b, blocks
    got = [f() for f in calls]
    torch.cuda.synchronize()
    for r, w in zip(got, want):
        for a, b in zip(r, w):
            assert torch.equal(a, b)


def test_freed_while_the_current_stream_reads(cp):  # noqa: F811
    """A result that the current stream has still to read is freed: its block does
    not go to the next allocation of the stream that the call ran on."""
    s = torch.cuda.Stream()
    call = _calls(cp, s)[0]
    copy = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    out, lse = call()
    s.synchronize()
    want = out.cpu()
    torch.cuda._sleep(400_000_000)
    copy.copy_(out)
    del out, lse
    with torch.cuda.stream(s):
        for _ in range(8):
            torch.empty_like(copy).fill_(7.0)
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), want)


def test_a_branch_of_a_captured_graph(cp):  # noqa: F811
    """The calls on a stream forked inside a capture, then replayed."""
    want = [f() for f in _calls(cp, None)]
    s = torch.cuda.Stream()
    calls = _calls(cp, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        got = [f() for f in calls]
        torch.cuda.current_stream().wait_stream(s)
        copies = [[o.clone() for o in r] for r in got]
    for _ in range(2):
        for r in copies:
            for o in r:
                o.zero_()
        graph.replay()
    torch.cuda.synchronize()
    # The first replay appends; the attention of the second reads what it wrote.
    for r, w in zip(copies[1:], want[1:]):
        for a, b in zip(r, w):
            assert torch.equal(a, b)
    again = _calls(cp, None)
    again[3]()
    for a, b in zip(copies[0], again[0]()):
        assert torch.equal(a, b)
