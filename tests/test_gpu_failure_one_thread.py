"""A CTA that starts while another's wait runs out: its threads may read different
values of the error word.  In the test-only build one thread of CTA 1 of every
attention kernel reads a timeout and the others do not.  The CTA has to leave as a
whole (a warp that stayed would wait for one that left), with its copies landed and
its tensor memory given back: the kernels end, CTA 1 writes nothing, and the
regular library is right afterwards in the same context."""

import ctypes
import time

import pytest
import torch

from helpers import default_scale, make_batch
from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fault(cp):  # noqa: F811
    from long_context_gb300 import build as lib_build
    lib = ctypes.CDLL(lib_build.build_fault_injection())
    for name in ("cpattn_fwd", "cpattn_bwd", "cpattn_paged_attn", "cpattn_poll_error"):
        f, g = getattr(cp._lib, name), getattr(lib, name)
        g.argtypes, g.restype = f.argtypes, f.restype
    return lib


def p(t):
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("D", [64, 128])
def test_packed_attention(cp, fault, D):  # noqa: F811
    lengths, H = [700, 300, 500], 2
    (_, _, _, cu), g = make_batch(lengths, H, D, seed=17)
    T = sum(lengths)
    out, lse = cp.fwd(g["q"], g["k"], g["v"], g["cu"], max_seqlen=700)
    marked = torch.full_like(out, 7.0)
    mlse = torch.full_like(lse, 7.0)
    ws = cp.alloc_workspace(T, 3, H, D, 1)
    torch.cuda.synchronize()
    t0 = time.time()
    assert fault.cpattn_fwd(p(g["q"]), p(g["k"]), p(g["v"]), p(g["cu"]), None, 3, T, 700, 1, H, D,
                            default_scale(D), 1, 0, p(marked), p(mlse), p(ws), ws.numel(),
                            _stream()) == cp.OK
    assert fault.cpattn_poll_error(p(ws), _stream()) == cp.ERR_DEVICE_TIMEOUT  # CTA 0's wait
    left = (marked == 7).all(-1)
    assert left.any() and (mlse[left] == 7).all()
    dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(1)).to(out).contiguous()
    want = cp.bwd(g["q"], g["k"], g["v"], out, dout, lse, g["cu"], max_seqlen=700)
    grads = [torch.full_like(out, 7.0) for _ in range(3)]
    bws = cp.alloc_bwd_workspace(T, 3, H, D, 1)
    assert fault.cpattn_bwd(p(g["q"]), p(g["k"]), p(g["v"]), p(out), p(dout), p(lse), p(g["cu"]),
                            None, 3, T, 700, 1, H, D, default_scale(D), 1, *map(p, grads), p(bws),
                            bws.numel(), _stream()) == cp.OK
    assert fault.cpattn_poll_error(p(bws), _stream()) == cp.ERR_DEVICE_TIMEOUT
    assert time.time() - t0 < 30.0
    assert all((x == 7).all(-1).any() for x in grads)
    again = cp.fwd(g["q"], g["k"], g["v"], g["cu"], max_seqlen=700)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for a, b in zip(cp.bwd(g["q"], g["k"], g["v"], out, dout, lse, g["cu"], max_seqlen=700), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_paged_tiles(cp, fault, D):  # noqa: F811
    kv = [250, 200, 256, 180, 100]
    x = Batch([70] * 5, kv, 4, 2, D, 16, seed=31)
    q, kc, vc, t, cu, kvl = x.on_gpu()
    want = cp.paged_attn(q, kc, vc, t, cu, kvl, **x.bounds())
    out, lse = torch.full_like(q, 7.0), torch.full((x.T, 4), 7.0, device="cuda")
    ws = cp.alloc_paged_workspace(x.T, 5, 4, 2, D, 70)
    torch.cuda.synchronize()
    assert fault.cpattn_paged_attn(p(q), p(kc), p(vc), kc.shape[0], 16, kc.stride(0), p(t),
                                   t.shape[1], p(cu), p(kvl), 5, x.T, 70, max(kv), 4, 2, D,
                                   D ** -0.5, 1, p(out), p(lse), p(ws), ws.numel(),
                                   _stream()) == cp.OK
    assert fault.cpattn_poll_error(p(ws), _stream()) == cp.ERR_DEVICE_TIMEOUT
    # CTA 1 is the second KV head of the first item.
    assert (out[:70, 2:] == 7).all() and (lse[:70, 2:] == 7).all()
    assert torch.equal(out[70:], want[0][70:])
    again = cp.paged_attn(q, kc, vc, t, cu, kvl, **x.bounds())
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
