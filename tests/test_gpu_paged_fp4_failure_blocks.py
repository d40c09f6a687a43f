"""Failure detection of the 4-bit cache's attention where a sequence has several blocks of
rows: over the codes (blocks of 16, joined by the last CTA of an item, whose count stays short
where a CTA left; blocks of 32 and the merge kernel) and through the tile kernel over 16-bit
pages.  In the test-only build of the library a copy is not started, or a tile of P not handed
on; the wait (2 s) runs out, the kernel ends by itself, the error word says so, and the
regular library then runs the same problem right in the same workspace.  The tile kernel's
caches are so short that no stage of its rings is filled twice."""

import ctypes
import time

import pytest
import torch

from test_gpu_paged_fp4 import Batch4, cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,kv,H,Hk,D,bound", [
    ([10] * 3, [2000, 900, 77], 8, 2, 128, 40000),
    ([10] * 3, [2000, 900, 77], 8, 2, 64, 40000),
    ([7] * 3, [2000, 900, 77], 16, 2, 128, 40000),
    ([70] * 63, [250, 200, 256] + [180] * 60, 4, 2, 128, 256),
    ([70] * 63, [500, 200, 512] + [300] * 60, 4, 2, 64, 512),
])
def test_a_bounded_wait_runs_out(cp, new, kv, H, Hk, D, bound):  # noqa: F811
    from long_context_gb300 import build as lib_build
    fault = ctypes.CDLL(lib_build.build_fault_injection())
    for name in ("cpattn_paged_attn_fp4", "cpattn_poll_error"):
        f, g = getattr(cp._lib, name), getattr(fault, name)
        g.argtypes, g.restype = f.argtypes, f.restype
    x = Batch4(new, kv, H, Hk, D, 16, seed=31)
    q, kc, vc, t, cu, kvl = x.on_gpu()
    out = torch.zeros_like(q)
    lse = torch.zeros(x.T, H, device="cuda")
    ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), H, Hk, D, max(new), bound)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda a: ctypes.c_void_p(a.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    t0 = time.time()
    st = fault.cpattn_paged_attn_fp4(p(q), p(kc), p(vc), kc.shape[0], 16, kc.stride(0), p(t),
                                     t.shape[1], p(cu), p(kvl), len(kv), x.T, max(new), bound, H,
                                     Hk, D, 1.0, 1.0, D ** -0.5, 1, p(out), p(lse), p(ws),
                                     ws.numel(), stream)
    assert st == cp.OK  # the launch itself is fine
    assert fault.cpattn_poll_error(p(ws), stream) == cp.ERR_DEVICE_TIMEOUT
    assert 1.5 < time.time() - t0 < 30.0
    out, lse = cp.paged_attn_fp4(q, kc, vc, t, cu, kvl, max_seqlen=max(new), max_kv_len=bound,
                                 workspace=ws)
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse)
