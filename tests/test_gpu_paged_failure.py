"""Failure detection of the paged tile kernel, as in test_gpu_failure.py: in the
test-only build of the library the first CTA withholds one hand-off to its MMA
warp, whose wait (2 s) runs out.  The kernel ends by itself, the error word says
so, and the regular library then runs the same problem right in the same context.
The caches are so short that no stage of the kernel's rings is filled twice."""

import ctypes
import time

import pytest
import torch

from test_gpu_paged import Batch, cp  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,kv", [(128, [250, 200, 256] + [180] * 60),
                                  (64, [500, 200, 512] + [300] * 60)])
def test_a_bounded_wait_runs_out(cp, D, kv):  # noqa: F811
    from long_context_gb300 import build as lib_build
    fault = ctypes.CDLL(lib_build.build_fault_injection())
    for name in ("cpattn_paged_attn", "cpattn_poll_error"):
        f, g = getattr(cp._lib, name), getattr(fault, name)
        g.argtypes, g.restype = f.argtypes, f.restype
    x = Batch([70] * len(kv), kv, 4, 2, D, 16, seed=31)
    q, kc, vc, t, cu, kvl = x.on_gpu()
    out = torch.zeros_like(q)
    lse = torch.zeros(x.T, 4, device="cuda")
    ws = cp.alloc_paged_workspace(x.T, len(kv), 4, 2, D, 70)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    p = lambda a: ctypes.c_void_p(a.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    t0 = time.time()
    st = fault.cpattn_paged_attn(p(q), p(kc), p(vc), kc.shape[0], 16, kc.stride(0), p(t),
                                 t.shape[1], p(cu), p(kvl), len(kv), x.T, 70, max(kv), 4, 2, D,
                                 D ** -0.5, 1, p(out), p(lse), p(ws), ws.numel(), stream)
    assert st == cp.OK  # the launch itself is fine
    assert fault.cpattn_poll_error(p(ws), stream) == cp.ERR_DEVICE_TIMEOUT
    assert time.time() - t0 < 30.0
    out, lse = cp.paged_attn(q, kc, vc, t, cu, kvl, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse)
