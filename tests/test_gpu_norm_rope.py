"""GPU parity of the norm + rotation (cpattn_qk_norm_rope, _bwd) against
oracle/norm_rope.py.

Tolerances.  The kernels hold everything in fp32 and round once to bf16 (half
a step: 2^-8 of the value).  In fp32, a mean of D <= 128 squares is off by at
most (D / 8 + 5) * 2^-24 < 2^-19 relative (8 products per lane, then log2 of
the lanes), the reciprocal root by half of that and two units, and the four to
six further operations on a term by 2^-24 each: under 2^-18 of the sum of the
terms' magnitudes, which the oracle gives.  Forward: 2^-8 |y| + 2^-18 size.
dx's terms pass through two such means: 2^-8 |dx| + 2^-17 size.  A weight's
gradient is a sum of at most N = T * heads terms taken along chains of at most
(rows per lane group) + 16 or 32 + 128 + 8 additions; in these tests that is
below 2^8, so 2^-16 of the terms' magnitudes; with the terms' own 2^-18:
2^-15 size."""

import numpy as np
import pytest
import torch

from oracle import norm_rope as on

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_gb300 import build as lib_build
    lib_build.build()
    from long_context_gb300 import cpattn
    return cpattn


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def table(max_pos, R, base=10000.0):
    j = torch.arange(R // 2, dtype=torch.float64)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * base ** (-2 * j / R)
    return torch.cat([a.cos(), a.sin()], 1).float()


def normal(*shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def check(got, ref, tol, what):
    got = f64(got)
    assert np.all(np.isfinite(got)), what
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)) if ref.size else 0.0
    assert worst <= 1.0, "%s: %g of the tolerance" % (what, worst)


# T, H, Hk, D, R, interleaved, norm
CASES = [
    (1, 1, 1, 128, 128, False, True),
    (1, 32, 8, 64, 64, True, True),
    (7, 5, 1, 128, 64, True, False),
    (33, 12, 3, 64, 16, False, True),
    (50, 3, 3, 128, 48, False, True),     # 24 angles: partners 3 lanes apart
    (129, 7, 2, 64, 48, True, True),
    (20, 4, 4, 128, 0, False, True),      # norm alone
    (200, 9, 2, 128, 128, False, False),
]


def _inputs(T, H, Hk, D, R, norm, strided, seed):
    qkv = normal(T, H + 2 * Hk, D, seed=seed, std=1.5).cuda()
    q, k = qkv[:, :H], qkv[:, H:H + Hk]
    if not strided:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(seed + 1),
                        dtype=torch.int32)
    pos[0] = 4999
    tab = table(5000, R) if R else None
    wq = (1 + 0.3 * normal(D, seed=seed + 2).float()).to(torch.bfloat16) if norm else None
    wk = (1 + 0.3 * normal(D, seed=seed + 3).float()).to(torch.bfloat16) if norm else None
    return q, k, pos, tab, wq, wk


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("T,H,Hk,D,R,inter,norm", CASES)
def test_forward_and_gradients(cp, T, H, Hk, D, R, inter, norm, strided):
    q, k, pos, tab, wq, wk = _inputs(T, H, Hk, D, R, norm, strided, seed=T + D)
    rows = None if tab is None else tab[pos.long()].numpy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dpos, dtab, dwq_, dwk_ = _cuda(pos, tab, wq, wk)
    kw = dict(q_weight=dwq_, k_weight=dwk_, eps=1e-5, interleaved=inter, status=status)
    qo, ko = cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    gq, gk = normal(T, H, D, seed=9).cuda(), normal(T, Hk, D, seed=10).cuda()
    dq, dk, dwq, dwk = cp.qk_norm_rope_bwd(gq, gk, q, k, dpos, dtab, **kw)
    assert int(status) == 0
    for x, w, y, g, dx, dw in ((q, wq, qo, gq, dq, dwq), (k, wk, ko, gk, dk, dwk)):
        w64 = None if w is None else f64(w)
        ref, size = on.forward(f64(x), w64, rows, D, inter, 1e-5)
        check(y, ref, 2 ** -8 * np.abs(ref) + 2 ** -18 * size, "y")
        rdx, rdw, sx, sw = on.backward(f64(g), f64(x), w64, rows, D, inter, 1e-5)
        check(dx, rdx, 2 ** -8 * np.abs(rdx) + 2 ** -17 * sx, "dx")
        if w is None:
            assert dw is None
        else:
            check(dw, rdw, 2 ** -15 * sw, "dw")
    # Equal inputs, equal bits (the weights' sums among them).
    again = cp.qk_norm_rope_bwd(gq, gk, q, k, dpos, dtab, **kw)
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert (a is None and b is None) or torch.equal(a, b)


def _whole(x, w, rows, R, inter, eps):
    """The oracle's forward on whole arrays, float64 on the device; also the size of
    its terms."""
    x = x.double()
    n = x if w is None else x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    c, s = rows.double()[:, None].chunk(2, -1)
    a = slice(0, R, 2) if inter else slice(0, R // 2)
    b = slice(1, R, 2) if inter else slice(R // 2, R)
    y, size = n.clone(), n.abs()
    y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., b] * c + n[..., a] * s
    size[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
    size[..., b] = (n[..., b] * c).abs() + (n[..., a] * s).abs()
    return y, size


def test_whole_arrays_are_the_oracle(cp):
    for inter in (False, True):
        x, w = normal(5, 3, 64, seed=1), normal(64, seed=2)
        rows = table(9, 32)[torch.tensor([8, 0, 3, 5, 1])]
        y, size = _whole(x, w, rows, 32, inter, 1e-5)
        ref, rs = on.forward(f64(x), f64(w), rows.numpy(), 64, inter, 1e-5)
        assert np.allclose(f64(y), ref, rtol=1e-13) and np.allclose(f64(size), rs, rtol=1e-13)


@pytest.mark.parametrize("T,H,Hk,D,inter", [
    (7400, 15, 13, 128, False),   # runs of eight heads that end inside a batch
    (7400, 16, 16, 128, True),
    (3701, 16, 14, 128, False),   # forward in runs of four
    (15001, 15, 3, 64, True),
])
def test_many_tokens(cp, T, H, Hk, D, inter):
    """Sizes that take the longer runs of heads, against float64 autograd of the
    same definition.  A weight's gradient adds its T * heads terms along chains of
    at most T * heads / lane groups + 64 < 2^9 additions: 2^-15 + 2^-18 of their
    magnitudes, so 2^-14 size holds with room; magnitudes as in the oracle."""
    R = D // 2
    q, k, pos, tab, wq, wk = _inputs(T, H, Hk, D, R, True, True, seed=T)
    dpos, dtab, dwq_, dwk_ = _cuda(pos, tab, wq, wk)
    kw = dict(q_weight=dwq_, k_weight=dwk_, eps=1e-5, interleaved=inter)
    qo, ko = cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    gq, gk = normal(T, H, D, seed=9).cuda(), normal(T, Hk, D, seed=10).cuda()
    dq, dk, dwq, dwk = cp.qk_norm_rope_bwd(gq, gk, q, k, dpos, dtab, **kw)
    rows = dtab[dpos.long()]
    for x, w, y, g, dx, dw in ((q, dwq_, qo, gq, dq, dwq), (k, dwk_, ko, gk, dk, dwk)):
        x64 = x.double().requires_grad_()
        w64 = w.double().requires_grad_()
        ref, size = _whole(x64, w64, rows, R, inter, 1e-5)
        rdx, rdw = torch.autograd.grad(ref, (x64, w64), g.double())
        x64, w64, ref, size = (t.detach() for t in (x64, w64, ref, size))
        assert ((y.double() - ref).abs() <= 2 ** -8 * ref.abs() + 2 ** -18 * size).all()
        # The magnitudes of the gradient's terms: |g| turned by |cos|, |sin|.
        gs = _whole(g, None, torch.cat([rows[:, :R // 2], -rows[:, R // 2:]], 1), R, inter, 0)[1]
        r = (x64.pow(2).mean(-1, keepdim=True) + 1e-5).rsqrt()
        u, hat = gs * w64.abs(), (x64 * r).abs()
        sx = r * (u + hat * (u * hat).mean(-1, keepdim=True))
        assert ((dx.double() - rdx).abs() <= 2 ** -8 * rdx.abs() + 2 ** -17 * sx).all()
        assert ((dw.double() - rdw).abs() <= 2 ** -14 * (gs * hat).sum((0, 1))).all()


def test_in_place_and_given_outputs(cp):
    """Outputs over the inputs, inside one projection's buffer: the values
    between and behind them stay."""
    T, H, Hk, D = 37, 6, 2, 64
    q, k, pos, tab, wq, wk = _inputs(T, H, Hk, D, 64, True, True, seed=5)
    dpos, dtab, dwq, dwk = _cuda(pos, tab, wq, wk)
    kw = dict(q_weight=dwq, k_weight=dwk)
    qo, ko = cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    buf = q._base if q._base is not None else q
    before = buf.clone()
    r = cp.qk_norm_rope(q, k, dpos, dtab, q_out=q, k_out=k, **kw)
    assert r[0] is q and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(buf[:, H + Hk:], before[:, H + Hk:])
    g = normal(T, H, D, seed=1).cuda()
    gk = normal(T, Hk, D, seed=2).cuda()
    x = before[:, :H], before[:, H:H + Hk]
    ref = cp.qk_norm_rope_bwd(g, gk, *x, dpos, dtab, **kw)
    got = cp.qk_norm_rope_bwd(g, gk, *x, dpos, dtab, dq=g, dk=gk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_positions_outside_the_table(cp):
    """Their rows stay, their gradients stay and count for nothing; the status
    word is set, and not cleared by a later good call."""
    T, H, Hk, D = 9, 3, 2, 128
    q, k, pos, tab, wq, wk = _inputs(T, H, Hk, D, 128, True, False, seed=6)
    bad = pos.clone()
    bad[2], bad[5] = -1, 5000
    good = [t for t in range(T) if t not in (2, 5)]
    dpos, dtab, dwq, dwk, dbad = _cuda(pos, tab, wq, wk, bad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=dwq, k_weight=dwk, status=status)
    ref = cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    assert int(status) == 0
    outs = [torch.full_like(q, 7.0), torch.full_like(k, 7.0)]
    cp.qk_norm_rope(q, k, dbad, dtab, q_out=outs[0], k_out=outs[1], **kw)
    assert int(status) == cp.ERR_INVALID_ARG
    for a, b in zip(outs, ref):
        assert torch.equal(a[good], b[good]) and (a[[2, 5]] == 7).all()
    cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    assert int(status) == cp.ERR_INVALID_ARG
    status.zero_()
    gq, gk = normal(T, H, D, seed=1).cuda(), normal(T, Hk, D, seed=2).cuda()
    dq, dk = torch.full_like(gq, 7.0), torch.full_like(gk, 7.0)
    _, _, a, b = cp.qk_norm_rope_bwd(gq, gk, q, k, dbad, dtab, dq=dq, dk=dk, **kw)
    assert int(status) == cp.ERR_INVALID_ARG and (dq[[2, 5]] == 7).all() and (dk[[2, 5]] == 7).all()
    rows = tab[pos.long()].numpy()
    for g, x, w, dw in ((gq, q, wq, a), (gk, k, wk, b)):
        _, rdw, _, sw = on.backward(f64(g)[good], f64(x)[good], f64(w), rows[good], D, False, 1e-6)
        check(dw, rdw, 2 ** -15 * sw, "dw")


def test_no_tokens(cp):
    D = 64
    e = lambda h: torch.empty(0, h, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    tab = table(4, 64).cuda()
    a, b = cp.qk_norm_rope(e(4), e(2), pos, tab, q_weight=w, k_weight=w)
    assert a.shape == (0, 4, D) and b.shape == (0, 2, D)
    _, _, dwq, dwk = cp.qk_norm_rope_bwd(e(4), e(2), e(4), e(2), pos, tab, q_weight=w, k_weight=w)
    assert (dwq == 0).all() and (dwk == 0).all()


def test_non_finite_rows_stay_theirs(cp):
    """A NaN or an infinity spoils its own row only; without norms an infinity
    outside the rotated features passes through."""
    T, H, D = 4, 2, 128
    q = normal(T, H, D, seed=8).cuda()
    k = normal(T, 1, D, seed=9).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    tab = table(8, 64).cuda()
    ref, _ = cp.qk_norm_rope(q, k, pos, tab)
    x = q.clone()
    x[1, 1, 5] = float("nan")
    x[2, 0, 100] = float("inf")
    y, _ = cp.qk_norm_rope(x, k, pos, tab)
    mask = torch.zeros_like(y, dtype=torch.bool)
    mask[1, 1, 5] = mask[1, 1, 37] = mask[2, 0, 100] = True
    assert torch.equal(y[~mask], ref[~mask])
    assert y[1, 1, 5].isnan() and y[1, 1, 37].isnan() and y[2, 0, 100] == float("inf")


def test_streams_and_graphs(cp):
    """On a stream of its own and captured, then replayed on new inputs."""
    T, H, Hk, D = 65, 8, 4, 128
    q, k, pos, tab, wq, wk = _inputs(T, H, Hk, D, 128, True, False, seed=11)
    dpos, dtab, dwq, dwk = _cuda(pos, tab, wq, wk)
    kw = dict(q_weight=dwq, k_weight=dwk)
    g, gk = normal(T, H, D, seed=1).cuda(), normal(T, Hk, D, seed=2).cuda()
    ref = cp.qk_norm_rope(q, k, dpos, dtab, **kw) + cp.qk_norm_rope_bwd(g, gk, q, k, dpos, dtab, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cp.qk_norm_rope(q, k, dpos, dtab, stream=s, **kw) + cp.qk_norm_rope_bwd(
        g, gk, q, k, dpos, dtab, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    qs, ks = torch.zeros_like(q), torch.zeros_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = cp.qk_norm_rope(qs, ks, dpos, dtab, **kw) + cp.qk_norm_rope_bwd(
            g, gk, qs, ks, dpos, dtab, **kw)
    qs.copy_(q)
    ks.copy_(k)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, cap))


def test_training_chain(cp):
    """Norm + rotation, causal attention and both backward passes against the
    float64 chain.  The two GPU paths differ from it by bf16 roundings at every
    hand-over, so the gradients of the whole chain are held in the mean: each of
    about ten roundings (q, k, P, O, dO, dS, dq, dk, the output) of relative
    size 2^-8 at most, so 2^-9 in the mean, adds up to sqrt(10) 2^-9 < 1 %."""
    from oracle import attention as oa
    from oracle import backward as ob
    lengths, H, D = [100, 37], 4, 64
    T = sum(lengths)
    q, k, _, tab, wq, wk = _inputs(T, H, H, D, 64, True, True, seed=21)
    v = normal(T, H, D, seed=22).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths])
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    dpos, dtab, dwq_, dwk_, dcu = _cuda(pos, tab, wq, wk, torch.from_numpy(cu))
    kw = dict(q_weight=dwq_, k_weight=dwk_)
    qn, kn = cp.qk_norm_rope(q, k, dpos, dtab, **kw)
    out, lse = cp.fwd(qn, kn, v, dcu, max_seqlen=100)
    dout = normal(T, H, D, seed=23).cuda()
    gq, gk, gv = cp.bwd(qn, kn, v, out, dout, lse, dcu, max_seqlen=100)
    dq, dk, dwq, dwk = cp.qk_norm_rope_bwd(gq, gk, q, k, dpos, dtab, **kw)
    rows = tab[pos.long()].numpy()
    rq, _ = on.forward(f64(q), f64(wq), rows, D, False, 1e-6)
    rk, _ = on.forward(f64(k), f64(wk), rows, D, False, 1e-6)
    ro, _ = oa.full_attention(rq, rk, f64(v), cu, D ** -0.5)
    ref = ob.full_attention_backward(rq, rk, f64(v), f64(dout), cu, D ** -0.5)
    rms = lambda x: np.sqrt(np.mean(np.square(x)))  # noqa: E731
    near = lambda a, b: rms(f64(a) - b) <= 1e-2 * rms(b)  # noqa: E731
    assert near(out, ro) and near(gv, ref["dv"])
    for g, x, w, dx, dw in ((ref["dq"], q, wq, dq, dwq), (ref["dk"], k, wk, dk, dwk)):
        rdx, rdw, _, _ = on.backward(g, f64(x), f64(w), rows, D, False, 1e-6)
        assert near(dx, rdx) and near(dw, rdw)
