"""GPU parity of the paged KV cache (cpattn_paged_append, cpattn_paged_attn)
against oracle/paged.py and oracle/norm_rope.py.

Tolerances of the attention.  A score is a sum of D products in fp32: off by at
most D * 2^-24 * span, with span the largest scale * sum |q_i k_i| of the row
(the oracle gives it); exponential, maximum, the weights of splits and sums add
2^-18 (terms of l and O are added along chains of at most N / 64 + 600; N <=
2^15 here).  P is rounded to bf16 (2^-8 of each term, so 2^-8 of the sum of
p |v|), and O once more (2^-8 |O|).  With e = D 2^-24 span + 2^-18, numerator
and denominator both off by e:  |dO| <= 2^-8 |O| + (2^-8 + 2 e) size, and
|dLSE| <= e + 2^-22 |LSE|.  The append is copies (equal bits) and the norm +
rotation's tolerance (see test_gpu_norm_rope.py)."""

import numpy as np
import pytest
import torch

from oracle import norm_rope as on
from oracle import paged as op
from test_gpu_norm_rope import check, f64, normal, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_gb300 import build as lib_build
    lib_build.build()
    from long_context_gb300 import cpattn
    return cpattn


class Batch:
    """A paged batch: shuffled pages, table entries behind the last page wild,
    cache rows behind kv_len NaN."""

    def __init__(self, new, kv, H, Hk, D, size, seed, std=1.0, pad=0, spoil=True):
        self.new, self.kv, self.H, self.Hk, self.D, self.size = new, kv, H, Hk, D, size
        rng = np.random.default_rng(seed)
        counts = [-(-n // size) for n in kv]
        pages = sum(counts) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(kv), max(counts + [1]) + 1), 2 ** 30, dtype=np.int32)
        self.kc = normal(pages, size, Hk, D, seed=seed, std=std)
        self.vc = normal(pages, size, Hk, D, seed=seed + 1, std=std)
        used = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[used:used + c]
            used += c
            if spoil and kv[b] % size:
                self.kc[self.table[b, c - 1], kv[b] % size:] = float("nan")
                self.vc[self.table[b, c - 1], kv[b] % size:] = float("nan")
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        self.q = normal(self.T, H, D, seed=seed + 2, std=std)
        self.scale = D ** -0.5

    def on_gpu(self):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
        return (self.q.cuda(), self.kc.cuda(), self.vc.cuda(), i32(self.table), i32(self.cu),
                i32(self.kv))

    def bounds(self):
        return dict(max_seqlen=max(self.new), max_kv_len=max(self.kv))

    def check(self, out, lse, causal=True, rows=None):
        ref, rl, size, span = op.attention(f64(self.q), f64(self.kc), f64(self.vc), self.table,
                                           self.cu, self.kv, self.scale, causal)
        n = int(self.cu[-1])
        ref, rl, size, span = ref[:n], rl[:n], size[:n], span[:n]
        e = self.D * 2.0 ** -24 * span + 2.0 ** -18
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * size
        check(out[:n], ref, tol, "O")
        got = f64(lse[:n])
        assert np.array_equal(np.isneginf(got), np.isneginf(rl))
        fin = np.isfinite(rl)
        assert np.all(f64(out[:n])[~fin] == 0)
        d = np.abs(got[fin] - rl[fin])
        assert np.all(d <= e[fin] + 2.0 ** -22 * np.abs(rl[fin])), d.max()


# new, kv, H, Hk, D, page size
CASES = [
    ([1], [1], 1, 1, 64, 16),
    ([1], [300], 8, 1, 128, 16),
    ([1, 1, 1], [5, 128, 1000], 4, 4, 64, 32),
    ([1, 1, 1, 1], [17, 64, 65, 700], 32, 4, 128, 64),
    ([1, 0, 1], [129, 40, 0], 6, 2, 128, 128),           # no new token; no key
    ([3, 1, 5], [3, 400, 201], 10, 2, 64, 16),           # groups of 5
    ([2, 4], [1000, 77], 7, 1, 128, 256),                # groups of 7
    ([2], [500], 33, 1, 64, 32),                         # 66 rows for one KV head
    ([20, 1, 33], [20, 90, 150], 8, 2, 128, 16),
    ([64, 7], [200, 7], 4, 2, 64, 64),
    ([5], [2], 3, 3, 128, 16),                           # rows that see no key
    ([130, 129, 128, 127, 1], [130, 300, 128, 640, 129], 4, 4, 128, 128),
    ([257, 3], [257, 515], 6, 1, 64, 16),
    ([300], [1000], 3, 1, 128, 32),                      # three heads to a token: 126 rows a tile
    ([40], [260], 128, 1, 64, 64),                       # the largest group
    ([70, 5], [390, 133], 71, 1, 128, 16),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,kv,H,Hk,D,size", CASES)
def test_attention(cp, new, kv, H, Hk, D, size, causal):
    x = Batch(new, kv, H, Hk, D, size, seed=sum(kv) % 97)
    out, lse = cp.paged_attn(*x.on_gpu(), causal=causal, **x.bounds())
    x.check(out, lse, causal)


@pytest.mark.parametrize("new,kv,H,Hk,D,size,std", [
    ([1], [9000], 4, 1, 64, 64, 1.0),                    # many splits of one token
    ([1, 1], [6000, 33], 2, 2, 128, 16, 2.5),            # scores over many powers of two
    ([2, 70], [3100, 5000], 4, 2, 128, 32, 2.0),         # splits beside whole items
    ([5, 3], [4000, 700], 10, 2, 64, 32, 1.0),           # up to 32 rows in splits
    ([4], [5000], 16, 2, 128, 16, 1.0),
    ([5], [20000], 5, 1, 64, 64, 1.0),                   # more splits than a round of the merge
    ([100, 60], [2600, 2000], 4, 4, 64, 16, 2.0),        # tiles cut at several places
    ([300, 10, 0, 700], [2300, 1800, 5, 2000], 16, 16, 64, 16, 1.0),  # more pieces than SMs
    ([100, 40, 0, 300], [6300, 5800, 5, 6000], 16, 16, 64, 16, 1.0),
    ([35] * 20, [1900 + 13 * i for i in range(20)], 16, 16, 64, 32, 1.0),   # long lists that
    ([35] * 40, [1900 + 13 * i for i in range(40)], 8, 8, 128, 16, 1.0),    # stay whole
    ([35] * 36, [200 + 17 * i for i in range(35)] + [9000], 2, 2, 64, 16, 1.0),  # one is cut
])
def test_long_caches(cp, new, kv, H, Hk, D, size, std):
    x = Batch(new, kv, H, Hk, D, size, seed=3, std=std)
    args = x.on_gpu()
    out, lse = cp.paged_attn(*args, **x.bounds())
    x.check(out, lse)
    ws = cp.alloc_paged_workspace(x.T, len(kv), H, Hk, D, max(new))
    again = cp.paged_attn(*args, workspace=ws, **x.bounds())
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)  # a fixed order of sums
    assert cp.poll_error(ws) == cp.OK


def test_many_sequences(cp):
    """More sequences than the schedule kernel has threads, some of them empty."""
    rng = np.random.default_rng(4)
    new = [int(n) for n in rng.integers(0, 3, 1500)]
    kv = [n + int(c) for n, c in zip(new, rng.integers(0, 20, 1500))]
    x = Batch(new, kv, 2, 1, 64, 16, seed=9)
    out, lse = cp.paged_attn(*x.on_gpu(), **x.bounds())
    x.check(out, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_many_blocks(cp, D):
    """More blocks of tiles than the schedule kernel has threads, most of one key
    tile, and one long cache that is cut: the blocks are listed by size over
    several rounds."""
    new, kv = [40] * 180 + [7], [60] * 180 + [3500]
    x = Batch(new, kv, 33, 1, D, 64, seed=17)
    args = x.on_gpu()
    out, lse = cp.paged_attn(*args, **x.bounds())
    again = cp.paged_attn(*args, **x.bounds())
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    # A few of the equal sequences and the long one against the oracle.
    ref, rl, size, span = op.attention(
        f64(x.q[-47:]), f64(x.kc), f64(x.vc), x.table[-2:], [0, 40, 47], kv[-2:], x.scale)
    e = D * 2.0 ** -24 * span + 2.0 ** -18
    check(out[-47:], ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * size, "O")
    assert np.all(np.abs(f64(lse[-47:]) - rl) <= e + 2.0 ** -22 * np.abs(rl))
    # And every sequence by itself (another schedule, no cuts for the short ones).
    q, kc, vc, t, cu, kvl = args
    for b in (0, 1, 90, 179):
        one, _ = cp.paged_attn(q[40 * b:40 * b + 40], kc, vc, t[b:b + 1], cu[:2], kvl[b:b + 1],
                               max_seqlen=40, max_kv_len=60)
        assert torch.equal(one, out[40 * b:40 * b + 40])


def test_padded_batch_and_larger_bounds(cp):
    """Rows behind the last sequence stay, and bounds above the lengths (a
    captured program's) choose other kernels and splits for the same answer."""
    for new, bound in (([1, 2, 1], 2), ([1, 2, 1], 9), ([1, 2, 1], 400), ([30, 1, 0], 2000)):
        x = Batch(new, [40, 1100, 17], 8, 2, 128, 16, seed=6, pad=5)
        out = torch.full((x.T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((x.T, 8), 7.0, device="cuda")
        cp.paged_attn(*x.on_gpu(), max_seqlen=bound, max_kv_len=5000, out=out, lse=lse)
        x.check(out, lse)
        assert (out[x.cu[-1]:] == 7).all() and (lse[x.cu[-1]:] == 7).all()


def test_caches_inside_a_larger_tensor(cp):
    """K and V pages side by side, [pages, 2, size, Hk, D], and a single page."""
    x = Batch([2, 1], [70, 33], 4, 2, 64, 32, seed=7)
    q, kc, vc, t, cu, kv = x.on_gpu()
    both = torch.stack([kc, vc], 1)
    for bound in (2, 9, 200):
        out, lse = cp.paged_attn(q, both[:, 0], both[:, 1], t, cu, kv, max_seqlen=bound,
                                 max_kv_len=70)
        x.check(out, lse)
    k, v = normal(3, 2, 64, seed=1).cuda(), normal(3, 2, 64, seed=2).cuda()
    want = both.clone()
    cp.paged_append(k, v, both[:, 0], both[:, 1], t, cu, kv)
    for (i, _, _, pg, row) in op.places(x.cu, x.kv, x.table, 32):
        want[pg, 0, row], want[pg, 1, row] = k[i], v[i]
    assert torch.equal(both.nan_to_num(9), want.nan_to_num(9))
    y = Batch([1], [9], 4, 2, 64, 32, seed=8)
    q, kc, vc, t, cu, kv = y.on_gpu()
    page = int(y.table[0, 0])
    t[0, 0] = 0
    out, lse = cp.paged_attn(q, kc[page:page + 1], vc[page:page + 1], t, cu, kv, **y.bounds())
    y.check(out, lse)


def test_bad_lengths_and_pages(cp):
    """Lengths that contradict the bounds write nothing; a page number outside
    the cache reads nothing.  Both are reported, and the next good call is clean."""
    x = Batch([1, 2], [40, 50], 4, 2, 64, 16, seed=10)
    q, kc, vc, t, cu, kv = x.on_gpu()
    ws = cp.alloc_paged_workspace(x.T, 2, 4, 2, 64, 2)
    for bad_cu, bad_kv, bad_bound in (([0, 1, 3], [40, -1], 50), ([0, 1, 3], [40, 51], 50),
                                      ([0, 1, 4], [40, 50], 50), ([0, 2, 1], [40, 50], 50),
                                      ([1, 1, 3], [40, 50], 50), ([0, 3, 3], [40, 50], 50),
                                      ([0, 1, 3], [40, 16 * t.shape[1] + 1], 4000)):
        out = torch.full_like(q, 7.0)
        cp.paged_attn(q, kc, vc, t, torch.tensor(bad_cu, dtype=torch.int32, device="cuda"),
                      torch.tensor(bad_kv, dtype=torch.int32, device="cuda"), max_seqlen=2,
                      max_kv_len=bad_bound, out=out, workspace=ws)
        assert cp.poll_error(ws) == cp.ERR_INVALID_ARG and (out == 7).all()
    for bound in (2, 300):
        ws = cp.alloc_paged_workspace(x.T, 2, 4, 2, 64, bound)
        for page in (-1, kc.shape[0], 2 ** 31 - 1):
            bad = t.clone()
            bad[1, 1] = page
            out, _ = cp.paged_attn(q, kc, vc, bad, cu, kv, max_seqlen=bound, max_kv_len=50,
                                   workspace=ws)
            assert cp.poll_error(ws) == cp.ERR_INVALID_ARG and out[:1].isfinite().all()
        out, lse = cp.paged_attn(q, kc, vc, t, cu, kv, max_seqlen=bound, max_kv_len=50,
                                 workspace=ws)
        assert cp.poll_error(ws) == cp.OK
        x.check(out, lse)


def test_no_work(cp):
    x = Batch([0, 0], [5, 0], 4, 2, 64, 16, seed=12)
    q, kc, vc, t, cu, kv = x.on_gpu()
    ws = cp.alloc_paged_workspace(0, 2, 4, 2, 64, 1)
    out, lse = cp.paged_attn(q, kc, vc, t, cu, kv, max_seqlen=1, max_kv_len=5, workspace=ws)
    assert out.shape == (0, 4, 64) and cp.poll_error(ws) == cp.OK
    out, _ = cp.paged_attn(q, kc, vc, t[:0], cu[:1], kv[:0], max_seqlen=1, max_kv_len=0)
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("new,kv,H,Hk,D,size,R,inter,norm,with_q", [
    ([1, 1, 1], [1, 16, 17], 8, 2, 128, 16, 128, False, True, True),
    ([5, 0, 1, 40], [9, 3, 100, 40], 5, 5, 64, 32, 32, True, True, True),
    ([33, 2], [40, 66], 6, 3, 128, 64, 64, False, False, True),
    ([7, 3], [7, 130], 4, 1, 64, 128, 64, True, True, False),
    ([3, 4], [300, 4], 4, 4, 128, 256, 0, False, False, False),   # copies alone
    ([3, 4], [300, 4], 4, 4, 128, 16, 0, False, True, True),      # norms alone
])
def test_append(cp, new, kv, H, Hk, D, size, R, inter, norm, with_q):
    x = Batch(new, kv, H, Hk, D, size, seed=sum(kv), pad=3, spoil=False)
    _, kc, vc, t, cu, kvl = x.on_gpu()
    qkv = normal(x.T, H + 2 * Hk, D, seed=2, std=1.5).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    tab = table(max(kv), R).cuda() if R else None
    w = [(1 + 0.3 * normal(D, seed=s).float()).to(torch.bfloat16).cuda() if norm else None
         for s in (3, 4)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((x.T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    extra = dict(q=q, q_weight=w[0], q_out=qo) if with_q else {}
    r = cp.paged_append(k, v, kc, vc, t, cu, kvl, rope_table=tab, interleaved=inter, k_weight=w[1],
                        eps=1e-5, status=status, **extra)
    assert int(status) == 0 and (r is qo if with_q else r is None)
    at = op.places(x.cu, kv, x.table, size)
    tok = [a[0] for a in at]
    rows = None if tab is None else f64(tab)[[a[2] for a in at]]
    new_k, new_v = x.kc.clone(), x.vc.clone()
    for (i, _, _, page, row) in at:
        new_v[page, row] = v[i].cpu()
        new_k[page, row] = kc[page, row].cpu()      # checked below
    assert torch.equal(vc.cpu(), new_v) and torch.equal(kc.cpu(), new_k)
    got = torch.stack([kc[page, row] for (_, _, _, page, row) in at])
    w64 = [None if a is None else f64(a) for a in w]
    ref, s = on.forward(f64(k)[tok], w64[1], rows, D, inter, 1e-5)
    check(got, ref, 2 ** -8 * np.abs(ref) + 2 ** -18 * s, "k")
    if R == 0 and not norm:
        assert torch.equal(got, k[tok])
    if with_q:
        ref, s = on.forward(f64(q)[tok], w64[0], rows, D, inter, 1e-5)
        check(qo[tok], ref, 2 ** -8 * np.abs(ref) + 2 ** -18 * s, "q")
        assert (qo[x.cu[-1]:] == 7).all()


def test_append_of_many_tokens(cp):
    """A size that takes the longer runs of heads: the bits of qk_norm_rope and of
    the values."""
    H, Hk, D, size, new = 16, 8, 128, 64, [3000, 1, 4500]
    kv = [3100, 900, 4500]
    x = Batch(new, kv, 1, 1, 64, size, seed=18, spoil=False)
    _, _, _, t, cu, kvl = x.on_gpu()
    pages = x.kc.shape[0]
    kc, vc = (torch.zeros(pages, size, Hk, D, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    qkv = normal(x.T, H + 2 * Hk, D, seed=2, std=1.5).cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    w = (1 + 0.3 * normal(D, seed=3).float()).to(torch.bfloat16).cuda()
    tab = table(4500, 128).cuda()
    qo = cp.paged_append(k, v, kc, vc, t, cu, kvl, rope_table=tab, k_weight=w, q=q, q_weight=w)
    at = op.places(x.cu, kv, x.table, size)
    pos = torch.tensor([a[2] for a in at], dtype=torch.int32, device="cuda")
    rq, rk = cp.qk_norm_rope(q, k, pos, tab, q_weight=w, k_weight=w)
    page = torch.tensor([a[3] for a in at], device="cuda")
    row = torch.tensor([a[4] for a in at], device="cuda")
    assert torch.equal(qo, rq) and torch.equal(kc[page, row], rk) and torch.equal(vc[page, row], v)
    rest = torch.ones(pages, size, dtype=torch.bool, device="cuda")
    rest[page, row] = False
    assert (kc[rest] == 0).all() and (vc[rest] == 0).all()


def test_append_leaves_out_bad_tokens(cp):
    """A page outside the cache, a position outside the rotation's table, a
    cache shorter than its new tokens or than its table: those tokens are left
    out and reported, the others are placed."""
    x = Batch([2, 3, 1], [40, 20, 9], 2, 2, 64, 16, seed=14, spoil=False)
    _, kc0, vc0, t, cu, kv = x.on_gpu()
    k, v = normal(6, 2, 64, seed=1).cuda(), normal(6, 2, 64, seed=2).cuda()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    bad_page = t.clone()
    bad_page[1, 1] = kc0.shape[0]
    tab = table(39, 64).cuda()
    cap = 16 * t.shape[1]
    for pages, kv_, table_, left in ((bad_page, kv, None, [2, 3, 4]), (t, kv, tab, [1]),
                                     (t, i32([40, 2, 9]), None, [2]),
                                     (t, i32([40, -5, 9]), None, [2, 3, 4]),
                                     (t, i32([40, cap + 1, 9]), None, [2, 3, 4])):
        kc, vc = kc0.clone(), vc0.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cp.paged_append(k, v, kc, vc, pages, cu, kv_, rope_table=table_, status=status)
        assert int(status) == cp.ERR_INVALID_ARG
        want = vc0.clone()
        for (i, _, _, page, row) in op.places(x.cu, kv_.clamp(max=40).tolist(), x.table, 16):
            if i not in left:
                want[page, row] = v[i]
        assert torch.equal(vc, want)


def test_append_then_attend_step_by_step(cp):
    """A prompt in chunks, then single tokens, as a server runs them: every
    step's output against attention over the cache that the steps wrote, and
    the last against the packed forward of the whole sequences."""
    H, Hk, D, size, total = 8, 2, 64, 16, [75, 41]
    rng = np.random.default_rng(0)
    x = [normal(n, H + 2 * Hk, D, seed=30 + b) for b, n in enumerate(total)]
    tab = table(128, D).cuda()
    w = (1 + 0.3 * normal(D, seed=3).float()).to(torch.bfloat16).cuda()
    pages = 16
    t = torch.from_numpy(rng.permutation(pages)[:12].reshape(2, 6).astype(np.int32)).cuda()
    kc, vc = (torch.full((pages, size, Hk, D), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    done = [0, 0]
    outs = [[], []]
    for step in ([40, 1], [20, 30], [0, 8], [1, 1], [14, 1]):
        new = [min(s, n - d) for s, n, d in zip(step, total, done)]
        qkv = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(2)]).cuda()
        done = [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0, new[0], new[0] + new[1]], dtype=torch.int32, device="cuda")
        kv = torch.tensor(done, dtype=torch.int32, device="cuda")
        q = cp.paged_append(qkv[:, H:H + Hk], qkv[:, H + Hk:], kc, vc, t, cu, kv, rope_table=tab,
                            k_weight=w, q=qkv[:, :H], q_weight=w)
        out, lse = cp.paged_attn(q, kc, vc, t, cu, kv, max_seqlen=max(new), max_kv_len=max(done))
        b = Batch(new, done, H, Hk, D, size, seed=1, spoil=False)
        b.q, b.kc, b.vc, b.table = q, kc.nan_to_num(), vc.nan_to_num(), t.cpu().numpy()
        b.check(out, lse)
        outs[0].append(out[:new[0]])
        outs[1].append(out[new[0]:])
    assert done == total
    # The whole sequences at once through the training path, repeated KV heads.
    qkv = torch.cat(x).cuda()
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in total]).cuda()
    q, k = cp.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hk], pos, tab, q_weight=w, k_weight=w)
    rep = lambda a: a.repeat_interleave(H // Hk, 1).contiguous()  # noqa: E731
    cu = torch.tensor([0, total[0], sum(total)], dtype=torch.int32, device="cuda")
    whole, _ = cp.fwd(q, rep(k), rep(qkv[:, H + Hk:]), cu, max_seqlen=max(total))
    got = torch.cat(outs[0] + outs[1])
    # Both round P and O to bf16: each is within 2^-8 (|O| + size) of the exact
    # value, and |v| <= 5 bounds size.
    assert (got.float() - whole.float()).abs().max() <= 2 * 2 ** -8 * (whole.abs().max().float() + 5)


def test_streams_graphs_and_two_workspaces(cp):
    """A captured decoding step replayed with other lengths, beside calls on
    another stream with a workspace of their own."""
    x = Batch([1, 1, 1], [700, 20, 333], 8, 2, 128, 16, seed=15, spoil=False)
    q, kc, vc, t, cu, kv = x.on_gpu()
    first = kv.clone()
    kvs = torch.tensor([1, 1, 1], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    bounds = dict(max_seqlen=1, max_kv_len=700)
    ref = cp.paged_attn(q, kc, vc, t, cu, first, **bounds)
    with torch.cuda.graph(graph):
        cap = cp.paged_attn(q, kc, vc, t, cu, kvs, **bounds)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        kvs.copy_(first)
        graph.replay()
        other = cp.paged_attn(q, kc, vc, t, cu, first, stream=s, **bounds)
    torch.cuda.synchronize()
    for got in (cap, other):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    x.check(*ref)


def test_a_cache_past_32_bit_offsets(cp):
    """Pages whose element offsets lie beyond 2^31 (about 4.4 GB a cache)."""
    H, Hk, D, size = 8, 8, 128, 256
    pages = 2 ** 31 // (size * Hk * D) + 64
    kc = torch.zeros(pages, size, Hk, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = Batch([1, 200], [600, 500], H, Hk, D, size, seed=16, spoil=False)
    table_ = np.full((2, 3), -1, dtype=np.int32)
    table_[0], table_[1, :2] = [pages - 1, pages - 5, 1], [pages - 2, pages - 3]
    for b in range(2):
        for i in range(-(-x.kv[b] // size)):
            kc[int(table_[b, i])] = x.kc[x.table[b, i]].cuda()
            vc[int(table_[b, i])] = x.vc[x.table[b, i]].cuda()
    _, _, _, _, cu, kv = x.on_gpu()
    t = torch.from_numpy(table_).cuda()
    out, lse = cp.paged_attn(x.q.cuda(), kc, vc, t, cu, kv, **x.bounds())
    x.check(out, lse)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    few, _ = cp.paged_attn(x.q[[0, x.T - 1]].cuda(), kc, vc, t, one, kv, max_seqlen=1,
                           max_kv_len=600)
    # The same two rows by the other kernel: each within 2^-8 (2 |O| + size) of the
    # exact value, |v| <= 6.
    assert (few.float() - out[[0, x.T - 1]].float()).abs().max() <= 2 * 2 ** -8 * 3 * 6
    k, v = normal(x.T, Hk, D, seed=1).cuda(), normal(x.T, Hk, D, seed=2).cuda()
    cp.paged_append(k, v, kc, vc, t, cu, kv)
    for (i, _, _, page, row) in op.places(x.cu, x.kv, table_, size)[::37]:
        assert torch.equal(kc[page, row], k[i]) and torch.equal(vc[page, row], v[i])


def test_refused_tensors(cp):
    """Types, shapes and layouts are refused before anything is enqueued."""
    x = Batch([2, 1], [40, 20], 4, 2, 64, 16, seed=19)
    q, kc, vc, t, cu, kv = x.on_gpu()
    k = normal(3, 2, 64, seed=1).cuda()
    pos, tab = torch.zeros(3, dtype=torch.int32, device="cuda"), table(8, 64).cuda()
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, k_cache=kc, v_cache=vc, page_table=t, cu_seqlens=cu, kv_lens=kv)
    bounds = dict(max_seqlen=2, max_kv_len=40)
    stacked = torch.stack([kc, vc], 1)
    for change, error in (
            (dict(q=q.float()), TypeError), (dict(q=q.cpu()), ValueError),
            (dict(q=q.transpose(0, 1)), ValueError), (dict(q=q[:, ::2]), ValueError),
            (dict(q=q[..., :32]), ValueError), (dict(q=q[0]), ValueError),
            (dict(k_cache=kc.half()), TypeError), (dict(k_cache=kc[:-1]), ValueError),
            (dict(v_cache=vc.transpose(1, 2)), ValueError), (dict(k_cache=kc[..., 0]), ValueError),
            (dict(k_cache=stacked[:, 0]), ValueError),           # another page stride than v's
            (dict(page_table=t.long()), TypeError), (dict(page_table=t[:1]), ValueError),
            (dict(page_table=t[:, ::2]), ValueError), (dict(page_table=t[0]), ValueError),
            (dict(cu_seqlens=cu[:-1]), ValueError), (dict(kv_lens=kv.long()), TypeError),
            (dict(kv_lens=kv[None]), ValueError), (dict(q=None), TypeError)):
        with pytest.raises(error):
            cp.paged_attn(**{**good, **change}, **bounds)
    for change, error in ((dict(out=q[:2]), ValueError), (dict(out=q.float()), TypeError),
                          (dict(lse=torch.zeros(3, 4, device="cuda").double()), TypeError),
                          (dict(workspace=torch.zeros(64, device="cuda")), TypeError),
                          (dict(max_seqlen=1 << 40), ValueError), (dict(max_kv_len="x"), TypeError),
                          (dict(softmax_scale="x"), TypeError), (dict(stream=3), AttributeError)):
        with pytest.raises(error):
            cp.paged_attn(**good, **{**bounds, **change})
    for change, status in ((dict(out=q), cp.ERR_INVALID_ARG),
                           (dict(softmax_scale=-1.0), cp.ERR_INVALID_ARG),
                           (dict(workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")),
                            cp.ERR_WORKSPACE_TOO_SMALL)):
        with pytest.raises(cp.CpattnError) as e:
            cp.paged_attn(**good, **{**bounds, **change})
        assert e.value.status == status
    for args, kw, error in (
            ((k, k[:2], kc, vc, t, cu, kv), {}, ValueError),
            ((k, k, kc, vc, t, cu, kv), dict(q_weight=w), ValueError),
            ((k, k, kc, vc, t, cu, kv), dict(rope_table=tab[0]), ValueError),
            ((k, k, kc, vc, t, cu, kv), dict(rope_table=tab.double()), TypeError),
            ((k, k, kc, vc, t, cu, kv), dict(k_weight=w[:32]), ValueError),
            ((k, k, kc[:, :, :1], vc[:, :, :1], t, cu, kv), {}, ValueError),
            ((k, k, kc, kc, t, cu, kv), {}, cp.CpattnError),     # one cache for both
            ((k[:, :, :32].contiguous(),) * 2 + (kc, vc, t, cu, kv), {}, ValueError),
            ((k.transpose(0, 1).contiguous().transpose(0, 1), k, kc, vc, t, cu, kv), {}, ValueError)):
        with pytest.raises(error):
            cp.paged_append(*args, **kw)
    for args, kw, error in (
            ((q, k, pos.long(), tab), {}, TypeError), ((q, k, pos[:2], tab), {}, ValueError),
            ((q, k[:2], pos, tab), {}, ValueError), ((q, k, None, tab), {}, TypeError),
            ((q, k, pos, tab), dict(q_weight=w), cp.CpattnError),  # one weight of two
            ((q, k, None, None), {}, cp.CpattnError),              # nothing to do
            ((q[:1].expand(3, 4, 64), k, pos, tab), {}, cp.CpattnError),
            ((q, k, pos, tab), dict(q_out=q[:2]), ValueError),
            ((q, k, pos, tab), dict(status=pos), ValueError),
            ((q, k, pos, table(8, 40).cuda()), {}, cp.CpattnError)):
        with pytest.raises(error):
            cp.qk_norm_rope(*args, **kw)
    with pytest.raises(ValueError):
        cp.qk_norm_rope_bwd(q, k, q, k, pos, tab, dq_weight=torch.zeros(64, device="cuda"))
    with pytest.raises(TypeError):
        cp.qk_norm_rope_bwd(q, k, None, None, pos, tab, q_weight=w, k_weight=w)
    out, lse = cp.paged_attn(**good, **bounds)
    x.check(out, lse)
