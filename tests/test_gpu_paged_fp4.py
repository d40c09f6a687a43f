"""GPU parity of the 4-bit paged KV cache (cpattn_paged_append_fp4,
cpattn_paged_gather_fp4, cpattn_paged_attn_fp4) against oracle/paged_fp4.py and
oracle/paged.py.

The cache's bytes and what is read back are compared bit for bit.  The attention's
tolerances start from the cached values, which are exact.  A score is a sum of D
products in fp32: off by at most D * 2^-24 * span, with span the largest scale *
sum |q_i k_i| of the row; exponential, maximum and the weights of splits add 2^-18,
and terms of l and O are added along chains of at most N / 32 + 700 (a warp takes two
products a tile of 16 keys and every fourth step, a split has four warps, a merge
joins at most 608 splits), 2^-24 each.
With e the sum of these, numerator and denominator are both off by e.  P is rounded to
fp16 (2^-11 of each term, and of one below 2^-14 by 2^-25).  Up to 64 rows of a KV head
the row's largest p is at least 2^11, with more 2^7: f = 2^-36 or 2^-32 of it, N times.
O is rounded to bf16 once (2^-8 |O|):
|dO| <= 2^-8 |O| + (2^-11 + 2 e) size + N f max |v|, and |dLSE| <= e + 2^-22 |LSE|."""

import numpy as np
import pytest
import torch

from oracle import paged as op
from oracle import paged_fp4 as o4
from test_gpu_norm_rope import check, f64, normal, table
from test_gpu_paged import CASES

pytestmark = pytest.mark.gpu

MANY = 64  # rows of a KV head from which on the tile kernel works


@pytest.fixture(scope="module")
def cp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_gb300 import build as lib_build
    lib_build.build()
    from long_context_gb300 import cpattn
    return cpattn


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_cache(pages, Hk, size, D, rng, mean=0x38):
    """Random codes, scales about 1 (e4m3 0x38), in the library's layout: the scales are
    the last D / 16 * 16 bytes of each tile of 9 D."""
    cache = rng.integers(0, 256, (pages, Hk, size // 16, 9 * D)).astype(np.uint8)
    cache[..., 8 * D:] = rng.integers(mean - 12, mean + 9, cache[..., 8 * D:].shape)
    return cache.reshape(pages, Hk, size, 9 * D // 16)


class Batch4:
    """A 4-bit paged batch: shuffled pages, table entries behind the last page wild,
    what lies behind kv_len random bytes with NaN for scales."""

    def __init__(self, new, kv, H, Hk, D, size, seed, std=0.3, pad=0, units=(1.0, 1.0),
                 spoil=True):
        self.new, self.kv, self.H, self.Hk, self.D, self.size = new, kv, H, Hk, D, size
        rng = np.random.default_rng(seed)
        counts = [-(-n // size) for n in kv]
        pages = sum(counts) + 2
        order = rng.permutation(pages)
        self.table = np.full((len(kv), max(counts + [1]) + 1), 2 ** 30, dtype=np.int32)
        self.kc = random_cache(pages, Hk, size, D, rng)
        self.vc = random_cache(pages, Hk, size, D, rng)
        self.units = units
        used = 0
        behind = []
        for b, c in enumerate(counts):
            self.table[b, :c] = order[used:used + c]
            used += c
            if spoil:
                behind += [(int(self.table[b, c - 1]), r) for r in range(kv[b] % size or size, size)
                           if c]
        self.k, self.v = o4.unpack(self.kc, D, units[0]), o4.unpack(self.vc, D, units[1])
        at = [o4.scale_place(r, j, D) for r in range(size) for j in range(D // 16)]
        for page, r in behind:
            self.kc[page].reshape(Hk, -1)[:, at[r * D // 16:(r + 1) * D // 16]] = 0x7F
            self.vc[page].reshape(Hk, -1)[:, at[r * D // 16:(r + 1) * D // 16]] = 0xFF
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad
        self.q = normal(self.T, H, D, seed=seed + 2, std=std / units[0])
        self.scale = D ** -0.5

    def on_gpu(self):
        return (self.q.cuda(), torch.from_numpy(self.kc).cuda(), torch.from_numpy(self.vc).cuda(),
                i32(self.table), i32(self.cu), i32(self.kv))

    def bounds(self):
        return dict(max_seqlen=max(self.new), max_kv_len=max(self.kv), k_scale=self.units[0],
                    v_scale=self.units[1])

    def check(self, out, lse, causal=True, bound=None):
        ref, rl, size, span = op.attention(f64(self.q), self.k, self.v, self.table, self.cu,
                                           self.kv, self.scale, causal)
        n = int(self.cu[-1])
        ref, rl, size, span = ref[:n], rl[:n], size[:n], span[:n]
        N = max(self.kv)
        e = self.D * 2.0 ** -24 * span + 2.0 ** -18 + (N / 32 + 700) * 2.0 ** -24
        many = (bound or max(self.new)) * self.H // self.Hk > MANY
        tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * e[..., None]) * size
               + N * 2.0 ** (-32 if many else -36) * np.abs(self.v).max())
        check(out[:n], ref, tol, "O")
        got = f64(lse[:n])
        assert np.array_equal(np.isneginf(got), np.isneginf(rl))
        fin = np.isfinite(rl)
        assert np.all(f64(out[:n])[~fin] == 0)
        d = np.abs(got[fin] - rl[fin])
        assert np.all(d <= e[fin] + 2.0 ** -22 * np.abs(rl[fin])), d.max()


# ---------------------------------------------------------- append, gather --

def appended(x, k, v):
    """The caches of ``x`` after the new tokens, from the oracle."""
    kc, vc = x.kc.copy(), x.vc.copy()
    for cache, rows, u in ((kc, k, x.units[0]), (vc, v, x.units[1])):
        code, scale = o4.quantise(rows, u)
        for (i, _, _, page, row) in op.places(x.cu, x.kv, x.table, x.size):
            for h in range(x.Hk):
                o4.write(cache, page, h, row, code[i, h], scale[i, h])
    return kc, vc


APPENDS = [
    ([1], [1], 1, 64, 16, (1.0, 1.0)),
    ([1, 1, 1], [1, 16, 17], 2, 128, 16, (1.0, 1.0)),
    ([5, 0, 1, 40], [9, 3, 100, 40], 5, 64, 32, (0.25, 8.0)),
    ([33, 2], [40, 66], 3, 128, 64, (2.0 ** -20, 2.0 ** 12)),
    ([7, 3], [7, 300], 9, 64, 256, (1.0, 0.125)),
    ([19] * 40, [19 + b for b in range(40)], 1, 128, 128, (1.0, 1.0)),
    ([70, 1], [75, 130], 4, 128, 128, (0.5, 4.0)),
]


@pytest.mark.parametrize("new,kv,Hk,D,size,units", APPENDS)
def test_append_and_gather(cp, new, kv, Hk, D, size, units):
    x = Batch4(new, kv, Hk, Hk, D, size, seed=sum(kv), pad=3, units=units)
    _, kc, vc, t, cu, kvl = x.on_gpu()
    rows = normal(x.T, 4 * Hk, D, seed=5, std=1.5).cuda()
    # Magnitudes over many powers of two, groups of zeros, features on a border.
    rows *= torch.exp2(torch.randint(-14, 12, (x.T, 4 * Hk, 1), device="cuda",
                                     generator=torch.Generator("cuda").manual_seed(1))).to(
                                         torch.bfloat16)
    rows[::5, :, :16] = 0
    rows[1::4, :, 16:32] = torch.tensor([6, -5, 3.5, 2.5, 1.75, -1.25, 0.75, 0.25] * 2).cuda().to(
        torch.bfloat16)
    rows[2::4, :, 32:48] *= 0.0
    rows[2::4, :, 32:40] = -0.0
    k, v = rows[:, Hk:2 * Hk], rows[:, 3 * Hk:]
    for r, u in ((k, units[0]), (v, units[1])):
        r *= u
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = dict(k_scale=units[0], v_scale=units[1], status=status)
    assert cp.paged_append_fp4(k, v, kc, vc, t, cu, kvl, **s) is None
    want_k, want_v = appended(x, f64(k), f64(v))
    assert torch.equal(kc.cpu(), torch.from_numpy(want_k))
    assert torch.equal(vc.cpu(), torch.from_numpy(want_v))
    # Back, into rows of a larger array.
    out = torch.full((x.T, 3 * Hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    gk, gv = cp.paged_gather_fp4(kc, vc, t, cu, kvl, total_tokens=x.T, k_out=out[:, :Hk],
                                 v_out=out[:, 2 * Hk:], **s)
    assert int(status) == 0
    assert gk.data_ptr() == out.data_ptr() and (out[:, Hk:2 * Hk] == 7).all()
    ref_k, ref_v = o4.unpack(want_k, D, units[0]), o4.unpack(want_v, D, units[1])
    for (i, _, _, page, row) in op.places(x.cu, kv, x.table, size):
        assert np.array_equal(f64(gk[i]), ref_k[page, row])
        assert np.array_equal(f64(gv[i]), ref_v[page, row])
    assert (out[x.cu[-1]:] == 7).all()
    fresh = cp.paged_gather_fp4(kc, vc, t, cu, kvl, total_tokens=int(x.cu[-1]), **s)
    assert torch.equal(fresh[0], gk[:x.cu[-1]]) and torch.equal(fresh[1], gv[:x.cu[-1]])


def test_every_border(cp):
    """Groups of every scale and every quotient that a bf16 feature can have to it."""
    top = torch.arange(0x3F80, 0x4000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    # A group: a largest value of 1 .. 2 and fifteen others of all mantissas below it.
    x = torch.zeros(128, 64, 16, dtype=torch.bfloat16)
    x[..., 0] = top[:, None]
    rest = (torch.arange(64 * 15) % 896 + 0x3C80).to(torch.int16).view(torch.bfloat16)
    x[..., 1:] = rest.view(64, 15)
    x[:, 1::2] *= -1
    k = x.reshape(128, 16, 64).cuda()
    t, cu, kv = i32([[0, 1, 2, 3, 4, 5, 6, 7]]), i32([0, 128]), i32([128])
    kc, vc = cp.alloc_fp4_cache(8, 16, 16, 64), cp.alloc_fp4_cache(8, 16, 16, 64)
    for unit in (1.0, 2.0 ** -32, 2.0 ** 32):
        y = k * unit
        cp.paged_append_fp4(y, -y, kc, vc, t, cu, kv, k_scale=unit, v_scale=unit)
        code, scale = o4.quantise(f64(k))
        want = o4.values(code, scale)
        gk, gv = cp.paged_gather_fp4(kc, vc, t, cu, kv, total_tokens=128, k_scale=unit,
                                     v_scale=unit)
        assert np.array_equal(f64(gk) / unit, want) and np.array_equal(f64(gv) / unit, -want)


def test_the_ends_of_the_range(cp):
    """Values below the smallest scale, above the largest, subnormal, infinite, NaN."""
    k = torch.zeros(16, 1, 64, dtype=torch.bfloat16)
    for r, v in enumerate([2.0 ** -133, 1e-38, 2.0 ** -11, 2.0 ** -10, 3 * 2.0 ** -12, 0.0117, 0.012,
                           2600.0, 2688.0, 2700.0, 1e6, 3.3e38, float("inf"), -float("inf"),
                           float("nan"), 1.0]):
        k[r, 0, :16] = torch.linspace(-1, 1, 16).to(torch.bfloat16) if np.isfinite(v) else 0.5
        k[r, 0, :16] *= v if np.isfinite(v) else 1.0
        k[r, 0, 3] = v
    kc, vc = cp.alloc_fp4_cache(1, 16, 1, 64), cp.alloc_fp4_cache(1, 16, 1, 64)
    args = (kc, vc, i32([[0]]), i32([0, 16]), i32([16]))
    for unit in (1.0, 2.0 ** -32, 2.0 ** 32):
        cp.paged_append_fp4(k.cuda(), k.cuda(), *args, k_scale=unit)
        code, scale = o4.quantise(f64(k), unit)
        gk, gv = cp.paged_gather_fp4(*args, total_tokens=16, k_scale=unit)
        assert np.array_equal(f64(gk), o4.values(code, scale, unit), equal_nan=True)
        assert np.array_equal(np.isnan(f64(gk)).all(-1)[:, 0], [False] * 12 + [False] * 4)
        assert np.isnan(f64(gk)[12:15, 0, :16]).all() and np.isfinite(f64(gk)[15]).all()
        assert np.array_equal(f64(gk)[12:, 0, 16:], np.zeros((4, 48)))


def test_append_and_gather_leave_out_bad_tokens(cp):
    x = Batch4([2, 3, 1], [40, 20, 9], 2, 2, 64, 16, seed=14, spoil=False)
    _, kc0, vc0, t, cu, kv = x.on_gpu()
    k, v = normal(6, 2, 64, seed=1).cuda(), normal(6, 2, 64, seed=2).cuda()
    good_k, good_v = kc0.clone(), vc0.clone()
    cp.paged_append_fp4(k, v, good_k, good_v, t, cu, kv)
    all_k, all_v = cp.paged_gather_fp4(good_k, good_v, t, cu, kv, total_tokens=6)
    bad_page, low_page = t.clone(), t.clone()
    bad_page[1, 1], low_page[1, 1] = kc0.shape[0], -1
    cap = 16 * t.shape[1]
    for pages, kv_, left in ((bad_page, kv, [2, 3, 4]), (low_page, kv, [2, 3, 4]),
                             (t, i32([40, 2, 9]), [2]), (t, i32([40, -5, 9]), [2, 3, 4]),
                             (t, i32([40, cap + 1, 9]), [2, 3, 4]),
                             (t, i32([40, 2 ** 31 - 1, 9]), [2, 3, 4])):
        kc, vc = kc0.clone(), vc0.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cp.paged_append_fp4(k, v, kc, vc, pages, cu, kv_, status=status)
        assert int(status) == cp.ERR_INVALID_ARG
        keep = [i for i in range(6) if i not in left]
        out = [torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        status.zero_()
        cp.paged_gather_fp4(kc, vc, pages, cu, kv_, total_tokens=6, k_out=out[0], v_out=out[1],
                            status=status)
        assert int(status) == cp.ERR_INVALID_ARG
        assert torch.equal(out[0][keep], all_k[keep]) and torch.equal(out[1][keep], all_v[keep])
        assert (out[0][left] == 7).all() and (out[1][left] == 7).all()
    for bad_cu in ([0, 2, 1, 6], [-1, 2, 5, 6], [0, 2, 5, 2 ** 31 - 1]):
        cp.paged_append_fp4(k, v, kc0.clone(), vc0.clone(), t, i32(bad_cu), kv)
        cp.paged_gather_fp4(kc0, vc0, t, i32(bad_cu), kv, total_tokens=6)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- attention --

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,kv,H,Hk,D,size", CASES)
def test_attention(cp, new, kv, H, Hk, D, size, causal):
    x = Batch4(new, kv, H, Hk, D, size, seed=sum(kv) % 97, units=(0.25, 4.0))
    ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), H, Hk, D, max(new), max(kv))
    out, lse = cp.paged_attn_fp4(*x.on_gpu(), causal=causal, workspace=ws, **x.bounds())
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse, causal)


@pytest.mark.parametrize("new,kv,H,Hk,D,size,std", [
    ([1], [9000], 4, 1, 64, 64, 0.3),                    # many splits of one token
    ([1], [9000], 12, 1, 128, 128, 0.3),                 # 9 to 16 rows
    ([1, 1], [6000, 33], 2, 2, 128, 16, 1.5),            # scores over many powers of two
    ([2, 70], [3100, 5000], 4, 2, 128, 32, 1.0),         # blocks of 32 rows beside short ones
    ([5, 3], [4000, 700], 10, 2, 64, 32, 0.3),           # up to 32 rows in splits
    ([4], [5000], 16, 2, 128, 16, 0.3),
    ([5], [20000], 5, 1, 64, 64, 0.3),                   # more splits than a round of the merge
    ([100, 60], [2600, 2000], 4, 4, 64, 16, 0.6),        # four blocks of 32 rows
    ([1] * 65, [327 + 5 * b for b in range(65)], 8, 4, 128, 16, 0.3),    # more than a plan's
    ([2] * 70, [100 + 31 * b for b in range(70)], 10, 2, 64, 64, 0.3),   # the same, 9 to 16 rows
    ([3] * 40, [2 + 60 * b for b in range(1, 41)], 16, 2, 128, 32, 0.3),  # and 17 to 32
    ([300, 10, 0, 700], [2300, 1800, 5, 2000], 16, 16, 64, 16, 0.3),     # tiles
    ([100, 40, 0, 300], [1300, 800, 5, 1000], 8, 2, 128, 256, 0.3),
])
def test_long_caches(cp, new, kv, H, Hk, D, size, std):
    x = Batch4(new, kv, H, Hk, D, size, seed=3, std=std)
    args = x.on_gpu()
    ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), H, Hk, D, max(new), max(kv))
    out, lse = cp.paged_attn_fp4(*args, **x.bounds())
    x.check(out, lse)
    again = cp.paged_attn_fp4(*args, workspace=ws, **x.bounds())
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)  # a fixed order of sums
    assert cp.poll_error(ws) == cp.OK


def test_many_sequences(cp):
    rng = np.random.default_rng(4)
    new = [int(n) for n in rng.integers(0, 3, 1500)]
    kv = [n + int(c) for n, c in zip(new, rng.integers(0, 20, 1500))]
    x = Batch4(new, kv, 2, 1, 64, 16, seed=9)
    out, lse = cp.paged_attn_fp4(*x.on_gpu(), **x.bounds())
    x.check(out, lse)


def test_padded_batch_and_larger_bounds(cp):
    """Rows behind the last sequence stay, and bounds above the lengths choose other
    kernels and splits for the same answer."""
    for new, bound in (([1, 2, 1], 2), ([1, 2, 1], 4), ([1, 2, 1], 9), ([1, 2, 1], 32),
                       ([1, 2, 1], 400), ([30, 1, 0], 2000)):
        x = Batch4(new, [40, 1100, 17], 8, 2, 128, 16, seed=6, pad=5)
        out = torch.full((x.T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((x.T, 8), 7.0, device="cuda")
        cp.paged_attn_fp4(*x.on_gpu(), max_seqlen=bound, max_kv_len=5000, out=out, lse=lse)
        x.check(out, lse, bound=bound)
        assert (out[x.cu[-1]:] == 7).all() and (lse[x.cu[-1]:] == 7).all()


def test_caches_inside_a_larger_tensor(cp):
    """K and V pages side by side, [pages, 2, Hk, size, 9 D / 16]."""
    x = Batch4([2, 1], [70, 33], 4, 2, 64, 32, seed=7)
    q, kc, vc, t, cu, kv = x.on_gpu()
    both = torch.stack([kc, vc], 1)
    for bound in (2, 9, 20, 200):
        out, lse = cp.paged_attn_fp4(q, both[:, 0], both[:, 1], t, cu, kv, max_seqlen=bound,
                                     max_kv_len=70)
        x.check(out, lse, bound=bound)
    k, v = normal(3, 2, 64, seed=1).cuda(), normal(3, 2, 64, seed=2).cuda()
    cp.paged_append_fp4(k, v, both[:, 0], both[:, 1], t, cu, kv)
    cp.paged_append_fp4(k, v, kc, vc, t, cu, kv)
    assert torch.equal(both, torch.stack([kc, vc], 1))
    a = cp.paged_gather_fp4(both[:, 0], both[:, 1], t, cu, kv, total_tokens=3)
    b = cp.paged_gather_fp4(kc, vc, t, cu, kv, total_tokens=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bound", [1, 40])
def test_queries_of_all_magnitudes(cp, bound):
    """Rows from 2^-100 to 2^100 with features 2^20 apart, one of them zero: a row's
    power of two keeps them exact.  (A feature that is below 2^-28 of its row's largest
    may lose bits: 2^-39 of the largest, here under 2^-18 of the span.)"""
    x = Batch4([1] * 6, [200, 33, 64, 500, 16, 90], 8, 2, 64, 16, seed=21)
    spread = torch.exp2(torch.randint(-20, 1, (6, 8, 64), generator=torch.Generator().manual_seed(2))
                        .float())
    row = torch.exp2(torch.linspace(-100, 100, 48).round()).view(6, 8, 1)
    x.q = (x.q.float() * spread * row).to(torch.bfloat16)
    x.q[1, 3] = 0
    x.scale = 2.0 ** -3
    for scale_row in range(6):
        s = float(2.0 ** -3 / row[scale_row].mean())
        if not 2.0 ** -100 < s < 2.0 ** 100:
            continue
        y = Batch4([1] * 6, x.kv, 8, 2, 64, 16, seed=21)
        y.q = x.q.clone()
        y.q[[i for i in range(6) if i != scale_row]] = 0
        y.scale = s
        out, lse = cp.paged_attn_fp4(*y.on_gpu(), max_seqlen=bound, max_kv_len=500,
                                     softmax_scale=s)
        y.check(out, lse, bound=bound)


def test_rising_scores_and_one_far_key(cp):
    """The reference moves many times; and one key outweighs 2^17 faint ones whose
    share is still seen."""
    x = Batch4([1], [3000], 4, 1, 128, 64, seed=22, spoil=False)
    kc = cp.alloc_fp4_cache(x.kc.shape[0], 64, 1, 128)
    vc = torch.from_numpy(x.vc).cuda()
    _, _, _, t, cu, kv = x.on_gpu()
    for order in (1, -1):
        k = torch.ones(3000, 1, 128) * torch.linspace(-2 * order, 2 * order, 3000).reshape(-1, 1, 1)
        k = k.to(torch.bfloat16).cuda()
        cp.paged_append_fp4(k, k, kc, torch.empty_like(kc), t, i32([0, 3000]), kv)
        x.k = o4.unpack(kc.cpu().numpy(), 128)
        x.q = torch.full((1, 4, 128), 1.5, dtype=torch.bfloat16)
        out, lse = cp.paged_attn_fp4(x.q.cuda(), kc, vc, t, cu, kv, **x.bounds())
        x.check(out, lse)
    N = 131072
    kc, vc = cp.alloc_fp4_cache(N // 256, 256, 1, 64), cp.alloc_fp4_cache(N // 256, 256, 1, 64)
    k = torch.zeros(N, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    k[77] = 6.0
    v[77] = 0.0
    t = torch.arange(N // 256, dtype=torch.int32, device="cuda")[None]
    cp.paged_append_fp4(k, v, kc, vc, t, i32([0, N]), i32([N]))
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    one = float(o4.values(*o4.quantise(np.ones(16)))[0])    # as the cache holds it
    assert o4.values(*o4.quantise(np.full(16, 6.0)))[0] == 6
    for far in (8, 16, 20, 24):    # powers of two between the far key and the others
        s = far * np.log(2.0) / (6 * 64)
        out, lse = cp.paged_attn_fp4(q, kc, vc, t, i32([0, 1]), i32([N]), max_seqlen=1,
                                     max_kv_len=N, softmax_scale=s)
        share = (N - 1) * 2.0 ** -far
        want = one * share / (1 + share)
        e = 2.0 ** -18 + 64 * 2.0 ** -24 * far + (N / 32 + 700) * 2.0 ** -24
        tol = 2.0 ** -8 * want + (2.0 ** -11 + 2 * e) * want + N * 2.0 ** -36 * one
        assert (out.double() - want).abs().max() <= tol
        assert abs(float(lse) - (far * np.log(2.0) + np.log1p(share))) <= e + 2.0 ** -22 * float(lse)


def test_bad_lengths_and_pages(cp):
    x = Batch4([1, 2], [40, 50], 4, 2, 64, 16, seed=10)
    q, kc, vc, t, cu, kv = x.on_gpu()
    for bound in (2, 20, 300):
        ws = cp.alloc_paged_fp4_workspace(x.T, 2, 4, 2, 64, bound, 4000)
        for bad_cu, bad_kv, bad_bound in (
                ([0, 1, 3], [40, -1], 50), ([0, 1, 3], [40, 51], 50), ([0, 1, 4], [40, 50], 50),
                ([0, 2, 1], [40, 50], 50), ([1, 1, 3], [40, 50], 50),
                ([0, 1, 3], [40, 16 * t.shape[1] + 1], 4000)):
            out = torch.full_like(q, 7.0)
            cp.paged_attn_fp4(q, kc, vc, t, i32(bad_cu), i32(bad_kv), max_seqlen=bound,
                              max_kv_len=bad_bound, out=out, workspace=ws)
            assert cp.poll_error(ws) == cp.ERR_INVALID_ARG and (out == 7).all()
        out, lse = cp.paged_attn_fp4(q, kc, vc, t, cu, kv, max_seqlen=bound, max_kv_len=50,
                                     workspace=ws)
        assert cp.poll_error(ws) == cp.OK
        x.check(out, lse, bound=bound)
        want = out
        for page in (-1, kc.shape[0], 2 ** 31 - 1):
            bad = t.clone()
            bad[1, 1] = page
            out, lse = cp.paged_attn_fp4(q, kc, vc, bad, cu, kv, max_seqlen=bound, max_kv_len=50,
                                         workspace=ws)
            assert cp.poll_error(ws) == cp.ERR_INVALID_ARG
            assert torch.equal(out[:1], want[:1])
            # That page's keys and values count as zeros.
            y = Batch4([1, 2], [40, 50], 4, 2, 64, 16, seed=10)
            gone = int(y.table[1, 1])
            y.k[gone], y.v[gone] = 0, 0
            y.check(out, lse, bound=bound)


def test_no_work(cp):
    x = Batch4([0, 0], [5, 0], 4, 2, 64, 16, seed=12)
    q, kc, vc, t, cu, kv = x.on_gpu()
    ws = cp.alloc_paged_fp4_workspace(0, 2, 4, 2, 64, 1, 5)
    out, lse = cp.paged_attn_fp4(q, kc, vc, t, cu, kv, max_seqlen=1, max_kv_len=5, workspace=ws)
    assert out.shape == (0, 4, 64) and cp.poll_error(ws) == cp.OK
    out, _ = cp.paged_attn_fp4(q, kc, vc, t[:0], cu[:1], kv[:0], max_seqlen=1, max_kv_len=0)
    assert out.shape == (0, 4, 64)
    gk, gv = cp.paged_gather_fp4(kc, vc, t, cu, kv, total_tokens=0)
    assert gk.shape == gv.shape == (0, 2, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cp.paged_append_fp4(none, none, kc, vc, t, cu, kv)
    # Rows without a key.
    for bound in (1, 40, 200):
        ws = cp.alloc_paged_fp4_workspace(2, 2, 4, 2, 64, bound, 0)
        out, lse = cp.paged_attn_fp4(torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda"), kc,
                                     vc, t, i32([0, 1, 2]), i32([0, 0]), max_seqlen=bound,
                                     max_kv_len=0, workspace=ws)
        assert cp.poll_error(ws) == cp.OK
        assert (out == 0).all() and torch.isneginf(lse).all()


# ----------------------------------------------------------------- together --

@pytest.mark.parametrize("H,Hk,D", [(8, 2, 64), (10, 2, 128)])
def test_a_prompt_in_chunks_then_tokens(cp, H, Hk, D):
    """As a server runs them: norm + rotation, append, attention, and read back; each
    step's output against attention in 64 bits over what the cache then holds, and the
    4-bit cache's kernels against the bf16 cache's over the values read back."""
    size, total = 16, [75, 41]
    rng = np.random.default_rng(0)
    x = [normal(n, H + 2 * Hk, D, seed=30 + b) for b, n in enumerate(total)]
    tab = table(128, D).cuda()
    w = (1 + 0.3 * normal(D, seed=3).float()).to(torch.bfloat16).cuda()
    pages = 16
    t = torch.from_numpy(rng.permutation(pages)[:12].reshape(2, 6).astype(np.int32)).cuda()
    kc, vc = (torch.full((pages, Hk, size, 9 * D // 16), 0x7F, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    units = dict(k_scale=0.5, v_scale=0.25)
    done = [0, 0]
    for step in ([40, 1], [20, 30], [0, 8], [1, 1], [14, 1]):
        new = [min(s, n - d) for s, n, d in zip(step, total, done)]
        qkv = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(2)]).cuda()
        pos = torch.cat([torch.arange(d, d + n, dtype=torch.int32) for d, n in zip(done, new)])
        done = [d + n for d, n in zip(done, new)]
        cu, kv = i32([0, new[0], new[0] + new[1]]), i32(done)
        q, k = cp.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hk], pos.cuda(), tab, q_weight=w,
                               k_weight=w)
        cp.paged_append_fp4(k, qkv[:, H + Hk:], kc, vc, t, cu, kv, **units)
        out, lse = cp.paged_attn_fp4(q, kc, vc, t, cu, kv, max_seqlen=max(new),
                                     max_kv_len=max(done), **units)
        b = Batch4(new, done, H, Hk, D, size, seed=1, spoil=False)
        b.q, b.table = q, t.cpu().numpy()
        b.k = np.nan_to_num(o4.unpack(kc.cpu().numpy(), D, 0.5))
        b.v = np.nan_to_num(o4.unpack(vc.cpu().numpy(), D, 0.25))
        b.check(out, lse)
    assert done == total
    # The whole caches as packed keys and values: the packed decode over them.
    cu, kv = i32([0, total[0], sum(total)]), i32(total)
    k, v = cp.paged_gather_fp4(kc, vc, t, cu, kv, total_tokens=sum(total), **units)
    rep = lambda a: a.repeat_interleave(H // Hk, 1).contiguous()  # noqa: E731
    q1 = normal(2, H, D, seed=9).cuda()
    one, lse1 = cp.paged_attn_fp4(q1, kc, vc, t, i32([0, 1, 2]), kv, max_seqlen=1, max_kv_len=75,
                                  **units)
    ref, lse2 = cp.decode(q1, rep(k), rep(v), cu, cp=1)
    # Both are within 2^-8 |O| + 2^-8 size of the exact value, and |v| <= 5 bounds size.
    assert (one.float() - ref.float()).abs().max() <= 2 * 2 ** -8 * (ref.abs().max().float() + 5)
    assert (lse1 - lse2).abs().max() <= 2 ** -12


def test_streams_graphs_and_two_workspaces(cp):
    """A captured decoding step -- append, attention, read back -- replayed with other
    lengths and tokens, beside calls on another stream with a workspace of their own."""
    for new, H, most in (([1, 1, 1], 8, 700), ([1, 2, 3], 20, 700), ([40, 1, 1], 8, 700),
                         ([1, 1, 1], 8, 30000), ([1, 2, 3], 20, 30000), ([1, 2, 12], 8, 30000)):
        x = Batch4(new, [700, 20, 333], H, 2, 128, 16, seed=15, spoil=False)
        q, kc, vc, t, cu, kv = x.on_gpu()
        k, v = normal(x.T, 2, 128, seed=1).cuda(), normal(x.T, 2, 128, seed=2).cuda()
        first = kv.clone()
        bounds = dict(max_seqlen=max(new), max_kv_len=most)
        kc1, vc1 = kc.clone(), vc.clone()
        cp.paged_append_fp4(k, v, kc1, vc1, t, cu, first)
        ref = cp.paged_attn_fp4(q, kc1, vc1, t, cu, first, **bounds)
        back = cp.paged_gather_fp4(kc1, vc1, t, cu, first, total_tokens=x.T)
        kvs = i32([max(n, 3) for n in new])
        ins = torch.zeros_like(k), torch.zeros_like(v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cp.paged_append_fp4(*ins, kc, vc, t, cu, kvs)
            cap = cp.paged_attn_fp4(q, kc, vc, t, cu, kvs, **bounds)
            got = cp.paged_gather_fp4(kc, vc, t, cu, kvs, total_tokens=x.T)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            kvs.copy_(first)
            ins[0].copy_(k)
            ins[1].copy_(v)
            graph.replay()
            other = cp.paged_attn_fp4(q, kc1, vc1, t, cu, first, stream=s, **bounds)
            gath = cp.paged_gather_fp4(kc1, vc1, t, cu, first, total_tokens=x.T, stream=s)
        torch.cuda.synchronize()
        for r in (cap, other):
            assert torch.equal(r[0], ref[0]) and torch.equal(r[1], ref[1])
        for r in (got, gath):
            assert torch.equal(r[0], back[0]) and torch.equal(r[1], back[1])
        assert torch.equal(kc, kc1) and torch.equal(vc, vc1)


def test_a_cache_past_32_bit_offsets(cp):
    """Pages whose byte offsets lie beyond 2^32."""
    H, Hk, D, size = 8, 8, 128, 256
    pages = 2 ** 32 // (size * Hk * 9 * D // 16) + 64
    kc = torch.zeros(pages, Hk, size, 9 * D // 16, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    x = Batch4([1, 200], [600, 500], H, Hk, D, size, seed=16, spoil=False)
    table_ = np.full((2, 3), -1, dtype=np.int32)
    table_[0], table_[1, :2] = [pages - 1, pages - 5, 1], [pages - 2, pages - 3]
    for b in range(2):
        for i in range(-(-x.kv[b] // size)):
            kc[int(table_[b, i])] = torch.from_numpy(x.kc[x.table[b, i]]).cuda()
            vc[int(table_[b, i])] = torch.from_numpy(x.vc[x.table[b, i]]).cuda()
    _, _, _, _, cu, kv = x.on_gpu()
    t = torch.from_numpy(table_).cuda()
    out, lse = cp.paged_attn_fp4(x.q.cuda(), kc, vc, t, cu, kv, **x.bounds())
    x.check(out, lse)
    y = Batch4([1, 1], [600, 500], H, Hk, D, size, seed=16, spoil=False)
    y.q = x.q[[0, x.T - 1]]
    few = cp.paged_attn_fp4(y.q.cuda(), kc, vc, t, i32([0, 1, 2]), kv, **y.bounds())
    y.check(*few)
    k, v = normal(x.T, Hk, D, seed=1).cuda(), normal(x.T, Hk, D, seed=2).cuda()
    cp.paged_append_fp4(k, v, kc, vc, t, cu, kv)
    gk, gv = cp.paged_gather_fp4(kc, vc, t, cu, kv, total_tokens=x.T)
    for got, src in ((gk, k), (gv, v)):
        assert np.array_equal(f64(got), o4.values(*o4.quantise(f64(src))))


def test_refused_tensors(cp):
    """Types, shapes, layouts and scales are refused before anything is enqueued."""
    x = Batch4([2, 1], [40, 20], 4, 2, 64, 16, seed=19)
    q, kc, vc, t, cu, kv = x.on_gpu()
    k = normal(3, 2, 64, seed=1).cuda()
    good = dict(q=q, k_cache=kc, v_cache=vc, page_table=t, cu_seqlens=cu, kv_lens=kv)
    bounds = dict(max_seqlen=2, max_kv_len=40)
    bf16 = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for change, error in (
            (dict(q=q.float()), TypeError), (dict(q=q.cpu()), ValueError),
            (dict(q=q.transpose(0, 1)), ValueError), (dict(q=q[..., :32].contiguous()), ValueError),
            (dict(k_cache=bf16), TypeError), (dict(k_cache=kc[:-1]), ValueError),
            (dict(v_cache=vc.transpose(1, 2)), ValueError), (dict(k_cache=kc[..., 0]), ValueError),
            (dict(k_cache=kc.cpu()), ValueError), (dict(k_cache=kc[:, :1]), ValueError),
            (dict(page_table=t.long()), TypeError), (dict(page_table=t[:1]), ValueError),
            (dict(cu_seqlens=cu[:-1]), ValueError), (dict(kv_lens=kv.long()), TypeError),
            (dict(k_cache=kc[..., :27].contiguous()), ValueError)):
        with pytest.raises(error):
            cp.paged_attn_fp4(**{**good, **change}, **bounds)
    small = torch.zeros(512, dtype=torch.uint8, device="cuda")
    for change, status in ((dict(out=q), cp.ERR_INVALID_ARG), (dict(k_scale=3.0), cp.ERR_INVALID_ARG),
                           (dict(v_scale=0.0), cp.ERR_INVALID_ARG),
                           (dict(v_scale=-1.0), cp.ERR_INVALID_ARG),
                           (dict(k_scale=2.0 ** 33), cp.ERR_INVALID_ARG),
                           (dict(k_scale=float("nan")), cp.ERR_INVALID_ARG),
                           (dict(softmax_scale=1e38, k_scale=2.0 ** 20), cp.ERR_INVALID_ARG),
                           (dict(workspace=small), cp.ERR_WORKSPACE_TOO_SMALL)):
        with pytest.raises(cp.CpattnError) as e:
            cp.paged_attn_fp4(**good, **{**bounds, **change})
        assert e.value.status == status
    for args, kw, error in (
            ((k, k[:2], kc, vc, t, cu, kv), {}, ValueError),
            ((k, k, kc, kc, t, cu, kv), {}, cp.CpattnError),
            ((k, k, bf16, bf16, t, cu, kv), {}, TypeError),
            ((k, k, kc[:, :1], vc[:, :1], t, cu, kv), {}, ValueError),
            ((k, k, kc, vc, t, cu, kv), dict(k_scale=1.5), cp.CpattnError),
            ((k, k, kc, vc, t, cu, kv), dict(status=kv), ValueError),
            ((k.transpose(0, 1).contiguous().transpose(0, 1), k, kc, vc, t, cu, kv), {}, ValueError)):
        with pytest.raises(error):
            cp.paged_append_fp4(*args, **kw)
    for kw, error in ((dict(total_tokens=-1), ValueError), (dict(total_tokens="x"), TypeError),
                      (dict(total_tokens=3, k_out=k[:2]), ValueError),
                      (dict(total_tokens=3, k_out=k, v_out=k), cp.CpattnError),
                      (dict(total_tokens=3, v_scale=0.3), cp.CpattnError),
                      (dict(total_tokens=3, v_out=k.float()), TypeError)):
        with pytest.raises(error):
            cp.paged_gather_fp4(kc, vc, t, cu, kv, **kw)
    with pytest.raises(ValueError):
        cp.paged_gather_fp4(kc.cpu(), vc, t, cu, kv, total_tokens=3)
    with pytest.raises(cp.CpattnError):
        cp.alloc_fp4_cache(4, 16, 2, 96)
    out, lse = cp.paged_attn_fp4(**good, **bounds)
    x.check(out, lse)


@pytest.mark.parametrize("bound", [1, 5, 12, 40])
def test_bounds_far_above_the_lengths(cp, bound):
    """A captured program's bounds: a million keys, more sequences than have keys."""
    x = Batch4([1, 0, 1, 1], [300, 0, 7, 129], 8, 2, 64, 32, seed=33)
    ws = cp.alloc_paged_fp4_workspace(x.T, 4, 8, 2, 64, bound, 1 << 20)
    out, lse = cp.paged_attn_fp4(*x.on_gpu(), max_seqlen=bound, max_kv_len=1 << 20, workspace=ws)
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse, bound=bound)


def test_two_calls_and_two_workspaces_at_once(cp):
    """Two streams, each with its own workspace, in every form of the work list."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    for new, kv, bound in (([1, 1], [900, 70], 900), ([1, 1], [900, 70], 30000),
                           ([4, 3], [900, 70], 30000), ([1] * 40, [60 + b for b in range(40)], 99),
                           ([1] * 40, [60 + b for b in range(40)], 30000), ([30, 40], [900, 70], 900)):
        xs = [Batch4(new, kv, 10, 2, 128, 16, seed=41 + i) for i in range(2)]
        args = [x.on_gpu() for x in xs]
        ws = [cp.alloc_paged_fp4_workspace(x.T, len(kv), 10, 2, 128, max(new), bound) for x in xs]
        torch.cuda.synchronize()
        outs = [None, None]
        for _ in range(3):
            for i in range(2):
                outs[i] = cp.paged_attn_fp4(*args[i], max_seqlen=max(new), max_kv_len=bound,
                                            workspace=ws[i], stream=streams[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert cp.poll_error(ws[i]) == cp.OK
            xs[i].check(*outs[i])


@pytest.mark.parametrize("D", [64, 128])
def test_rising_scores_of_many_rows(cp, D):
    """The tile kernel's references move with every key tile, up and far up; and stay
    where the scores fall."""
    x = Batch4([40], [2000], 4, 1, D, 64, seed=23, spoil=False)
    _, _, vc, t, cu, kv = x.on_gpu()
    kc, junk = cp.alloc_fp4_cache(x.kc.shape[0], 64, 1, D), cp.alloc_fp4_cache(x.kc.shape[0], 64, 1, D)
    for top in (2.0, -2.0, 30.0):
        k = (torch.ones(2000, 1, D) * torch.linspace(-top, top, 2000).reshape(-1, 1, 1)).to(
            torch.bfloat16).cuda()
        cp.paged_append_fp4(k, k, kc, junk, t, i32([0, 2000]), kv)
        x.k = o4.unpack(kc.cpu().numpy(), D)
        x.q = torch.full((40, 4, D), 1.5, dtype=torch.bfloat16)
        x.q[3] = -1.5
        out, lse = cp.paged_attn_fp4(x.q.cuda(), kc, vc, t, cu, kv, **x.bounds())
        x.check(out, lse)


@pytest.mark.parametrize("size", [64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_splits_that_start_inside_a_page(cp, D, size):
    """Splits begin at multiples of 64 keys, steps have up to 128, pages up to 256: by
    the plan, by the list and in the parts of a cluster, for 8, 16 and 32 rows."""
    for new, kv, H, Hk, bound in (([1, 2], [5000, 3333], 4, 4, 60000), ([1], [16000], 2, 2, 60000),
                                  ([1] * 40, [1700 + 64 * b for b in range(40)], 8, 8, 60000),
                                  ([1, 1, 1], [961, 700, 1023], 4, 4, 1023),
                                  ([1], [450], 2, 1, 500), ([3], [900], 4, 1, 1000),
                                  ([5, 3], [2900, 4000], 10, 2, 60000),
                                  ([20], [3000], 3, 1, 60000)):
        x = Batch4(new, kv, H, Hk, D, size, seed=51)
        ws = cp.alloc_paged_fp4_workspace(x.T, len(kv), H, Hk, D, max(new), bound)
        out, lse = cp.paged_attn_fp4(*x.on_gpu(), max_seqlen=max(new), max_kv_len=bound,
                                     workspace=ws)
        assert cp.poll_error(ws) == cp.OK
        x.check(out, lse)


@pytest.mark.parametrize("bound,most", [(1, 700), (1, 30000), (12, 30000), (100, 700)])
def test_sequences_without_new_tokens_are_not_read(cp, bound, most):
    """Their page table may hold anything: a server's sequences that pause a step."""
    x = Batch4([1, 0, 1, 0], [200, 700, 65, 300], 8, 2, 64, 32, seed=61)
    q, kc, vc, t, cu, kv = x.on_gpu()
    t[1], t[3] = 2 ** 30, -5
    ws = cp.alloc_paged_fp4_workspace(x.T, 4, 8, 2, 64, bound, most)
    out, lse = cp.paged_attn_fp4(q, kc, vc, t, cu, kv, max_seqlen=bound, max_kv_len=most,
                                 workspace=ws)
    assert cp.poll_error(ws) == cp.OK
    x.check(out, lse, bound=bound)
