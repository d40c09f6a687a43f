"""A random sweep of the 4-bit cache's attention: sizes, head groups, pages, bounds above
the lengths, pages that are not there, sequences without new tokens; against float64 over
what cpattn_paged_gather_fp4 reads back (bit for bit the oracle's values, see
test_gpu_paged_fp4.py, which has the tolerance and its reasons)."""

import random

import pytest
import torch

from test_gpu_paged_fp4 import MANY, cp, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def spread(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


@pytest.mark.parametrize("seed", range(60))
def test_random(cp, seed):  # noqa: F811
    rng = random.Random(seed)
    g = torch.Generator("cuda").manual_seed(seed)
    D, Hk = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 33])
    size, B = rng.choice([16, 32, 64, 128, 256]), spread(rng, 1, 80)
    most = spread(rng, 1, rng.choice([2, 6, 20, 60]))
    ctx = spread(rng, 1, max(2, 30000 // B))
    new = [rng.randint(0, most) for _ in range(B)]
    new[rng.randrange(B)] = most
    kv = [n + rng.randint(0, ctx) if rng.random() < 0.95 else rng.randint(0, 3) for n in new]
    bounds = dict(max_seqlen=most + rng.choice([0, 0, 3]),
                  max_kv_len=max(kv) + rng.choice([0, 0, 1000, 50000]))
    causal = rng.random() < 0.8
    counts = [-(-n // size) for n in kv]
    pages = sum(counts) + 2
    order = torch.randperm(pages - 1, generator=g, device="cuda").cpu()
    table = torch.full((B, max(counts + [1]) + 1), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c

    def cache():
        shape = (pages, Hk, size // 16, 9 * D)
        c = torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8)
        c[..., 8 * D:] = torch.randint(0x2E, 0x3E, shape[:3] + (D,), generator=g,
                                       device="cuda").to(torch.uint8)
        c[-1] = 0   # in the place of pages that are not there
        return c.view(pages, Hk, size, 9 * D // 16)

    kc, vc = cache(), cache()
    good = table.clone()
    bad = False
    for _ in range(rng.choice([0, 0, 1, 3])):
        b = rng.randrange(B)
        if counts[b]:
            j = rng.randrange(counts[b])
            table[b, j], good[b, j] = rng.choice([-1, pages, 2 ** 31 - 1]), pages - 1
            bad = bad or new[b] > 0
    T, units = sum(new), dict(k_scale=0.5, v_scale=2.0)
    q = (0.6 * torch.randn(T + 3, H, D, generator=g, device="cuda")).to(torch.bfloat16)
    cu = i32([0] + new).cumsum(0, dtype=torch.int32)
    ws = cp.alloc_paged_fp4_workspace(T + 3, B, H, Hk, D, bounds["max_seqlen"], bounds["max_kv_len"])
    ws.random_(0, 256)
    args = (q, kc, vc, table.cuda(), cu, i32(kv))
    out, lse = cp.paged_attn_fp4(*args, causal=causal, workspace=ws, **bounds, **units)
    assert cp.poll_error(ws) == (cp.ERR_INVALID_ARG if bad else cp.OK)
    again = cp.paged_attn_fp4(*args, causal=causal, **bounds, **units)
    assert torch.equal(again[0][:T], out[:T]) and torch.equal(again[1][:T], lse[:T])

    whole = i32([0] + kv).cumsum(0, dtype=torch.int32)
    k, v = cp.paged_gather_fp4(kc, vc, good.cuda(), whole, i32(kv), total_tokens=sum(kv), **units)
    N, scale = max(kv), D ** -0.5
    many = bounds["max_seqlen"] * H // Hk > MANY
    faint = N * 2.0 ** (-32 if many else -36) * (v.abs().max().double() if N else 0)
    row = first = 0
    for n, total in zip(new, kv):
        kb, vb = k[first:first + total].double(), v[first:first + total].double()
        qb = q[row:row + n].double().view(n, Hk, H // Hk, D)
        s = scale * torch.einsum("nhgd,khd->hgnk", qb, kb)
        span = scale * torch.einsum("nhgd,khd->hgnk", qb.abs(), kb.abs())
        hidden = (torch.arange(total, device="cuda")
                  > torch.arange(total - n, total, device="cuda")[:, None]) if causal else None
        if causal:
            s, span = s.masked_fill(hidden, -torch.inf), span.masked_fill(hidden, 0)
        ref_lse = torch.logsumexp(s, -1)
        p = (s - ref_lse[..., None]).exp().nan_to_num(0)
        ref = torch.einsum("hgnk,khd->nhgd", p, vb).reshape(n, H, D)
        width = torch.einsum("hgnk,khd->nhgd", p, vb.abs()).reshape(n, H, D)
        ref_lse = ref_lse.permute(2, 0, 1).reshape(n, H)
        top = span.amax(-1) if total else torch.zeros(Hk, H // Hk, n, device="cuda")
        e = (D * 2.0 ** -24 * top.permute(2, 0, 1).reshape(n, H) + 2.0 ** -18
             + (N / 32 + 700) * 2.0 ** -24)
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e[..., None]) * width + faint
        assert ((out[row:row + n].double() - ref).abs() <= tol).all()
        got = lse[row:row + n].double()
        seen = torch.isfinite(ref_lse)
        assert torch.equal(torch.isneginf(got), ~seen)
        assert ((got - ref_lse).abs()[seen] <= (e + 2.0 ** -22 * ref_lse.abs())[seen]).all()
        row, first = row + n, first + total
