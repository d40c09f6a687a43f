"""Refusals of the 4-bit cache's calls and the sizes of its workspaces, on the host
(see test_serve_refusals.py)."""

import random

import pytest

from test_serve_refusals import INVALID, SMALL, UNSUPPORTED, call, cp, mem  # noqa: F401

NAN, INF = float("nan"), float("inf")


def append(p):
    return dict(k=p, ks=256, v=p, vs=256, kc=p, vc=p + 16384, pages=3, size=16,
                stride=16 * 4 * 36, table=p, max_pages=4, cu=p, kv=p, B=2, T=4, Hk=4, D=64, ku=1.0,
                vu=1.0, status=None, stream=None)


def gather(p):
    return dict(kc=p, vc=p + 16384, pages=3, size=16, stride=16 * 4 * 36, table=p, max_pages=4, cu=p,
                kv=p, B=2, T=4, Hk=4, D=64, ku=1.0, vu=1.0, k=p, ks=256, v=p + 4096, vs=256,
                status=None, stream=None)


def attend(p):
    return dict(q=p, kc=p, vc=p + 16384, pages=3, size=16, stride=16 * 4 * 36, table=p, max_pages=4,
                cu=p, kv=p, B=2, T=4, max_q=2, max_kv=64, H=8, Hk=4, D=64, ku=1.0, vu=1.0,
                scale=0.125, causal=1, out=p + 4096, lse=None, ws=p, ws_bytes=1 << 40, stream=None)


CACHE = [
    (dict(D=96), UNSUPPORTED), (dict(size=8), UNSUPPORTED), (dict(size=48), UNSUPPORTED),
    (dict(size=512), UNSUPPORTED), (dict(pages=0), INVALID), (dict(pages=1 << 31), INVALID),
    (dict(stride=16 * 4 * 36 - 16), INVALID), (dict(stride=16 * 4 * 36 + 8), INVALID),
    (dict(max_pages=-1), INVALID), (dict(Hk=0), INVALID), (dict(Hk=65536), INVALID),
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(cu=None), INVALID),
    (dict(kv=None), INVALID), (dict(table=None), INVALID)] + [
    ({name: u}, INVALID) for name in ("ku", "vu")
    for u in (0.0, -1.0, 3.0, 1.5, 2.0 ** 33, 2.0 ** -33, NAN, INF)]

CALLS = dict(append=(append, "cpattn_paged_append_fp4"), gather=(gather, "cpattn_paged_gather_fp4"),
             attend=(attend, "cpattn_paged_attn_fp4"))


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("change,want", CACHE)
def test_cache(cp, mem, name, change, want):  # noqa: F811
    args, fn = CALLS[name]
    assert call(getattr(cp._lib, fn), args(mem), **change) == want


@pytest.mark.parametrize("name", list(CALLS))
def test_alignment_and_one_cache(cp, mem, name):  # noqa: F811
    args, fn = CALLS[name]
    good = args(mem)
    fn = getattr(cp._lib, fn)
    for arg in ("kc", "vc", "table", "cu", "kv", "k", "v", "q", "out", "status", "lse", "ws"):
        if arg in good:
            assert call(fn, good, **{arg: mem + 2}) == INVALID, arg
    assert call(fn, good, vc=mem) == INVALID
    if name != "attend":
        for change in (dict(k=None), dict(v=None), dict(ks=248), dict(vs=260), dict(T=1 << 30)):
            assert call(fn, good, **change) == INVALID, change
        assert call(fn, good, T=0) == 0 and call(fn, good, B=0) == 0
        assert call(fn, good, T=0, k=None, v=None, kc=None, vc=None) == 0
    if name == "gather":
        assert call(fn, good, v=mem) == INVALID    # one array for both outputs


@pytest.mark.parametrize("change,want", [
    (dict(H=516), UNSUPPORTED), (dict(H=7), INVALID), (dict(H=0), INVALID), (dict(H=65540), INVALID),
    (dict(max_q=0), INVALID), (dict(max_q=-1), INVALID), (dict(max_q=1 << 30), INVALID),
    (dict(max_kv=-1), INVALID), (dict(max_kv=(1 << 30) + 1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=1e38, ku=2.0 ** 30), INVALID),
    (dict(scale=1e-37, ku=2.0 ** -30), INVALID), (dict(causal=2), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=0), SMALL),
    (dict(max_q=100, ws_bytes=1 << 20), SMALL),
    (dict(B=1 << 20, T=1 << 20, max_kv=1 << 30), UNSUPPORTED)])
def test_attend(cp, mem, change, want):  # noqa: F811
    assert call(cp._lib.cpattn_paged_attn_fp4, attend(mem), **change) == want


def test_out_may_not_be_q(cp, mem):  # noqa: F811
    assert call(cp._lib.cpattn_paged_attn_fp4, attend(mem), out=mem) == INVALID


def test_a_workspace_does_for_smaller_batches(cp):  # noqa: F811
    size = cp._lib.cpattn_paged_attn_fp4_workspace_size
    rng = random.Random(1)
    for _ in range(4000):
        Hk = rng.choice([1, 2, 4, 8, 16, 200])
        H, D = Hk * rng.choice([1, 2, 3, 5, 8, 9, 16, 17, 32, 33, 71, 128]), rng.choice([64, 128])
        B = rng.choice([1, 2, 31, 32, 33, 64, 100, 1500])
        most = rng.choice([0, 1, 2, 3, 4, 8, 16, 33, 129, 1000])
        kv = rng.choice([0, 1, 127, 128, 129, 1000, 40000])
        T = rng.choice([0, B, B * most, rng.randint(0, B * most + 1)])
        whole = size(T, B, H, Hk, D, most, kv)
        assert whole > 0
        less = (rng.choice([T, rng.randint(0, T)]), rng.choice([rng.randint(0, B), min(B, 32)]),
                rng.choice([0, most // 2, min(most, 1), most, rng.randint(0, most)]),
                rng.choice([0, kv, rng.randint(0, kv)]))
        assert size(less[0], less[1], H, Hk, D, *less[2:]) <= whole, (T, B, H, Hk, D, most, kv, less)
    for bad in ((-1, 1, 4, 2, 64, 1, 1), (1, 1, 4, 3, 64, 1, 1), (1, 1, 4, 2, 96, 1, 1),
                (1, 1, 258, 2, 64, 1, 1), (1, 1, 4, 2, 64, 1, -1), (1, 1, 4, 2, 64, 1, (1 << 30) + 1),
                (1, 1 << 20, 4, 2, 64, 1, 1 << 30)):
        assert size(*bad) == 0
