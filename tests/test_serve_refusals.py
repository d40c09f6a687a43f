"""Refusals of the norm + rotation and paged-cache calls.  All are found on the
host before anything is enqueued, so no GPU is needed: host memory stands in for
device pointers that are never read."""

import ctypes

import pytest
import torch

from long_context_gb300 import build as lib_build

INVALID, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def cp():
    lib_build.build()
    from long_context_gb300 import cpattn
    return cpattn


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    mem.keep = buf
    return base


def call(fn, good, **change):
    args = dict(good)
    assert set(change) <= set(args), change
    args.update(change)
    return fn(*args.values())


def norm_rope(p):
    return dict(q=p, qs=512, k=p, ks=256, pos=p, table=p, rot=64, max_pos=10, wq=p, wk=p, eps=1e-6,
                inter=0, T=4, H=8, Hk=4, D=64, qo=p, qos=512, ko=p, kos=256, status=None,
                stream=None)


def norm_rope_bwd(p):
    return dict(gq=p, gqs=512, gk=p, gks=256, q=p, qs=512, k=p, ks=256, pos=p, table=p, rot=64,
                max_pos=10, wq=p, wk=p, eps=1e-6, inter=0, T=4, H=8, Hk=4, D=64, dq=p, dqs=512,
                dk=p, dks=256, dwq=p, dwk=p, ws=p, ws_bytes=1 << 20, status=None, stream=None)


COMMON = [
    (dict(D=96), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=24), INVALID),
    (dict(rot=80), INVALID), (dict(max_pos=0), INVALID), (dict(wq=None), INVALID),
    (dict(wk=None), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(inter=2), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(T=(1 << 31) // 12 + 1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(qs=504), INVALID), (dict(ks=257), INVALID), (dict(qs=513), INVALID),
    (dict(pos=None), INVALID), (dict(table=None, wq=None, wk=None), INVALID),
]


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(kos=100), INVALID),
    (dict(qos=516), INVALID)])
def test_norm_rope(cp, mem, change, want):
    assert call(cp._lib.cpattn_qk_norm_rope, norm_rope(mem), **change) == want


@pytest.mark.parametrize("name", ["q", "k", "wq", "wk", "table", "qo", "ko", "pos", "status"])
def test_norm_rope_alignment(cp, mem, name):
    assert call(cp._lib.cpattn_qk_norm_rope, norm_rope(mem), **{name: mem + 2}) == INVALID


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(q=None), INVALID), (dict(gq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dqs=511), INVALID), (dict(gks=4), INVALID), (dict(dwq=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=1000), SMALL)])
def test_norm_rope_bwd(cp, mem, change, want):
    assert call(cp._lib.cpattn_qk_norm_rope_bwd, norm_rope_bwd(mem), **change) == want
    assert cp._lib.cpattn_qk_norm_rope_bwd_workspace_size(96) == 0


def append(p):
    return dict(k=p, ks=256, v=p, vs=256, kc=p, vc=p + 4096, pages=8, size=16, stride=16 * 256,
                table=p, max_pages=4, cu=p, kv=p, B=2, T=4, Hk=4, D=64, rope=p, rot=64, max_pos=64,
                inter=0, wq=p, wk=p, eps=1e-6, q=p, qs=512, H=8, qo=p, qos=512, status=None,
                stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(D=80), UNSUPPORTED), (dict(size=8), UNSUPPORTED), (dict(size=48), UNSUPPORTED),
    (dict(size=512), UNSUPPORTED), (dict(pages=0), INVALID), (dict(pages=1 << 31), INVALID),
    (dict(stride=16 * 256 - 8), INVALID), (dict(stride=16 * 256 + 4), INVALID),
    (dict(max_pages=-1), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID),
    (dict(Hk=0), INVALID), (dict(H=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(kc=None), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID),
    (dict(kv=None), INVALID), (dict(qo=None), INVALID), (dict(ks=248), INVALID),
    (dict(vs=260), INVALID), (dict(rot=40), INVALID), (dict(wq=None), INVALID),
    (dict(q=None), INVALID), (dict(q=None, H=0, qo=None), INVALID), (dict(T=1 << 28), INVALID)])
def test_append(cp, mem, change, want):
    assert call(cp._lib.cpattn_paged_append, append(mem), **change) == want


def test_append_of_one_cache(cp, mem):
    assert call(cp._lib.cpattn_paged_append, append(mem), vc=mem) == INVALID
    assert call(cp._lib.cpattn_paged_append, append(mem), T=0) == 0
    assert call(cp._lib.cpattn_paged_append, append(mem), B=0) == 0


def attend(p):
    return dict(q=p, kc=p, vc=p, pages=8, size=16, stride=16 * 256, table=p, max_pages=4, cu=p,
                kv=p, B=2, T=4, max_q=2, max_kv=64, H=8, Hk=4, D=64, scale=0.125, causal=1,
                out=p + 4096, lse=None, ws=p, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(D=96), UNSUPPORTED), (dict(size=24), UNSUPPORTED), (dict(size=1), UNSUPPORTED),
    (dict(H=516), UNSUPPORTED),                                  # 129 query heads a KV head
    (dict(H=7), INVALID), (dict(Hk=0), INVALID), (dict(H=0), INVALID), (dict(H=65540), INVALID),
    (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(B=-1), INVALID),
    (dict(max_q=0), INVALID), (dict(max_q=-1), INVALID), (dict(max_q=1 << 30), INVALID),
    (dict(max_kv=-1), INVALID), (dict(max_kv=(1 << 30) + 1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(causal=2), INVALID), (dict(pages=0), INVALID),
    (dict(stride=0), INVALID), (dict(max_pages=-1), INVALID), (dict(q=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(out=None), INVALID),
    (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=4096), SMALL)])
def test_attend(cp, mem, change, want):
    assert call(cp._lib.cpattn_paged_attn, attend(mem), **change) == want


@pytest.mark.parametrize("name", ["q", "kc", "vc", "out", "table", "cu", "kv", "lse", "ws"])
def test_attend_alignment(cp, mem, name):
    assert call(cp._lib.cpattn_paged_attn, attend(mem), **{name: mem + 2}) == INVALID


def test_attend_in_place_and_sizes(cp, mem):
    assert call(cp._lib.cpattn_paged_attn, attend(mem), out=mem) == INVALID
    size = cp._lib.cpattn_paged_attn_workspace_size
    assert size(4, 2, 8, 4, 64, 2) > 0
    for bad in ((-1, 2, 8, 4, 64, 2), (4, 2, 8, 3, 64, 2), (4, 2, 8, 4, 96, 2),
                (4, 2, 516, 4, 64, 2), (4, 2, 8, 4, 64, -1)):
        assert size(*bad) == 0
    with pytest.raises(cp.CpattnError):
        cp.paged_workspace_size(4, 2, 8, 3, 64, 2)


def test_binding_refuses_host_tensors(cp):
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    pos, tab = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 64)
    i32 = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cp.qk_norm_rope(q, k, pos, tab)
    with pytest.raises(ValueError):
        cp.qk_norm_rope_bwd(q, k, q, k, pos, tab)
    with pytest.raises(ValueError):
        cp.paged_append(k, k, cache, cache.clone(), i32[None], i32[:2], i32[:1])
    with pytest.raises(ValueError):
        cp.paged_attn(q, cache, cache, i32[None], i32[:2], i32[:1], max_seqlen=4, max_kv_len=4)
    with pytest.raises(TypeError):
        cp.qk_norm_rope(q.float(), k, pos, tab)
