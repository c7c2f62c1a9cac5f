"""The blocked-cache calls without a GPU: workspaces are sized and bad
arguments rejected before any CUDA call."""
import ctypes

import pytest

import top_sparse_decode_paged_b200 as sd
from top_sparse_decode_paged_b200 import api

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from top_sparse_decode_paged_b200 import build
    build.build()
    return sd.load_library()


def _kv(kind=1, bs=16, D=64, k=256, v=256, ks=256, vs=256, kb=256):
    return api.KvDesc(k, v, ks, vs, kb, kind, bs, D)


PD = api.PagedDesc(8, 32, 4, 2)

BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(kind=3), INVALID), (dict(kind=-1), INVALID), (dict(bs=0), INVALID), (dict(bs=12), INVALID), (dict(k=264), INVALID),
    (dict(v=260), INVALID), (dict(kb=264), INVALID), (dict(ks=258), INVALID), (dict(D=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED),
]


def _store(lib, kv=None, pd=PD, q=256, k=256, v=256, qs=256, ks=128, vs=128, ts=256, bt=256, ln=256, B=0, T=4, H=4, qw=256, kw=256,
           eps=1e-6, f=256, rot=64, qo=256):
    return lib.sd_kv_store(q, k, v, qs, ks, vs, ts, None, bt, ln, pd, kv or _kv(), B, T, H, qw, kw, eps, f, rot, 0, qo, None)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_every_call_checks_the_cache(lib, over, status):
    kv = _kv(**over)
    assert _store(lib, kv) == status
    assert lib.sd_kv_load(kv, 256, 256, 256, PD, 1, 4, 256, 256, None) == status
    assert lib.sd_kv_attn(256, kv, 256, 256, None, 0, 1, PD, 1, 4, F(0.1), 256, None, None, 0, None) == status
    assert lib.sd_block_topk(256, kv, 256, 256, PD, 1, 4, 100, 4, 1, 1, 256, None, 0, None) == status
    assert lib.sd_kv_block_step(256, kv, 256, 256, PD, 1, 4, 100, 4, 1, 1, F(0.1), 256, 256, None, None, 0, None) == status
    assert lib.sd_last_launch_count() == 0


def test_geometry(lib):
    for pd, status in ((api.PagedDesc(0, 32, 4, 2), INVALID), (api.PagedDesc(8, 32, 4, 0), INVALID),
                       (api.PagedDesc(1 << 27, 32, 4, 2), UNSUPPORTED), (api.PagedDesc(8, 32, 1 << 25, 2), UNSUPPORTED)):
        assert _store(lib, pd=pd) == status
    assert _store(lib, _kv(bs=256), pd=api.PagedDesc(8, 256, 4, 2)) == UNSUPPORTED  # blocks of at most 128 slots


def test_store_arguments(lib):
    assert _store(lib) == OK and _store(lib, B=1, T=0) == OK  # nothing to do: nothing launched
    for bad in (dict(H=0), dict(qo=None), dict(eps=-1.0), dict(eps=float("nan")), dict(rot=12), dict(rot=72), dict(rot=-8),
                dict(f=None), dict(T=-1), dict(B=-1)):
        assert _store(lib, **bad) == INVALID, bad
    for bad in (dict(k=None), dict(v=None), dict(ts=None), dict(bt=None), dict(ln=None), dict(q=260), dict(k=260), dict(v=260),
                dict(qo=260), dict(qw=260), dict(kw=260), dict(ks=130), dict(vs=126), dict(qs=252), dict(ks=64)):
        assert _store(lib, B=1, **bad) == INVALID, bad
    assert lib.sd_last_launch_count() == 0


def test_load_arguments(lib):
    assert lib.sd_kv_load(_kv(), None, None, None, PD, 1, 0, None, None, None) == OK
    assert lib.sd_kv_load(_kv(), 256, 256, 256, PD, 1, 4, 264, 256, None) == INVALID
    assert lib.sd_kv_load(_kv(), 256, 256, 256, PD, 1, 4, 256, None, None) == INVALID
    assert lib.sd_kv_load(_kv(), None, 256, 256, PD, 1, 4, 256, 256, None) == INVALID


def _attn(lib, kv=None, q=256, idx=None, n=0, ib=1, B=1, H=4, scale=0.1, out=256, ws=None, nws=0, pd=PD):
    return lib.sd_kv_attn(q, kv or _kv(), 256, 256, idx, n, ib, pd, B, H, F(scale), out, None, ws, nws, None)


def test_attention_arguments(lib):
    assert _attn(lib, B=0, ws=256, nws=1 << 30) == OK
    for bad in (dict(q=None), dict(q=264), dict(out=None), dict(out=260), dict(H=3), dict(H=0), dict(B=-1), dict(scale=float("inf")),
                dict(idx=256, n=0), dict(idx=256, n=4, ib=0)):
        assert _attn(lib, **bad) == INVALID, bad
    for bad in (dict(kv=_kv(kind=0)), dict(H=512), dict(idx=256, n=1 << 20, ib=1 << 10), dict(B=1 << 30, H=4)):
        assert _attn(lib, **bad) == UNSUPPORTED, bad
    # 2^36 tokens over all requests, in the table or in listed blocks, are too many; half as many are not
    for walk in (dict(pd=api.PagedDesc(8, 32, 1 << 24, 2)), dict(idx=256, n=1, ib=1 << 29), dict(idx=256, n=1 << 20, ib=512, pd=api.PagedDesc(8, 32, 1 << 24, 2))):
        assert _attn(lib, B=128, **walk) == UNSUPPORTED, walk
        assert _attn(lib, B=64, **walk) == WORKSPACE, walk
    need = lib.sd_kv_attn_workspace_size(1, 2, 4, 64)
    assert need > 0 and need % 256 == 0
    assert _attn(lib) == WORKSPACE
    assert _attn(lib, ws=256, nws=need - 1) == WORKSPACE
    assert _attn(lib, ws=264, nws=need) == WORKSPACE
    assert lib.sd_kv_attn_workspace_size(1, 3, 4, 64) == 0
    assert lib.sd_last_launch_count() == 0


def test_block_selection_arguments(lib):
    f = lambda kv=None, H=4, L=100, n=4, a=1, b=1, idx=256, B=1, ws=None, nws=0, pd=PD: lib.sd_block_topk(  # noqa: E731
        256, kv or _kv(), 256, 256, pd, B, H, L, n, a, b, idx, ws, nws, None)
    need = lib.sd_block_topk_workspace_size(1, 2, 100, 16)
    assert f(B=0, ws=256, nws=need) == OK
    for bad in (dict(kv=_kv(kb=None)), dict(H=5), dict(L=-1), dict(n=0), dict(a=3, b=2), dict(a=-1), dict(b=-1), dict(idx=None),
                dict(a=2147483647, b=2147483647)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(n=2049), dict(H=512), dict(B=40000), dict(L=2147483647, kv=_kv(bs=1))):
        assert f(**bad) == UNSUPPORTED, bad
    assert f() == WORKSPACE and f(ws=256, nws=need - 1) == WORKSPACE
    assert lib.sd_block_topk_workspace_size(1, 2, 100, 0) == 0
    assert lib.sd_kv_block_step_workspace_size(1, 2, 4, 64, 100, 16) == need + lib.sd_kv_attn_workspace_size(1, 2, 4, 64)
    assert lib.sd_last_launch_count() == 0


def test_the_binding_wants_gpu_tensors():
    import torch
    z = torch.zeros((2, 16, 1, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        sd.KvCache(z, z, torch.zeros((2, 1, 1)), torch.zeros((2, 1, 1)))
