"""What the blocked-cache binding hands to the library, without a GPU: CPU
tensors, and the library's functions replaced by ones that look at the call."""
import types

import pytest
import torch

import top_sparse_decode_paged_b200 as sd
from top_sparse_decode_paged_b200 import api

B, G, H, D, P, PAGES = 2, 2, 4, 64, 16, 3


@pytest.fixture
def fake(monkeypatch):
    """A KvCache over CPU tensors whose calls go to ``lib``'s stand-ins."""
    cache = object.__new__(sd.KvCache)
    cache.device, cache._dev = torch.device("cpu"), -1
    cache.num_pages, cache.page_size, cache.G, cache.D, cache.block_tokens = 8, P, G, D, P
    cache.kv_type, cache._kv, cache._descs = api.SD_KV_INT8, api.KvDesc(), {}
    cache._call = lambda stream, fn, *args: fn(*args)
    lib = types.SimpleNamespace(calls=[])
    for name in ("sd_kv_attn", "sd_block_topk", "sd_kv_block_step"):
        setattr(lib, name, lambda *args, name=name: lib.calls.append((name, args)))
        setattr(lib, name + "_workspace_size", lambda *args: 4096)
    monkeypatch.setattr(api, "load_library", lambda: lib)
    return cache, lib


def _inputs():
    q = torch.zeros((B, H, D), dtype=torch.bfloat16)
    return q, torch.zeros((B, PAGES), dtype=torch.int32), torch.full((B,), 20, dtype=torch.int32)


def test_a_list_without_entries_is_refused(fake):
    """Its null address would mean every token."""
    cache, lib = fake
    q, table, lens = _inputs()
    with pytest.raises(ValueError):
        sd.sd_kv_attn(q, cache, table, lens, 0.1, indices=torch.empty((B, G, 0), dtype=torch.int32))
    assert not lib.calls
    sd.sd_kv_attn(q, cache, table, lens, 0.1, indices=torch.zeros((B, G, 1), dtype=torch.int32))
    sd.sd_kv_attn(q, cache, table, lens, 0.1)
    (_, listed), (_, every) = lib.calls
    assert listed[4] and listed[5] == 1 and every[4] is None


@pytest.mark.parametrize("call", ["sd_kv_attn", "sd_block_topk", "sd_kv_block_step"])
def test_the_default_workspace_lives_until_the_call_is_enqueued(fake, call):
    """Freed earlier, its memory could be handed to another thread's tensor
    before this call's kernels are in the stream."""
    import gc
    import weakref
    cache, lib = fake
    made, seen = [], []
    empty = cache._empty

    def recorded(shape, dtype, stream):
        t = empty(shape, dtype, stream)
        if dtype is torch.uint8:
            made.append(weakref.ref(t))
        return t

    def enter(*args):
        gc.collect()
        t = made[0]()
        seen.append(t is not None and (t.data_ptr(), t.nbytes) == (args[-2], args[-1]))

    cache._empty = recorded
    setattr(lib, call, enter)
    q, table, lens = _inputs()
    args = {"sd_kv_attn": (0.1,), "sd_block_topk": (2, 20), "sd_kv_block_step": (2, 20, 0.1)}[call]
    getattr(sd, call)(q, cache, table, lens, *args)
    assert len(made) == 1 and seen == [True]
