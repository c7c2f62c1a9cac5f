"""Eviction on the pools of a bf16 KvCache, and the block selection after it:
the compaction moves keys between blocks and knows no bounds, and reading the
kept tokens and storing them again as they are rebuilds the bounds."""
import numpy as np
import pytest

from oracle import kv_oracle as oracle
from kv_helpers import bf16_normal, f64, table

pytestmark = pytest.mark.gpu


def _bounds(pool, t, P, bs, lens):
    """(page, block) -> [G, 2, D] smallest and largest key of every block that holds tokens."""
    out = {}
    for b, L in enumerate(lens):
        for c in range(-(-int(L) // bs)):
            page, slot = int(t[b, c * bs // P]), (c * bs) % P
            rows = pool[page, slot:slot + min(bs, int(L) - c * bs)]
            out[page, slot // bs] = np.stack([rows.min(0), rows.max(0)], 1)
    return out


def test_bounds_after_an_eviction():
    import torch
    import top_sparse_decode_paged_b200 as sd
    P, bs, G, H, D = 32, 16, 2, 8, 64
    lens = [300, 41, 200]
    t, N = table([L + 40 for L in lens], P, 3)
    cache = sd.alloc_kv_cache(N, P, G, D, torch.bfloat16, bs)
    tt = torch.from_numpy(t).cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    qkv = bf16_normal((sum(lens), 2 * G, D), 4).cuda()
    k, v = qkv.split([G, G], 1)
    sd.device_errors(clear=True)
    sd.sd_kv_store(None, k, v, cache, tt, dev(lens), dev([0, 300, 341, 541]), None)
    q_cal = bf16_normal((H, D), 5).cuda()
    new = sd.sd_tri_compact(q_cal, cache.k_pages, cache.v_pages, tt, dev(lens), max(lens), 4, 16, 100)
    kept = new.cpu().numpy()
    assert (kept <= lens).all() and kept[0] < lens[0] and kept[2] < lens[2]
    q = bf16_normal((3, H, D), 6, 2.0).cuda()
    pool = f64(cache.k_pages)
    want_bounds = _bounds(pool, t, P, bs, kept)
    stale = f64(cache.k_bounds)
    assert any(not np.array_equal(stale[p, c], x) for (p, c), x in want_bounds.items())  # what the rebuild is for
    # the kept tokens, read and stored again as they are
    start = torch.zeros(4, dtype=torch.int32, device="cuda")
    torch.cumsum(new, 0, out=start[1:])
    ko, vo = sd.sd_kv_load(cache, tt, new, start, int(kept.sum()))
    sd.sd_kv_store(None, ko, vo, cache, tt, new, start, None)
    torch.cuda.synchronize()
    assert np.array_equal(f64(cache.k_pages), pool)
    got = f64(cache.k_bounds)
    for (p, c), x in want_bounds.items():
        assert np.array_equal(got[p, c], x)
    idx = sd.sd_block_topk(q, cache, tt, new, 4, max(lens), 1, 1).cpu().numpy()
    assert np.array_equal(idx, oracle.block_topk(f64(q), got, t, P, bs, kept, 4, 1, 1))
    # and a decode step on top merges into bounds of what the block holds
    one = bf16_normal((3, 2 * G, D), 7, 3.0).cuda()
    k1, v1 = one.split([G, G], 1)
    sd.sd_kv_store(None, k1, v1, cache, tt, new + 1, dev([0, 1, 2, 3]), None)
    torch.cuda.synchronize()
    pool, got = f64(cache.k_pages), f64(cache.k_bounds)
    for (p, c), x in _bounds(pool, t, P, bs, kept + 1).items():
        assert np.array_equal(got[p, c], x)
    assert sd.device_errors() == 0
