"""Selection of blocks by the bound on their scores (sd_block_topk): the
indices equal the fp64 oracle's exactly."""
import numpy as np
import pytest

from oracle import kv_oracle as oracle
from kv_helpers import bf16_normal, f64, table

pytestmark = pytest.mark.gpu


def _cache(lens, P, bs, G, D, seed, bounds=None):
    import torch
    import top_sparse_decode_paged_b200 as sd
    t, N = table(lens, P, seed)
    cache = sd.alloc_kv_cache(N, P, G, D, torch.int8, bs)
    if bounds is None:
        x = bf16_normal((N, P // bs, G, 2, D), seed)
        bounds = torch.stack([torch.minimum(x[..., 0, :], x[..., 1, :]), torch.maximum(x[..., 0, :], x[..., 1, :])], 3)
    cache.k_bounds.copy_(bounds)
    return cache, t


def _check(lens, P, bs, G, H, D, n, n_first, n_last, seed, bounds=None, q=None, max_seqlen=None):
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    cache, t = _cache(lens, P, bs, G, D, seed, bounds)
    q = bf16_normal((len(lens), H, D), seed + 1) if q is None else q
    idx = sd.sd_block_topk(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), n,
                           max(lens) if max_seqlen is None else max_seqlen, n_first, n_last)
    want = oracle.block_topk(f64(q), f64(cache.k_bounds), t, P, bs, lens, n, n_first, n_last)
    assert np.array_equal(idx.cpu().numpy(), want)
    assert sd.device_errors() == 0
    return want


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(32, 8), (3, 3), (5, 1), (14, 2), (128, 1)])
def test_against_the_oracle(D, H, G):
    _check([0, 1, 16, 17, 900, 3333], 32, 16, G, H, D, 12, 1, 2, seed=H + G)


@pytest.mark.parametrize("P,bs,n,n_first,n_last", [(1, 1, 7, 0, 0), (24, 8, 1, 0, 1), (128, 128, 3, 3, 0), (64, 32, 100, 0, 40),
                                                  (48, 12, 2048, 1, 1)])
def test_pages_and_forced_blocks(P, bs, n, n_first, n_last):
    _check([5, 2 * P, 1700], P, bs, 2, 8, 64, n, n_first, n_last, seed=P + n)


def test_a_long_list_of_blocks():
    _check([70_000], 16, 2, 1, 2, 64, 64, 1, 1, seed=3, max_seqlen=131072)


def test_ties_go_to_the_lower_block():
    import torch
    lens = [640]
    b = torch.zeros((12, 4, 1, 2, 64), dtype=torch.bfloat16)  # 10 pages in use and 2 spare
    want = _check(lens, 64, 16, 1, 4, 64, 9, 0, 0, seed=4, bounds=b)
    assert want[0, 0].tolist() == list(range(9))
    want = _check(lens, 64, 16, 1, 4, 64, 9, 1, 2, seed=4, bounds=b)
    assert want[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 38, 39]


def test_sums_that_fp32_cannot_hold():
    """Terms that cancel: the scores' order is that of small rests under large
    terms, which a sum in fp32 loses."""
    import torch
    lens, P, bs = [512], 32, 8
    x = bf16_normal((18, 4, 1, 1, 64), 5) * 2.0 ** -8
    x[..., 0], x[..., 1] = 2.0 ** 14, -(2.0 ** 14)
    b = x.expand(-1, -1, -1, 2, -1).contiguous()
    q = bf16_normal((1, 2, 64), 6)
    q[:, :, 0] = q[:, :, 1] = 1.0
    _check(lens, P, bs, 1, 2, 64, 10, 0, 0, seed=7, bounds=b, q=q)


def test_values_of_every_size():
    import torch
    g = torch.Generator().manual_seed(8)
    e = torch.randint(-125, 60, (18, 4, 1, 1, 64), generator=g).float()
    x = bf16_normal((18, 4, 1, 2, 64), 9).float() * torch.exp2(e)
    b = torch.sort(x.to(torch.bfloat16).float(), dim=3).values.to(torch.bfloat16)
    q = (bf16_normal((1, 2, 64), 10).float() * torch.exp2(torch.randint(-60, 30, (1, 2, 64), generator=g).float())).to(torch.bfloat16)
    _check([512], 32, 8, 1, 2, 64, 10, 0, 0, seed=7, bounds=b, q=q)


def test_bad_page_is_flagged_and_scores_least():
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    cache, t = _cache([320], 32, 16, 1, 64, 11)
    t[0, 4] = -5
    q = bf16_normal((1, 4, 64), 12)
    idx = sd.sd_block_topk(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor([320], dtype=torch.int32).cuda(), 18, 320, 1, 1)
    assert sd.device_errors() == sd.SD_DEVERR_PAGE
    assert idx.cpu().numpy()[0, 0].tolist() == [c for c in range(20) if c not in (8, 9)]


def test_captured_and_replayed():
    import torch
    import top_sparse_decode_paged_b200 as sd
    lens = [900, 40]
    cache, t = _cache(lens, 32, 16, 2, 64, 13)
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = bf16_normal((2, 4, 64), 14).cuda()
    q2 = bf16_normal((2, 4, 64), 15).cuda()
    sd.sd_kv_block_step(q, cache, tt, ln, 8, 900, 0.1)
    lse = torch.empty((2, 4), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, out = sd.sd_kv_block_step(q, cache, tt, ln, 8, 900, 0.1, lse=lse)
    q.copy_(q2)
    g.replay()
    i2, o2 = sd.sd_kv_block_step(q2, cache, tt, ln, 8, 900, 0.1)
    assert torch.equal(idx, i2) and torch.equal(out, o2)


def test_refusals():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache, t = _cache([100], 16, 16, 2, 64, 16)
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor([100], dtype=torch.int32).cuda()
    q = bf16_normal((1, 4, 64), 17).cuda()
    for n, n_first, n_last in ((0, 0, 0), (2, 2, 1), (4, -1, 0), (4096, 1, 1)):
        with pytest.raises(sd.SdError):
            sd.sd_block_topk(q, cache, tt, ln, n, 100, n_first, n_last)
    with pytest.raises(sd.SdError):  # a cache without bounds
        sd.sd_block_topk(q, sd.alloc_kv_cache(4, 16, 2, 64, torch.int8, bounds=False), tt, ln, 4, 100)
    with pytest.raises(sd.SdError):
        sd.sd_kv_block_step(q, cache, tt, ln, 4, 100, float("nan"))


# Calls with room for many blocks score by matrix instructions first and
# exactly only near the border: 4096 blocks a row, 8 rows or more.
MANY = dict(P=16, bs=4, max_seqlen=16384)
MANY_LENS = [16384, 9000, 5, 0, 1, 4097, 12001, 16383]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(8, 8), (10, 2), (24, 1)])
@pytest.mark.parametrize("n,n_first,n_last", [(1, 0, 0), (129, 3, 2), (2048, 0, 1)])
def test_many_blocks(D, H, G, n, n_first, n_last):
    _check(MANY_LENS, G=G, H=H, D=D, n=n, n_first=n_first, n_last=n_last, seed=D + H + n, **MANY)


@pytest.mark.parametrize("value", [0.0, 1.0])
def test_many_ties(value):
    import torch
    lens = [16384, 4100, 900] * 3
    b = torch.full((table(lens, 16, 20)[1], 4, 1, 2, 64), value, dtype=torch.bfloat16)
    want = _check(lens, G=1, H=4, D=64, n=40, n_first=1, n_last=2, seed=20, bounds=b, **MANY)
    assert want[0, 0].tolist() == list(range(38)) + [4094, 4095]


@pytest.mark.parametrize("size", [4, 14, 60])
def test_many_sums_that_cancel(size):
    """The rests under terms of 2^size that cancel decide: some blocks, or
    nearly all, are too close for the first scores."""
    import torch
    lens = [16384, 9001] * 4
    N = table(lens, 16, 21)[1]
    x = bf16_normal((N, 4, 1, 1, 128), 22) * 2.0 ** -3
    x[..., 0], x[..., 1] = 2.0 ** size, -(2.0 ** size)
    b = x.expand(-1, -1, -1, 2, -1).contiguous()
    q = bf16_normal((8, 3, 128), 23)
    q[:, :, 0] = q[:, :, 1] = 1.0
    # A sum may be off by 2^-46 of its terms' magnitudes. At 2^60 that is
    # 2^-46 * 2^61 = 2^15, and the rests (at most 126 products below 2^3, so
    # below 2^10) are lost whatever the order of the sum: the blocks are equal
    # within the bound, and the selection has to be one of 100 distinct blocks.
    if size < 60:
        _check(lens, G=1, H=3, D=128, n=100, n_first=0, n_last=0, seed=21, bounds=b, q=q, **MANY)
        return
    import top_sparse_decode_paged_b200 as sd
    cache, t = _cache(lens, 16, 4, 1, 128, 21, b)
    idx = sd.sd_block_topk(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 100, 16384, 0, 0)
    idx = idx.cpu().numpy()[:, 0]
    assert (np.diff(idx, axis=1) > 0).all() and idx.min() >= 0
    assert all(row[-1] < -(-L // 4) for row, L in zip(idx, lens))
    assert sd.device_errors() == 0


def test_many_queries_of_every_kind():
    """Queries that are zero, subnormal, tiny, huge or not finite."""
    import torch
    lens = [9000, 8001, 7000, 6000, 5000, 16384, 4000, 300]
    q = bf16_normal((8, 4, 64), 24)
    q[0] = 0.0
    q[1, 2] = float("inf")
    q[2, 0, 5] = float("nan")
    q[3] *= 2.0 ** -132
    q[4, 1, 3] = 2.0 ** -130
    q[5] *= 2.0 ** 70
    q[6] *= 2.0 ** -60
    _check(lens, G=1, H=4, D=64, n=33, n_first=0, n_last=1, seed=24, q=q, **MANY)


def test_many_values_of_every_size():
    import torch
    lens = [8192] * 8
    N = table(lens, 16, 25)[1]
    g = torch.Generator().manual_seed(26)
    e = torch.randint(-140, 60, (N, 4, 1, 1, 64), generator=g).float()
    x = bf16_normal((N, 4, 1, 2, 64), 27).float() * torch.exp2(e)
    b = torch.sort(x.to(torch.bfloat16).float(), dim=3).values.to(torch.bfloat16)
    q = (bf16_normal((8, 2, 64), 28).float() * torch.exp2(torch.randint(-60, 30, (8, 2, 64), generator=g).float())).to(torch.bfloat16)
    _check(lens, G=1, H=2, D=64, n=50, n_first=0, n_last=0, seed=25, bounds=b, q=q, **MANY)


@pytest.mark.parametrize("H", [4, 24])
def test_many_blocks_with_a_bad_page(H):
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    lens = [16384] * 8
    cache, t = _cache(lens, 16, 4, 1, 64, 29)
    t[3, 7], t[5, 1000] = 1 << 30, 2 ** 31 - 1
    q = bf16_normal((8, H, 64), 30)
    idx = sd.sd_block_topk(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 2048, 16384, 1, 1).cpu().numpy()
    assert sd.device_errors() == sd.SD_DEVERR_PAGE
    sd.device_errors(clear=True)
    ok = t.copy()
    ok[3, 7], ok[5, 1000] = t[3, 6], t[5, 999]
    bounds = f64(cache.k_bounds)
    for b in range(8):
        bad = {3: range(28, 32), 5: range(4000, 4004)}.get(b, ())
        s = oracle.block_scores(f64(q), bounds, ok, 16, 4, b, 0, H, 4096).astype(np.float64)
        s[list(bad)] = -np.inf
        s[0] = s[4095] = np.inf
        want = np.sort(np.lexsort((np.arange(4096), -s))[:2048])
        assert np.array_equal(idx[b, 0], want)
