"""Block selection over rows whose scores lie awkwardly for a digit histogram:
around a power of two, around zero, with a block that scores -inf. The indices
are those of the exact scores, and such a row costs what any other costs."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

D, G, BS = 128, 8, 8


def _cache(bounds):
    """A cache with these bounds and pools of zeros, which the selection does not read."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    N = bounds.shape[0]
    pool = torch.zeros((N, BS, G, D), dtype=torch.int8, device="cuda")
    scales = torch.ones((N, 1, G), device="cuda")
    return sd.KvCache(pool, pool, scales, scales, bounds.cuda(), BS)


def _case(scores, bad, seed):
    """Queries of one at dims 0 and 1 whose blocks score ``scores`` [B, G, C]
    (to 2^-16: bf16 in dim 0, the rest in dim 1), the cache, and a table of C
    shuffled pages; ``bad`` pages of each request are not in the pool."""
    import torch
    B, _, C = scores.shape
    rng = np.random.default_rng(seed)
    top = torch.from_numpy(scores).to(torch.bfloat16)
    rest = (torch.from_numpy(scores) - top.double()).to(torch.bfloat16)
    table = np.stack([rng.permutation(C) + b * C for b in range(B)]).astype(np.int32)
    bounds = torch.zeros((B * C, 1, G, 2, D), dtype=torch.bfloat16)
    rows = torch.from_numpy(table.reshape(-1).astype(np.int64))
    for d, x in ((0, top), (1, rest)):
        y = x.permute(0, 2, 1).reshape(B * C, G)  # [pages in table order, G]
        bounds[rows, 0, :, 0, d] = y
        bounds[rows, 0, :, 1, d] = y
    bounds[..., 2:] = 0.01 * torch.randn((B * C, 1, G, 1, 1), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    q = torch.zeros((B, 4 * G, D), dtype=torch.bfloat16)
    q[..., :2] = 1
    exact = (top.double() + rest.double()).float().numpy()
    for b in range(B):
        at = rng.choice(np.arange(8, C - 8), bad, replace=False)
        table[b, at] = -1
        exact[b, :, at] = -np.inf
    return q.cuda(), _cache(bounds), torch.from_numpy(table).cuda(), exact


def _want(exact, n, first, last):
    B, _, C = exact.shape
    out = np.empty((B, G, n), dtype=np.int32)
    c = np.arange(C)
    forced = (c < first) | (c >= C - last)
    for b in range(B):
        for g in range(G):
            out[b, g] = np.sort(np.lexsort((c, -exact[b, g].astype(np.float64), ~forced))[:n])
    return out


def _time(call):
    import torch
    g = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(20):
            call()
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 20 * 1e3)
    return best


@pytest.mark.parametrize("B,C,n", [(16, 1024, 128), (4, 4096, 64), (16, 1024, 1000)])
def test_rows_that_straddle(B, C, n):
    import torch
    import top_sparse_decode_paged_b200 as sd
    rng = np.random.default_rng(C + n)
    x = rng.standard_normal((B, G, C))
    rows = {"plain": (20 + 3 * x, 0), "around 2": (2 + 0.2 * x, 0), "around 0": (x, 0), "a bad page": (20 + 3 * x, 1),
            "around 16, skewed": (15.9 + 0.2 * np.abs(x), 0)}
    took = {}
    for name, (scores, bad) in rows.items():
        q, cache, table, exact = _case(scores, bad, seed=C)
        lens = torch.full((B,), C * BS - 5, dtype=torch.int32, device="cuda")
        ws = sd.alloc_block_topk_workspace(B, G, C * BS, BS)
        out = torch.empty((B, G, n), dtype=torch.int32, device="cuda")
        sd.device_errors(clear=True)
        sd.sd_block_topk(q, cache, table, lens, n, C * BS, 1, 2, indices=out, workspace=ws)
        torch.cuda.synchronize()
        assert sd.device_errors(clear=True) == (sd.SD_DEVERR_PAGE if bad else 0)
        assert np.array_equal(out.cpu().numpy(), _want(exact, n, 1, 2)), name
        took[name] = _time(lambda: sd.sd_block_topk(q, cache, table, lens, n, C * BS, 1, 2, indices=out, workspace=ws))
        sd.device_errors(clear=True)
    print({k: round(v, 1) for k, v in took.items()})
    assert max(took.values()) < 1.6 * took["plain"], took


@pytest.mark.parametrize("seed", [1, 2])
def test_scores_that_cancel(seed):
    """Full-length products of which the second half takes the first away: the
    terms' sum, which the approximate scores' error is bounded by, is
    hundreds of times the scores' differences, and eight blocks or so of a row lie
    within the bound of the border."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    B, C, n = 16, 1024, 128
    g = torch.Generator().manual_seed(seed)
    q = (1 + torch.rand((B, 4 * G, D), generator=g)).to(torch.bfloat16)
    k = 1 + torch.rand((B * C, G, D), generator=g)
    k[..., D // 2:] *= -1
    k = k.to(torch.bfloat16)
    table = torch.randperm(B * C, generator=g).to(torch.int32).view(B, C)
    score = torch.einsum("bghd,bcgd->bghc", q.view(B, G, 4, D).double(), k[table.long()].double()).amax(2)
    cache = _cache(k[:, None, :, None].expand(B * C, 1, G, 2, D).contiguous())
    lens = torch.full((B,), C * BS, dtype=torch.int32, device="cuda")
    out = sd.sd_block_topk(q.cuda(), cache, table.cuda(), lens, n, C * BS, 1, 2)
    assert np.array_equal(out.cpu().numpy(), _want(score.float().numpy(), n, 1, 2))
