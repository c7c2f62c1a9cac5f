"""Attention over an 8-bit blocked cache (sd_kv_attn) against the fp64 oracle."""
import numpy as np
import pytest

from oracle import kv_oracle as oracle
from kv_helpers import assert_attention, bf16_normal, f64, random_cache

pytestmark = pytest.mark.gpu


def _run(kind, lens, P, bs, G, H, D, seed, picked=None, ib=1, expect=0, qscale=1.5, spread=1.0):
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    cache, t, view = random_cache(kind, lens, P, bs, G, D, seed, spread=spread)
    B = len(lens)
    q = bf16_normal((B, H, D), seed + 1, qscale)
    lse = torch.full((B, H), 7.0, device="cuda")
    idx = None if picked is None else torch.from_numpy(picked).cuda()
    out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        D ** -0.5, indices=idx, index_block=ib, lse=lse)
    torch.cuda.synchronize()
    assert sd.device_errors() == expect
    ref = oracle.attend(f64(q), view, t, P, lens, D ** -0.5, picked, ib)
    assert_attention(out, lse, ref, max(lens) if picked is None else picked.shape[2] * ib, (kind, lens, H, G, D))
    return out


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G", [(32, 8), (8, 8), (5, 1), (9, 3), (40, 2), (128, 1), (16, 16), (33, 11)])
def test_every_token(kind, D, H, G):
    _run(kind, [0, 1, 15, 16, 17, 200, 333], 32, 16, G, H, D, seed=H * 7 + G)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("P,bs", [(1, 1), (5, 5), (24, 8), (48, 12), (64, 64), (128, 128), (256, 64), (32, 1)])
def test_pages_and_scale_blocks(kind, P, bs):
    _run(kind, [3, P, 2 * P + 1, 500], P, bs, 2, 8, 128, seed=P + bs)


@pytest.mark.parametrize("lens", [[1], [4097], [1000] * 40, [0, 0, 0], [2500, 0, 0, 1, 0, 31]])
def test_lengths(lens):
    _run("int8", lens, 32, 32, 4, 8, 64, seed=len(lens))


def test_many_requests_span_several_scans():
    rng = np.random.default_rng(5)
    _run("e4m3", [int(x) for x in rng.integers(0, 40, 700)], 16, 8, 1, 2, 64, seed=6)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("ib", [1, 3, 16, 64])
def test_listed_blocks(kind, ib):
    """Rows of a list with holes, duplicates, a block cut by the length, an
    empty row, and entries behind the ones that count (never read as blocks)."""
    rng = np.random.default_rng(ib)
    lens, G, n = [700, 1, 0, 131], 4, 37
    picked = np.full((4, G, n), -1, dtype=np.int32)
    for b, L in enumerate(lens):
        units = -(-L // ib)
        for g in range(G):
            m = int(rng.integers(0, min(n, units) + 1)) if units else 0
            picked[b, g, :m] = rng.integers(0, max(units, 1), m)
            if m > 3:
                picked[b, g, 2] = -1
                picked[b, g, 0] = units - 1
        picked[b, 1] = -1
        picked[b, 0, min(n, units):] = 5
    _run(kind, lens, 32, 16, G, 12, 128, seed=ib, picked=picked, ib=ib)


def test_an_entry_past_the_length_is_flagged_and_skipped():
    import top_sparse_decode_paged_b200 as sd
    picked = np.array([[[0, 9, 3, 2, 1 << 30, -7]]], dtype=np.int32)  # 130 tokens: blocks 0 .. 8 of 16
    _run("int8", [130], 32, 16, 1, 4, 64, seed=1, picked=picked, ib=16, expect=sd.SD_DEVERR_INDEX)


def test_large_and_small_logits_and_scales():
    """Logits far from zero, and blocks whose scales differ by many powers of
    two: the weight of a token with a small V scale must not be lost."""
    _run("int8", [400, 90], 16, 8, 2, 8, 64, seed=3, qscale=40.0)
    _run("e4m3", [400, 90], 16, 8, 2, 8, 64, seed=4, qscale=1e-3, spread=6.0)


def test_dominant_token_with_a_tiny_value_scale():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache, t, view = random_cache("int8", [64], 16, 16, 1, 64, seed=9, spread=0.0)
    q = bf16_normal((1, 1, 64), 10, 1.0)
    # block 0 gets nearly all of the weight and values 2^-40 as large as the others'
    page = int(t[0, 0])
    cache.k_pages[page, :, 0] = (100 * torch.sign(q[0, 0])).to(torch.int8).cuda()
    cache.k_scales[page, 0, 0] = 0.5
    cache.v_scales[page, 0, 0] *= 2.0 ** -40
    view["k"][page, :, 0] = f64(cache.k_pages[page, :, 0])
    view["ks"][page, 0, 0], view["vs"][page, 0, 0] = 0.5, float(cache.v_scales[page, 0, 0])
    lse = torch.empty((1, 1), device="cuda")
    out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor([64], dtype=torch.int32).cuda(), 0.125, lse=lse)
    ref = oracle.attend(f64(q), view, t, 16, [64], 0.125)
    assert_attention(out, lse, ref, 64)


def test_blocks_of_zero_values():
    """A block whose V is zero, with a scale of zero or the store's smallest:
    its tokens keep their softmax weight."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    for kind in ("int8", "e4m3"):
        for scale in (0.0, 2.0 ** -100):
            cache, t, view = random_cache(kind, [64], 16, 16, 1, 64, seed=22, spread=0.0)
            q = bf16_normal((1, 3, 64), 23, 2.0)
            page = int(t[0, 1])
            cache.v_pages.view(torch.uint8)[page] = 0
            cache.v_scales[page] = scale
            view["v"][page], view["vs"][page] = 0, scale
            lse = torch.empty((1, 3), device="cuda")
            out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor([64], dtype=torch.int32).cuda(), 0.5, lse=lse)
            assert_attention(out, lse, oracle.attend(f64(q), view, t, 16, [64], 0.5), 64)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_warp_that_walks_many_tiles(kind):
    """So many KV heads that one CTA takes a whole request of more than 1024
    tiles per warp: integer sums are folded before they can overflow. Values and
    weights are all near their largest."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    G, D, P, L = 1184, 64, 64, 36000
    N = -(-L // P)
    g = torch.Generator(device="cuda").manual_seed(24)
    dt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    make = lambda lo, hi: torch.randint(lo, hi, (N, P, G, D), generator=g, device="cuda", dtype=torch.uint8).view(dt)  # noqa: E731
    k, v = make(0, 40), make(120, 127)  # e4m3: 0x78 .. 0x7e are 256 .. 448
    ks = torch.full((N, 1, G), 1e-3, device="cuda")
    vs = torch.full((N, 1, G), 0.01, device="cuda")
    cache = sd.KvCache(k, v, ks, vs)
    q = bf16_normal((1, G, D), 25).cuda()
    table = torch.randperm(N, generator=g, device="cuda").to(torch.int32)[None].contiguous()
    lse = torch.empty((1, G), device="cuda")
    out = sd.sd_kv_attn(q, cache, table, torch.tensor([L], dtype=torch.int32).cuda(), 0.125, lse=lse)
    for h in (0, 7, 8, 500, G - 1):
        row = table[0].long().repeat_interleave(P)[:L] * P + torch.arange(L, device="cuda") % P
        kk = k.view(N * P, G, D)[row, h].double() * 1e-3
        vv = v.view(N * P, G, D)[row, h].double() * float(vs[0, 0, 0])
        z = 0.125 * (kk @ q[0, h].double())
        ref = torch.softmax(z, 0) @ vv
        # the output's rounding, 2^-8; codes and weights are of one sign, so
        # every other error stays below 2^-10 of the value
        assert ((out[0, h].double() - ref).abs() <= 2.0 ** -8 * (1 + 2.0 ** -2) * ref.abs()).all()
        assert abs(float(lse[0, h]) - float(torch.logsumexp(z, 0))) < 1e-4


def test_two_calls_at_once():
    """Two streams, each with its own workspace."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    lens = [5000] * 8
    cache, t, _ = random_cache("int8", lens, 32, 32, 2, 64, seed=26)
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [bf16_normal((8, 8, 64), 27 + i).cuda() for i in range(2)]
    want = [sd.sd_kv_attn(q, cache, tt, ln, 0.1) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [sd.alloc_kv_attn_workspace(8, 2, 8, 64) for _ in range(2)]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, s, w, o in zip(qs, streams, ws, outs):
            sd.sd_kv_attn(q, cache, tt, ln, 0.1, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_zero_query_and_a_query_that_is_not_finite():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache, t, view = random_cache("e4m3", [100, 100], 32, 32, 2, 64, seed=11)
    q = bf16_normal((2, 4, 64), 12)
    q[0] = 0
    q[1, 1, 5] = float("nan")
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor([100, 100], dtype=torch.int32).cuda()
    out = f64(sd.sd_kv_attn(q.cuda(), cache, tt, ln, 0.125))
    qq = f64(q)
    qq[1, 1] = 0
    o, _, mass, _, _ = oracle.attend(qq, view, t, 32, [100, 100], 0.125)
    assert np.isnan(out[1, 1]).all()
    keep = [(0, 0), (0, 1), (0, 2), (0, 3), (1, 0), (1, 2), (1, 3)]
    for b, h in keep:  # a head that is not finite leaves its neighbours alone
        assert (np.abs(out[b, h] - o[b, h]) <= 2.0 ** -8 * np.abs(o[b, h]) + 2.0 ** -10 * mass[b, h] + 1e-6).all()


def test_bad_page_and_long_length_are_flagged_and_masked():
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    cache, t, view = random_cache("int8", [100], 16, 16, 1, 64, seed=13)
    q = bf16_normal((1, 2, 64), 14)
    bad = t.copy()
    bad[0, 3] = cache.num_pages + 3
    lse = torch.empty((1, 2), device="cuda")
    out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(bad).cuda(), torch.tensor([100], dtype=torch.int32).cuda(), 0.125, lse=lse)
    assert sd.device_errors() == sd.SD_DEVERR_PAGE
    picked = np.array([[[0, 1, 2, 4, 5, 6]]], dtype=np.int32)
    assert_attention(out, lse, oracle.attend(f64(q), view, t, 16, [100], 0.125, picked, 16), 100)
    out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(t).cuda(), torch.tensor([10_000], dtype=torch.int32).cuda(), 0.125, lse=lse)
    assert sd.device_errors() & sd.SD_DEVERR_SEQLEN  # read as the block table's 112 tokens


def test_pool_offsets_past_32_bits():
    import torch
    import top_sparse_decode_paged_b200 as sd
    G, D, P = 8, 128, 64
    N = (1 << 32) // (P * G * D) + 8                       # the last pages start past 2^32 bytes
    k = torch.zeros((N, P, G, D), dtype=torch.int8, device="cuda")
    v = torch.zeros((N, P, G, D), dtype=torch.int8, device="cuda")
    ks = torch.ones((N, 1, G), device="cuda")
    vs = torch.ones((N, 1, G), device="cuda")
    small, t, view = random_cache("int8", [200], P, P, G, D, seed=15, poison=False)
    n = small.num_pages
    for big, part in ((k, small.k_pages), (v, small.v_pages), (ks, small.k_scales), (vs, small.v_scales)):
        big[N - n:] = part
    cache = sd.KvCache(k, v, ks, vs, None, P)
    q = bf16_normal((1, 32, D), 16)
    lse = torch.empty((1, 32), device="cuda")
    out = sd.sd_kv_attn(q.cuda(), cache, torch.from_numpy(t + (N - n)).cuda(), torch.tensor([200], dtype=torch.int32).cuda(), 0.09, lse=lse)
    assert_attention(out, lse, oracle.attend(f64(q), view, t, P, [200], 0.09), 200)


def test_captured_replayed_and_on_another_stream():
    import torch
    import top_sparse_decode_paged_b200 as sd
    lens = [300, 4000, 5]
    cache, t, view = random_cache("e4m3", lens, 32, 16, 2, 128, seed=17)
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    q = bf16_normal((3, 8, 128), 18).cuda()
    plain = sd.sd_kv_attn(q, cache, tt, ln, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sd.sd_kv_attn(q, cache, tt, ln, 0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(plain, other)  # no atomics: the same bits each time
    out, ws = torch.empty_like(plain), sd.alloc_kv_attn_workspace(3, 2, 8, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sd.sd_kv_attn(q, cache, tt, ln, 0.1, out=out, workspace=ws)
        assert sd.last_launch_count() == 2
    q2 = bf16_normal((3, 8, 128), 19).cuda()
    want = sd.sd_kv_attn(q2, cache, tt, ln, 0.1)
    q.copy_(q2)
    ln2 = torch.tensor([299, 17, 0], dtype=torch.int32).cuda()
    g.replay()
    assert torch.equal(out, want)
    want = sd.sd_kv_attn(q2, cache, tt, ln2, 0.1)
    ln.copy_(ln2)
    g.replay()
    assert torch.equal(out, want)


def test_indexer_tokens_over_an_8_bit_cache():
    """The per-head indexer's selection, attended in the 8-bit cache."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    from helpers import to_device
    from top_sparse_decode_paged_b200 import workloads as W
    wl = W.make(W.spec("perhead_b16_gqa", seqlens=(700, 1300), k=256, seed=91))
    d, s = to_device(wl), wl.spec
    idx = sd.sd_indexer_topk(d["qi"], d["w"], d["ki_pages"], d["block_table"], d["seqlens"], s.k, wl.max_seqlen)
    lens = [700, 1300]
    cache, t, view = random_cache("int8", lens, 32, 32, 8, 128, seed=92)
    lse = torch.empty((2, 32), device="cuda")
    out = sd.sd_kv_attn(d["q"], cache, torch.from_numpy(t).cuda(), d["seqlens"], s.scale, indices=idx, lse=lse)
    ref = oracle.attend(f64(d["q"]), view, t, 32, lens, s.scale, idx.cpu().numpy(), 1)
    assert_attention(out, lse, ref, 256)


def test_refusals():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache, t, _ = random_cache("int8", [100], 16, 16, 2, 64, seed=20)
    tt, ln = torch.from_numpy(t).cuda(), torch.tensor([100], dtype=torch.int32).cuda()
    q = bf16_normal((1, 4, 64), 21).cuda()
    with pytest.raises(ValueError):
        sd.sd_kv_attn(q.float(), cache, tt, ln, 0.1)
    with pytest.raises(ValueError):
        sd.sd_kv_attn(q.cpu(), cache, tt, ln, 0.1)
    with pytest.raises(ValueError):
        sd.sd_kv_attn(q, cache, tt.long(), ln, 0.1)
    with pytest.raises(ValueError):
        sd.sd_kv_attn(q, cache, tt, ln, 0.1, indices=torch.zeros((1, 1, 4), dtype=torch.int32, device="cuda"))
    with pytest.raises(sd.SdError):  # heads that the KV heads do not divide
        sd.sd_kv_attn(q[:, :3].contiguous(), cache, tt, ln, 0.1)
    with pytest.raises(sd.SdError):
        sd.sd_kv_attn(q, cache, tt, ln, float("inf"))
    with pytest.raises(sd.SdError):
        sd.sd_kv_attn(q, cache, tt, ln, 0.1, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sd.SdError):  # bf16 pools have their own attention
        sd.sd_kv_attn(q, sd.alloc_kv_cache(4, 16, 2, 64, torch.bfloat16), tt, ln, 0.1)
    with pytest.raises(ValueError):
        sd.KvCache(cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, None, 5)
    with pytest.raises(ValueError):
        sd.KvCache(cache.k_pages, cache.v_pages)
