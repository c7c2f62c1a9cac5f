"""Norm + rotation + store into a blocked cache (sd_kv_store) and the
read-back (sd_kv_load), against the fp64 oracle, and runs of the blocked-cache
calls together as a serving loop makes them."""
import numpy as np
import pytest

from oracle import kv_oracle as oracle
from kv_helpers import DTYPE, QMAX, assert_attention, bf16_normal, codes_as_f64, f64, table

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _freqs(R, base=10000.0):
    import torch
    return None if R == 0 else (base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float()


def _close(got, ref, scale=None):
    """bf16 values: half a step of the value, 2^-8, and the fp32 arithmetic
    before it: under 2^-20 of the row's largest entry (norm: a sum of 128
    squares and a reciprocal root; rotation: two products of cosines off by
    2^-22)."""
    ref = np.asarray(ref)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(ref).max(-1, keepdims=True) + 1e-30
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()


class Loop:
    """A cache with its fp64 expectation: stores go through the library and the
    checks after each one follow from the codes that were there before."""

    def __init__(self, kind, lens, P, bs, G, D, H, seed, capacity=0):
        import torch
        import top_sparse_decode_paged_b200 as sd
        self.sd, self.kind, self.P, self.bs, self.G, self.D, self.H = sd, kind, P, bs, G, D, H
        self.t, N = table([max(L, capacity) for L in lens], P, seed)
        self.cache = sd.alloc_kv_cache(N, P, G, D, DTYPE[kind], bs)
        # what was in the cache before must not matter, nor change where nothing is stored
        g = torch.Generator().manual_seed(seed)
        for x in (self.cache.k_pages, self.cache.v_pages):
            if kind == "bf16":
                x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
            else:
                x.view(torch.uint8).copy_(torch.randint(0, 120, x.shape, generator=g, dtype=torch.uint8))
        self.cache.k_bounds.copy_(torch.randn(self.cache.k_bounds.shape, generator=g).to(torch.bfloat16))
        if kind != "bf16":
            self.cache.k_scales.fill_(3.0)
            self.cache.v_scales.fill_(5.0)
        self.tt = torch.from_numpy(self.t).cuda()

    def snapshot(self):
        c = self.cache
        s = dict(k=codes_as_f64(c.k_pages), v=codes_as_f64(c.v_pages), b=f64(c.k_bounds))
        for n, x in (("ks", c.k_scales), ("vs", c.v_scales)):
            s[n] = np.ones((c.num_pages, self.P // self.bs, self.G)) if x is None else x.cpu().numpy().astype(np.float64)
        return s

    def store(self, tok_start, seqlens, seed, R=None, interleaved=False, norm=True, positions=None, pad=0, big=None):
        import torch
        sd, G, H, D = self.sd, self.G, self.H, self.D
        R = D if R is None else R
        T = int(tok_start[-1])
        qkv = bf16_normal((T + pad, (H + 2 * G) * D), seed, 1.5)
        if big is not None:
            big(qkv.view(T + pad, H + 2 * G, D))
        qw, kw = (bf16_normal((D,), seed + 1) + 1, bf16_normal((D,), seed + 2) + 1) if norm else (None, None)
        f = _freqs(R)
        before = self.snapshot()
        dev = lambda x: None if x is None else x.cuda()  # noqa: E731
        q, k, v = qkv.cuda().view(T + pad, H + 2 * G, D).split([H, G, G], 1)
        q_out = torch.full((T + pad, H, D), 77.0, dtype=torch.bfloat16, device="cuda")
        self.ts = torch.tensor(tok_start, dtype=torch.int32).cuda()
        self.ln = torch.tensor(seqlens, dtype=torch.int32).cuda()
        sd.device_errors(clear=True)
        sd.sd_kv_store(q, k, v, self.cache, self.tt, self.ln, self.ts, dev(f), q_weight=dev(qw), k_weight=dev(kw), eps=EPS,
                       interleaved=interleaved, positions=None if positions is None else torch.tensor(positions, dtype=torch.int32).cuda(),
                       q_out=q_out)
        torch.cuda.synchronize()
        assert sd.device_errors() == 0
        self.check(before, f64(qkv.view(T + pad, H + 2 * G, D)), qw, kw, f, interleaved, positions, tok_start, seqlens, f64(q_out))
        return q_out[:T]

    def check(self, before, x, qw, kw, f, interleaved, positions, tok_start, seqlens, q_out):
        P, bs, G, H, kind = self.P, self.bs, self.G, self.H, self.kind
        after = self.snapshot()
        w = lambda t: None if t is None else f64(t)  # noqa: E731
        ff = None if f is None else f.double().numpy()
        T = int(tok_start[-1])
        assert (q_out[T:] == 77.0).all()
        touched = {}
        for b, row, pos in oracle.new_tokens(tok_start, seqlens):
            ang = pos if positions is None else positions[row]
            _close(q_out[row], oracle.norm_rotate(x[row, :H], w(qw), EPS, ff, interleaved, ang))
            y = oracle.norm_rotate(x[row, H:H + G], w(kw), EPS, ff, interleaved, ang)
            page, slot = oracle.token_slot(self.t, P, b, pos)
            touched.setdefault((page, slot // bs), []).append((slot, y, x[row, H + G:]))
            if not hasattr(self, "held"):
                self.held = {}
        for (page, blk), rows in touched.items():
            first = min(s for s, _, _ in rows)
            earlier = range(blk * bs, first)                     # rows the block held before
            new = [s for s, _, _ in rows]
            rest = [s for s in range(blk * bs, blk * bs + bs) if s >= first and s not in new]
            for n, at in (("k", 1), ("v", 2)):
                y = np.stack([r[at] for r in rows])              # [rows, G, D]
                got, old = after[n][page, new], before[n][page]
                if kind == "bf16":
                    _close(got, y)
                    assert np.array_equal(after[n][page, list(earlier)], old[list(earlier)])
                    continue
                s_old, s = before[n + "s"][page, blk], after[n + "s"][page, blk]
                want = np.maximum(np.abs(y).max((0, 2)) / QMAX[kind], 2.0 ** -100)
                if len(earlier):
                    want = np.maximum(want, s_old)
                assert (np.abs(s - want) <= 2.0 ** -19 * want).all()  # the fp32 norm and rotation, one division
                # half a step: int8 of the scale; e4m3 of the value (2^-4), or of its smallest step 2^-9
                step = 0.5 * s[None, :, None] if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[None, :, None])
                off = np.abs(got * s[None, :, None] - y)
                assert (off <= step + 2.0 ** -17 * np.abs(y).max(-1, keepdims=True)).all(), (off / step).max()
                for e in earlier:                                # coded anew where the scale grew, else as they were
                    value = old[e] * s_old[:, None]
                    grew = s > s_old
                    assert np.array_equal(after[n][page, e][~grew], old[e][~grew])
                    step = 0.5 * s[:, None] if kind == "int8" else np.maximum(2.0 ** -4 * np.abs(value), 2.0 ** -10 * s[:, None])
                    assert (np.abs(after[n][page, e] * s[:, None] - value) <= step * (1 + 2.0 ** -16)).all()
            for n in ("k", "v"):
                assert np.array_equal(after[n][page, rest], before[n][page, rest])
            yb = np.stack([r[1] for r in rows])
            lo, hi = yb.min(0), yb.max(0)
            if len(earlier):
                lo, hi = np.minimum(lo, before["b"][page, blk, :, 0]), np.maximum(hi, before["b"][page, blk, :, 1])
            big = np.abs(yb).max()
            for got, ref in ((after["b"][page, blk, :, 0], lo), (after["b"][page, blk, :, 1], hi)):
                assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * big).all()
        other = np.ones((self.cache.num_pages, P // bs), dtype=bool)
        for key in touched:
            other[key] = False
        for n in ("ks", "vs", "b"):
            assert np.array_equal(after[n][other], before[n][other], equal_nan=True)
        for n in ("k", "v"):
            rows = np.repeat(other, bs, 1)
            assert np.array_equal(after[n][rows], before[n][rows], equal_nan=True)
        self.after = after

    def check_load(self, tok_start):
        import torch
        T = int(tok_start[-1])
        out = [torch.full((T + 3, self.G, self.D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.sd.sd_kv_load(self.cache, self.tt, self.ln, self.ts, T + 3, k_out=out[0], v_out=out[1])
        for got, n in zip(out, ("k", "v")):
            got = f64(got)
            assert (got[T:] == 9.0).all()
            for b, row, pos in oracle.new_tokens(tok_start, self.ln.tolist()):
                page, slot = oracle.token_slot(self.t, self.P, b, pos)
                ref = self.after[n][page, slot] * self.after[n + "s"][page, slot // self.bs][:, None]
                assert (np.abs(got[row] - ref) <= 2.0 ** -8 * np.abs(ref)).all()


KINDS = ["bf16", "int8", "e4m3"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R,interleaved,norm", [(None, False, True), (None, True, False), (32, False, False), (48, False, True),
                                                (40, True, True), (0, False, True), (56, False, True)])
def test_prompts_then_decode_steps(kind, D, R, interleaved, norm):
    """Ragged prompts (one empty), a chunk, then single tokens: blocks fill up
    step by step and their scales grow."""
    lens = [37, 0, 1, 70, 16]
    c = Loop(kind, lens, 32, 16, 2, D, 6, seed=D + (R or 0), capacity=120)
    starts = np.concatenate([[0], np.cumsum(lens)])
    c.store(starts, lens, 1, R, interleaved, norm, pad=2)
    c.check_load(starts)
    new = [20, 3, 0, 9, 1]
    lens = [a + b for a, b in zip(lens, new)]
    starts = np.concatenate([[0], np.cumsum(new)])
    c.store(starts, lens, 2, R, interleaved, norm)
    for step in range(3):
        lens = [L + 1 for L in lens]
        grow = lambda x: x[:, 6:].mul_(1.0 + step)  # noqa: E731  (in place: later tokens are larger)
        c.store(np.arange(6), lens, 3 + step, R, interleaved, norm, pad=1, big=grow)
        c.check_load(np.arange(6))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("P,bs", [(1, 1), (6, 3), (48, 12), (128, 128), (256, 64), (20, 20)])
def test_pages_and_blocks(kind, P, bs):
    lens = [3, P + 1, 150]
    c = Loop(kind, lens, P, bs, 3, 128, 3, seed=P, capacity=400)
    c.store(np.concatenate([[0], np.cumsum(lens)]), lens, 5)
    new = [1, 130, 131]
    lens = [a + b for a, b in zip(lens, new)]
    c.store(np.concatenate([[0], np.cumsum(new)]), lens, 6)


@pytest.mark.parametrize("B", [1, 33, 300])
def test_decode_batches(B):
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(1, 60, B)]
    c = Loop("int8", lens, 16, 8, 1, 64, 2, seed=B)
    c.store(np.arange(B + 1), lens, 7, pad=5)


def test_many_prompts_are_found_in_several_scans():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 60, 600)]
    c = Loop("e4m3", lens, 16, 4, 1, 64, 1, seed=4)
    c.store(np.concatenate([[0], np.cumsum(lens)]), lens, 8, R=16)


def test_far_positions_keep_their_angles():
    lens = [40]
    c = Loop("bf16", lens, 16, 16, 1, 128, 2, seed=5)
    c.store([0, 40], lens, 9, positions=[i * 26214 + 1048576 for i in range(40)])
    c.store([0, 40], lens, 9, positions=[2 ** 31 - 1 - i for i in range(40)], R=8)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_zeros_tiny_huge_and_entries_that_are_not_finite(kind):
    import torch
    import top_sparse_decode_paged_b200 as sd
    c = Loop(kind, [16, 16, 16], 16, 8, 1, 64, 1, seed=6)

    def fill(x):
        x[0:8, 1:] = 0.0          # a block of zeros
        x[8:16, 1:] *= 1e-30      # below any useful scale
        x[16:24, 1:] *= 1e30
    c.store([0, 16, 32, 48], [16, 16, 16], 10, R=0, norm=False, big=fill)
    x = bf16_normal((16, 3, 64), 11)
    x[3, 1, 5], x[4, 1, 6], x[5, 2, 7], x[6, 2, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    q, k, v = x.cuda().split([1, 1, 1], 1)
    ts, ln = torch.tensor([0, 16, 16, 16], dtype=torch.int32).cuda(), torch.tensor([16, 0, 0], dtype=torch.int32).cuda()
    sd.sd_kv_store(q, k, v, c.cache, c.tt, ln, ts, None)
    a = c.snapshot()
    page = int(c.t[0, 0])
    clean = f64(x)
    clean[~np.isfinite(clean)] = 0
    for n, h in (("k", 1), ("v", 2)):
        s = a[n + "s"][page, :, 0]
        want = np.abs(clean[:, h]).reshape(2, 8, 64).max((1, 2)) / QMAX[kind]
        assert (np.abs(s - want) <= 2.0 ** -22 * want).all()
    top = QMAX[kind]
    assert a["k"][page, 3, 0, 5] == 0 and a["k"][page, 4, 0, 6] == top
    assert a["v"][page, 5, 0, 7] == -top and a["v"][page, 6, 0, 0] == 0


def test_store_without_queries_in_place_and_captured():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache = sd.alloc_kv_cache(8, 16, 2, 64, torch.int8, 16)
    other = sd.alloc_kv_cache(8, 16, 2, 64, torch.int8, 16)
    bt = torch.arange(8, dtype=torch.int32).cuda().view(2, 4)
    ln, ts = torch.tensor([20, 33], dtype=torch.int32).cuda(), torch.tensor([0, 20, 53], dtype=torch.int32).cuda()
    q, k, v = (bf16_normal((53, h, 64), 30 + h).cuda() for h in (4, 2, 2))
    f = _freqs(64).cuda()
    want = sd.sd_kv_store(q, k, v, cache, bt, ln, ts, f)
    assert sd.sd_kv_store(None, k, v, other, bt, ln, ts, f) is None
    for x, y in ((cache.k_pages, other.k_pages), (cache.v_scales, other.v_scales), (cache.k_bounds, other.k_bounds)):
        assert torch.equal(x, y)
    mine = q.clone()
    assert sd.sd_kv_store(mine, k, v, cache, bt, ln, ts, f, q_out=mine) is mine
    assert torch.equal(mine, want)
    g = torch.cuda.CUDAGraph()
    q_out = torch.empty_like(q)
    with torch.cuda.graph(g):
        sd.sd_kv_store(q, k, v, cache, bt, ln, ts, f, q_out=q_out)
        kd, vd = sd.sd_kv_load(cache, bt, ln, ts, 53)
    q.copy_(q.flip(0))
    k.copy_(k.flip(0))
    g.replay()
    assert torch.equal(q_out, sd.sd_kv_store(q, k, v, other, bt, ln, ts, f))
    assert torch.equal(kd, sd.sd_kv_load(other, bt, ln, ts, 53)[0])


def test_bad_page_and_more_rows_than_the_request_holds():
    import torch
    import top_sparse_decode_paged_b200 as sd
    sd.device_errors(clear=True)
    cache = sd.alloc_kv_cache(4, 16, 1, 64, torch.int8, 8)
    bt = torch.tensor([[0, 99], [1, 2]], dtype=torch.int32).cuda()
    ln, ts = torch.tensor([20, 5], dtype=torch.int32).cuda(), torch.tensor([0, 20, 30], dtype=torch.int32).cuda()
    k, v = bf16_normal((30, 1, 64), 1).cuda(), bf16_normal((30, 1, 64), 2).cuda()
    sd.sd_kv_store(None, k, v, cache, bt, ln, ts, None)
    assert sd.device_errors() == sd.SD_DEVERR_PAGE | sd.SD_DEVERR_INDEX
    assert (cache.k_pages[2:] == 0).all() and (cache.k_pages[0] != 0).any(-1).all()
    # request 1 holds 5 tokens: the last 5 of its 10 rows
    got = f64(sd.sd_kv_load(cache, bt, torch.tensor([0, 5], dtype=torch.int32).cuda(), torch.tensor([0, 0, 5], dtype=torch.int32).cuda(), 5)[1])
    ref = f64(v[25:30])
    assert (np.abs(got - ref) <= np.abs(ref).max() / 250 + 2.0 ** -8 * np.abs(ref)).all()
    out = sd.sd_kv_load(cache, bt, ln, ts, 30)
    assert sd.device_errors() == sd.SD_DEVERR_PAGE | sd.SD_DEVERR_INDEX
    assert (out[0][16:25] == 0).all()


def test_single_tokens_among_chunks():
    """Mixed batches: requests with one new token among some with a few, and
    one long prompt among single tokens."""
    for new in ([1, 1, 5, 1, 0, 2, 1, 1], [1, 1, 1, 90, 1, 1, 1], [3] * 20):
        old = [7 * i % 23 for i in range(len(new))]
        lens = [a + b for a, b in zip(old, new)]
        c = Loop("int8", lens, 32, 16, 3, 128, 2, seed=len(new))
        c.store(np.concatenate([[0], np.cumsum(old)]), old, 80)
        c.store(np.concatenate([[0], np.cumsum(new)]), lens, 81, pad=3)


def test_starts_out_of_order_touch_nothing_outside():
    """tok_start that is not ascending is the caller's error: flagged or
    ignored, and no row of another request's blocks changes hands outside the pools."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache = sd.alloc_kv_cache(6, 16, 1, 64, torch.int8, 16)
    bt = torch.arange(6, dtype=torch.int32).cuda().view(3, 2)
    ln = torch.tensor([20, 3, 32], dtype=torch.int32).cuda()
    k = bf16_normal((40, 1, 64), 1).cuda()
    for ts in ([0, 30, 10, 40], [0, -5, 20, 40], [5, 5, 5, 5], [40, 20, 10, 0], [0, 1000000, 3, 40]):
        t = torch.tensor(ts, dtype=torch.int32).cuda()
        sd.sd_kv_store(None, k, k, cache, bt, ln, t, None)
        sd.sd_kv_load(cache, bt, ln, t, 40)
    sd.device_errors(clear=True)
    t = torch.tensor([0, 20, 23, 40], dtype=torch.int32).cuda()
    sd.sd_kv_store(None, k, k, cache, bt, ln, t, None)
    got = f64(sd.sd_kv_load(cache, bt, ln, t, 40)[0])
    assert sd.device_errors() == 0
    ref = f64(k)
    # codes may have been coded anew under a scale of the calls above: one more half step
    assert (np.abs(got - ref) <= 2 * np.abs(ref).max() / 254 + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_a_serving_loop(kind):
    """Prompts, then decode steps with selected blocks, as a server runs them:
    every step's attention matches the oracle on the cache it left."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    lens = [200, 31, 90]
    P, bs, G, D, H = 32, 16, 2, 64, 8
    c = Loop(kind, lens, P, bs, G, D, H, seed=50, capacity=260)
    c.store(np.concatenate([[0], np.cumsum(lens)]), lens, 51)
    for step in range(4):
        lens = [L + 1 for L in lens]
        q = c.store(np.arange(4), lens, 60 + step)
        lse = torch.empty((3, H), device="cuda")
        idx, out = sd.sd_kv_block_step(q, c.cache, c.tt, c.ln, 6, 256, D ** -0.5, n_first=1, n_last=2, lse=lse)
        want = oracle.block_topk(f64(q), c.after["b"], c.t, P, bs, lens, 6, 1, 2)
        assert np.array_equal(idx.cpu().numpy(), want)
        view = dict(k=c.after["k"], v=c.after["v"], ks=c.after["ks"], vs=c.after["vs"], bs=bs)
        assert_attention(out, lse, oracle.attend(f64(q), view, c.t, P, lens, D ** -0.5, want, bs), 96)
        dense = sd.sd_kv_attn(q, c.cache, c.tt, c.ln, D ** -0.5, lse=lse)
        assert_attention(dense, lse, oracle.attend(f64(q), view, c.t, P, lens, D ** -0.5), 256)


def test_bf16_cache_with_selected_blocks_and_the_csr_attention():
    import torch
    import top_sparse_decode_paged_b200 as sd
    from helpers import assert_out_close
    lens = [300, 77]
    P, bs, G, D, H = 32, 16, 4, 128, 16
    c = Loop("bf16", lens, P, bs, G, D, H, seed=70)
    q = c.store(np.concatenate([[0], np.cumsum(lens)]), lens, 71)
    last = q[torch.tensor([299, 376]).cuda()].contiguous()
    idx = sd.sd_block_topk(last, c.cache, c.tt, c.ln, 5, 300)
    want = oracle.block_topk(f64(last), c.after["b"], c.t, P, bs, lens, 5, 1, 1)
    assert np.array_equal(idx.cpu().numpy(), want)
    offs = (torch.arange(2 * G + 1, dtype=torch.int32) * 5).cuda()
    out = sd.sd_sparse_attn_csr(last, c.cache.k_pages, c.cache.v_pages, c.tt, c.ln, idx, offs, bs, 5 * bs, D ** -0.5, D)
    view = dict(k=c.after["k"], v=c.after["v"], ks=c.after["ks"], vs=c.after["vs"], bs=bs)
    assert_out_close(f64(out), oracle.attend(f64(last), view, c.t, P, lens, D ** -0.5, want, bs)[0], "csr")


def test_refusals():
    import torch
    import top_sparse_decode_paged_b200 as sd
    cache = sd.alloc_kv_cache(4, 16, 1, 64, torch.int8, 8)
    bt, ln = torch.zeros((1, 2), dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda()
    ts = torch.tensor([0, 4], dtype=torch.int32).cuda()
    k = bf16_normal((4, 1, 64), 1).cuda()
    f = _freqs(64).cuda()
    with pytest.raises(ValueError):
        sd.sd_kv_store(None, k.float(), k, cache, bt, ln, ts, f)
    with pytest.raises(ValueError):
        sd.sd_kv_store(None, k, k, cache, bt, ln, ts[:1], f)
    with pytest.raises(ValueError):  # heads that are not dense
        sd.sd_kv_store(bf16_normal((4, 4, 64), 1).cuda()[:, ::2], k, k, cache, bt, ln, ts, f)
    with pytest.raises(sd.SdError):  # rows that are not 8-byte aligned
        odd = bf16_normal((4, 66), 1).cuda()[:, 2:].view(4, 1, 64)
        sd.sd_kv_store(None, odd, k, cache, bt, ln, ts, f)
    with pytest.raises(sd.SdError):  # a rotated width that is no multiple of 8
        sd.sd_kv_store(None, k, k, cache, bt, ln, ts, f[:6].contiguous())
    with pytest.raises(sd.SdError):  # wider than the head
        sd.sd_kv_store(None, k, k, cache, bt, ln, ts, torch.ones(40).cuda())
    with pytest.raises(sd.SdError):
        sd.sd_kv_store(None, k, k, cache, bt, ln, ts, f, eps=-1.0)
