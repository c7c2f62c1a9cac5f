"""The codes of the 8-bit store, bit for bit: without norm and rotation every
step of the definition is one fp32 operation on bf16 values,

    scale = max(amax / qmax, the scale of earlier rows, 2^-100)
    code  = round(y / scale), earlier codes round(code * (old / new)),

rounding to even, so nothing is left to a tolerance."""
import numpy as np
import pytest

from kv_helpers import DTYPE, QMAX, bf16_normal, table

pytestmark = pytest.mark.gpu

F = np.float32


def _round(z, kind):
    import torch
    if kind == "int8":
        return torch.from_numpy(np.clip(np.rint(z), -127, 127)).to(torch.int8).view(torch.uint8).numpy()
    return torch.from_numpy(z).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def _codes(pool):
    import torch
    return pool.view(torch.uint8).cpu().numpy()


def _values(raw, kind):
    import torch
    return torch.from_numpy(raw.copy()).view(DTYPE[kind]).float().numpy()


class Cache:
    """A cache and what its codes and scales have to be."""

    def __init__(self, kind, lens, P, bs, G, D, seed):
        import torch
        import top_sparse_decode_paged_b200 as sd
        self.sd, self.kind, self.P, self.bs, self.G, self.D = sd, kind, P, bs, G, D
        self.t, N = table(lens, P, seed)
        self.cache = sd.alloc_kv_cache(N, P, G, D, DTYPE[kind], bs)
        self.want = [np.zeros((N, P, G, D), np.uint8) for _ in range(2)]
        self.scales = [np.zeros((N, P // bs, G), F) for _ in range(2)]
        self.tt = torch.from_numpy(self.t).cuda()

    def store(self, kv, new, seqlens):
        """kv [T, 2 G, D] bf16: the last new[b] tokens of each request; then compares the whole cache."""
        import torch
        G, bs, P, kind = self.G, self.bs, self.P, self.kind
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        k, v = kv.cuda().split([G, G], 1)
        dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.sd.device_errors(clear=True)
        self.sd.sd_kv_store(None, k, v, self.cache, self.tt, dev(seqlens), dev(start), None)
        torch.cuda.synchronize()
        assert self.sd.device_errors() == 0
        rows = kv.float().numpy()
        for b, L in enumerate(seqlens):
            p0 = int(L) - int(new[b])
            for c in range(p0 // bs, -(-int(L) // bs)) if new[b] else ():
                lo, hi = max(p0, c * bs), min(int(L), c * bs + bs)
                page, slot = int(self.t[b, lo // P]), lo % P
                blk, first = slot // bs, (c * bs) % P
                y = rows[start[b] + lo - p0: start[b] + hi - p0]
                for i in range(2):
                    x, pool, sc = y[:, i * G:(i + 1) * G], self.want[i], self.scales[i]
                    finite = np.where(np.isfinite(x), np.abs(x), F(0))
                    s = np.maximum(finite.max((0, 2)) / F(QMAX[kind]), F(2.0 ** -100))
                    if lo > c * bs:
                        old = sc[page, blk].copy()
                        s = np.maximum(s, old)
                        held = _values(pool[page, first:slot], kind)
                        ratio = (old / s)[None, :, None]
                        grew = (s > old)[None, :, None]
                        pool[page, first:slot] = np.where(grew, _round(held * ratio, kind), pool[page, first:slot])
                    sc[page, blk] = s
                    with np.errstate(invalid="ignore"):
                        z = x / s[None, :, None]
                    pool[page, slot:slot + hi - lo] = _round(np.where(np.isnan(z), F(0), z), kind)
        for pool, want, sc, ws in ((self.cache.k_pages, self.want[0], self.cache.k_scales, self.scales[0]),
                                   (self.cache.v_pages, self.want[1], self.cache.v_scales, self.scales[1])):
            assert np.array_equal(sc.cpu().numpy(), ws)
            got = _codes(pool)
            zero = lambda x: np.where(x == 0x80, 0, x) if kind == "e4m3" else x  # noqa: E731  (-0 and 0)
            bad = zero(got) != zero(want)
            assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_chunks_and_steps(kind, D):
    lens = [300, 77, 1, 200]
    c = Cache(kind, [L + 60 for L in lens], 32, 16, 3, D, seed=D)
    c.store(bf16_normal((sum(lens), 6, D), 1, 1.5), lens, lens)
    chunk = [33, 0, 17, 40]
    now = [a + b for a, b in zip(lens, chunk)]
    c.store(bf16_normal((sum(chunk), 6, D), 2, 2.5), chunk, now)
    for i in range(8):
        now = [n + 1 for n in now]
        c.store(bf16_normal((4, 6, D), 3 + i, 1.0 + 0.5 * i), [1] * 4, now)
    c.store(bf16_normal((8, 6, D), 30, 4.0), [5, 1, 0, 2], [a + b for a, b in zip(now, [5, 1, 0, 2])])


def _tied(kind, D, rows, seed):
    """Rows whose quotients are ties again and again: the largest is qmax
    times a power of two (an exact scale) or 7/512 as in 6.125 / 448, and the others
    are scale * (odd multiples of half a step) where bf16 holds them."""
    import torch
    rng = np.random.default_rng(seed)
    scale = {"int8": 2.0 ** -5, "e4m3": 7.0 / 512}[kind]
    if kind == "int8":
        z = rng.integers(-127, 127, (rows, 2, D)) + 0.5
    else:
        e = rng.integers(-6, 8, (rows, 2, D))
        z = (8 + rng.integers(0, 8, (rows, 2, D)) + 0.5) * 2.0 ** (e - 3) * rng.choice([-1.0, 1.0], (rows, 2, D))
    x = torch.from_numpy(z * scale)
    kept = x.to(torch.bfloat16)
    x = torch.where(kept.double() == x, kept, torch.zeros_like(kept))
    x[:, :, 0] = scale * QMAX[kind]
    assert (x[:, :, 1:] != 0).float().mean() > 0.05
    return x


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_exact_ties_go_to_even(kind):
    c = Cache(kind, [200, 9], 32, 32, 1, 128, seed=4)
    c.store(_tied(kind, 128, 150, 5), [148, 2], [148, 2])     # blocks, by CTAs
    for i in range(3):                                        # rows, by warps
        c.store(_tied(kind, 128, 2, 6 + i), [1, 1], [149 + i, 3 + i])


def test_the_tie_of_a_scale_that_is_no_power_of_two():
    """Maximum 6.125: -1.5859375 is -116 scales, a tie between -112 and -120."""
    import torch
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    x[..., 0], x[..., 1] = 6.125, -1.5859375
    c = Cache("e4m3", [1], 16, 16, 1, 64, seed=1)
    c.store(x, [1], [1])
    assert _values(_codes(c.cache.v_pages), "e4m3").min() == -112.0


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -98, 2.0 ** -92, 2.0 ** -55, 1e30, 2.0 ** 125])
def test_scales_far_from_one(kind, size):
    lens = [50, 2]
    c = Cache(kind, [60, 20], 16, 16, 2, 64, seed=7)
    c.store(bf16_normal((52, 4, 64), 8, size), lens, lens)
    c.store(bf16_normal((2, 4, 64), 9, size), [1, 1], [51, 3])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_entries_that_are_not_finite(kind):
    lens = [40, 3]
    c = Cache(kind, [60, 20], 16, 16, 2, 64, seed=10)
    for n, at in ((lens, lens), ([1, 1], [41, 4])):
        x = bf16_normal((sum(n), 4, 64), 11, 2.0)
        x[::2, :, 5], x[::3, :, 6], x[:, 1, 7] = float("inf"), float("-inf"), float("nan")
        c.store(x, n, at)
