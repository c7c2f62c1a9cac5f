"""Inputs and conversions for the blocked-cache tests."""
import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
DTYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16}


def table(lens, P, seed, extra=2):
    """A shuffled block table: [B, width], -1 behind the last page, and the number of pages."""
    rng = np.random.default_rng(seed)
    pages = [-(-int(L) // P) for L in lens]
    N = sum(pages) + extra
    perm = rng.permutation(N).astype(np.int32)
    t = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, N


def codes_as_f64(pool):
    return pool.float().cpu().numpy().astype(np.float64)


def random_cache(kind, lens, P, bs, G, D, seed, poison=True, spread=1.0):
    """A filled 8-bit cache in device memory, its block table and its fp64
    view. Slots behind a request's last token and pages of nobody hold the
    codes of NaN (e4m3) or the most negative code (int8), and blocks without a
    token hold NaN scales."""
    import top_sparse_decode_paged_b200 as sd
    rng = np.random.default_rng(seed)
    t, N = table(lens, P, seed)
    used = np.zeros((N, P), dtype=bool)
    for b, L in enumerate(lens):
        for i in range(-(-int(L) // P)):
            used[t[b, i], : min(P, int(L) - i * P)] = True
    pools, scales, values = [], [], []
    for _ in range(2):
        x = rng.standard_normal((N, P, G, D)) * np.exp(spread * rng.standard_normal((N, 1, G, 1)))
        s = np.abs(x).reshape(N, P // bs, bs, G, D).max((2, 4)) / QMAX[kind]
        s = s.astype(np.float32)
        z = torch.from_numpy(x / np.repeat(s, bs, 1)[..., None])
        code = z.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else z.float().clamp(-448, 448).to(torch.float8_e4m3fn)
        raw = code.view(torch.uint8).numpy().copy()
        if poison:
            raw[~used] = 0x80 if kind == "int8" else 0x7F
            s[~used.reshape(N, P // bs, bs).any(2)] = np.nan
        code = torch.from_numpy(raw).view(DTYPE[kind])
        pools.append(code.cuda())
        scales.append(torch.from_numpy(s).cuda())
        values.append(code.float().numpy().astype(np.float64))
    cache = sd.KvCache(pools[0], pools[1], scales[0], scales[1], None, bs)
    view = dict(k=values[0], v=values[1], ks=scales[0].cpu().numpy().astype(np.float64),
                vs=scales[1].cpu().numpy().astype(np.float64), bs=bs)
    return cache, t, view


def bf16_normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def assert_attention(out, lse, ref, n_tokens, what=""):
    """Output and lse within what the arithmetic allows.

    A logit in fp32: a sum of 128 products in 8 matrix instructions and their
    inner sums, and three scalings, each step off by at most 2^-23 of
    zabs = scale * sum |q k|: under 2^-19 zabs, which is also the relative error of its
    weight (2^-21 more for the exponential), once in the numerator and once
    in the denominator. A weight's rounding to fp16: 2^-11 of the weighted sum of |v|,
    and below fp16's normal range 2^-25 of the largest |v| per token (weights are
    relative to a reference that no weight is below for the largest token).
    The output's rounding: half a bf16 step, 2^-8 of the value."""
    o, ls, mass, vmax, zabs = ref
    got, glse = f64(out), lse.cpu().numpy().astype(np.float64)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -20 + 2.0 ** -18 * zabs)[..., None] * mass * 1.01
    tol += n_tokens * 2.0 ** -25 * vmax[..., None] + 1e-30
    bad = np.abs(got - o) > tol
    assert np.isfinite(got).all(), what
    assert not bad.any(), (what, np.argwhere(bad)[:3], np.abs(got - o)[bad][:3], tol[bad][:3])
    empty = np.isneginf(ls)
    assert (np.isneginf(glse) == empty).all(), what
    assert (np.abs(glse[~empty] - ls[~empty]) <= 2.0 ** -18 * (1 + np.abs(ls) + zabs)[~empty]).all(), what
    assert (got[empty] == 0).all(), what
