"""The precision of the softmax weights in sd_kv_attn: weights far below the
largest one, products that cancel, V scales many powers of two apart."""
import numpy as np
import pytest

from kv_helpers import DTYPE, f64

pytestmark = pytest.mark.gpu

CODE = {"int8": 100, "e4m3": 96.0}  # a large value that either type holds


def _pool(x, kind):
    import torch
    return torch.as_tensor(x).to(DTYPE[kind]).cuda()


def _first_dim_queries(B, H, D):
    """q = (1, 0, 0, ...): the logit of a token is scale * its K's first dim."""
    import torch
    q = torch.zeros((B, H, D), dtype=torch.bfloat16)
    q[..., 0] = 1
    return q.cuda()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("qpk", [1, 5, 16])
def test_many_tokens_far_below_the_largest(kind, qpk):
    """2^18 tokens of weight 2^-25 each beside one of weight 1 with V = 0:
    together they are 1 / 129 of the softmax and all of the output. So many KV
    heads that one warp walks all tokens of a head; the tokens share a page.

    Weights: off by 2^-17 (logits of 12.5 in base 2, four roundings); the
    output's rounding 2^-8; fp32 sums that add 2^14 times, each cut at
    2^-23 of the sum: 2^-9."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    G, D, P, L = 1184, 64, 64, 1 << 18
    c = CODE[kind]
    k, v = np.zeros((2, P, G, D), np.float32), np.full((2, P, G, D), c, np.float32)
    k[..., 0] = -c
    k[0, 0, :, 0], v[0, 0] = c, 0
    ones = torch.ones((2, 1, G), device="cuda")
    cache = sd.KvCache(_pool(k, kind), _pool(v, kind), ones, ones.clone())
    table = torch.ones((1, L // P), dtype=torch.int32)
    table[0, 0] = 0
    scale = 25 * np.log(2) / (2 * c)
    lse = torch.empty((1, G * qpk), device="cuda")
    out = sd.sd_kv_attn(_first_dim_queries(1, G * qpk, D), cache, table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(), scale, lse=lse)
    w = np.exp(-2 * c * scale)
    n = (L - 1) * w
    got = f64(out)
    assert (np.abs(got - c * n / (1 + n)) <= (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -16) * c * n / (1 + n)).all(), (got.min(), got.max(), c * n / (1 + n))
    assert (np.abs(f64(lse) - (c * scale + np.log1p(n))) <= 2.0 ** -18 * (1 + 2 * c * scale)).all()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("qpk", [1, 3, 4, 5, 8, 16])
def test_products_that_cancel(kind, qpk):
    """Pairs of tokens with w_a v_a + w_b v_b = 0, so that neither the output's rounding
    nor its size hides what the weights lose. A weight: 2^-18.5 (logits of at
    most 6 in base 2, three roundings of them, the exponential's 2^-22, and
    the weight's own 2^-22 or less); 2^-11 more where a KV head has over 8
    query heads, whose weights are held in fp16."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    rng = np.random.default_rng(qpk)
    pairs, D, P = 12, 64, 8
    n = 2 * pairs
    codes = np.arange(64, 128) if kind == "int8" else np.arange(8, 16) * 16.0
    ca, cb = rng.choice(codes, pairs), rng.choice(codes, pairs)
    z = np.empty(n)
    z[1::2] = rng.uniform(-3, 3, pairs)
    z[0::2] = z[1::2] + np.log(cb / ca)
    sign = rng.choice([-1.0, 1.0], (pairs, D))
    v, k = np.empty((n, D), np.float32), np.zeros((n, D), np.float32)
    v[0::2], v[1::2], k[:, 0] = ca[:, None] * sign, -cb[:, None] * sign, 1
    order = rng.permutation(n)
    z, v = z[order].astype(np.float32), v[order]
    ks = torch.from_numpy(z.copy()).cuda()
    # logits of either sign from scales that are not negative
    k[z < 0, 0], ks = -1, ks.abs()
    shape = (n // P, P, 1, D)
    cache = sd.KvCache(_pool(k.reshape(shape), kind), _pool(v.reshape(shape), kind), ks.view(n // P, P, 1), torch.ones((n // P, P, 1), device="cuda"), None, 1)
    table = torch.arange(n // P, dtype=torch.int32)[None].cuda()
    out = f64(sd.sd_kv_attn(_first_dim_queries(1, qpk, D), cache, table, torch.tensor([n], dtype=torch.int32).cuda(), 1.0))
    w = np.exp(z.astype(np.float64) - z.max())
    ref, mass = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -18.5 + (2.0 ** -11 if qpk > 8 else 0)) * mass
    if qpk <= 8:  # the inputs can tell: weights of 11 bits alone miss this by far
        half = w.astype(np.float16).astype(np.float64)
        assert (np.abs(half @ v / w.sum() - ref) > 4 * tol).any()
    assert (np.abs(out - ref) <= tol).all(), (np.abs(out - ref) / mass).max()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("qpk", [1, 5, 16])
@pytest.mark.parametrize("G", [1, 1184])
@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("sv,zero", [(2.0 ** 20, 0.0), (2.0 ** 60, 2.0 ** -100), (2.0 ** 110, 2.0 ** -43)])
def test_zero_values_beside_large_ones(kind, qpk, G, first, sv, zero):
    """One token with a large V scale and half of the softmax; the other half
    belongs to 4095 tokens whose V is zero. Together with V scales the weights
    are 2^130 and more apart. One KV head: partials of many warps; 1184: one
    warp walks all tokens. The output's rounding 2^-8, weights and sums 2^-14."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    D, P, L = 64, 64, 4096
    c = CODE[kind]
    k, v = np.zeros((3, P, G, D), np.float32), np.zeros((3, P, G, D), np.float32)
    at = 0 if first else P - 1
    page = 0 if first else 2
    k[page, at, :, 0], v[page, at] = c, c
    scales = torch.full((3, 1, G), zero, device="cuda")
    scales[page] = sv
    cache = sd.KvCache(_pool(k, kind), _pool(v, kind), torch.ones((3, 1, G), device="cuda"), scales)
    table = torch.ones((1, L // P), dtype=torch.int32)
    table[0, 0], table[0, -1] = 0, 2
    scale = np.log(L - 1) / c
    lse = torch.empty((1, G * qpk), device="cuda")
    out = sd.sd_kv_attn(_first_dim_queries(1, G * qpk, D), cache, table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(), scale, lse=lse)
    got, want = f64(out), 0.5 * c * sv
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -14) * want).all(), (got.min() / want, got.max() / want)
    assert (np.abs(f64(lse) - np.log(2 * (L - 1))) <= 2.0 ** -14).all(), f64(lse).ravel()[:4]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("qpk", [1, 5, 16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27, 2.0 ** 28, 2.0 ** 40])
def test_logits_whose_last_place_is_above_one(kind, qpk, size):
    """Every token has the same V, so the output is V (its rounding 2^-8, weights and
    sums 2^-10) whatever the logits are: rising and falling ones that differ by
    single units in the last place of fp32, and by more."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    rng = np.random.default_rng(int(np.log2(size)))
    D, P, L, G = 64, 16, 16 * 148, 4
    c = CODE[kind]
    k = np.zeros((L // P, P, G, D), np.float32)
    k[..., 0] = 1
    steps = rng.integers(-3, 4, (L, G)).cumsum(0) + rng.integers(0, 30, (L, G)) * (rng.random((L, G)) < 0.2)
    ks = (np.float32(size) + steps * np.spacing(np.float32(size))).astype(np.float32)
    v = np.full((L // P, P, G, D), c, np.float32)
    cache = sd.KvCache(_pool(k, kind), _pool(v, kind), torch.from_numpy(ks).cuda().view(L // P, P, G),
                       torch.ones((L // P, P, G), device="cuda"), None, 1)
    table = torch.arange(L // P, dtype=torch.int32)[None].cuda()
    for scale in (float(np.log(2)), 1.0, 3.7):
        out = f64(sd.sd_kv_attn(_first_dim_queries(1, G * qpk, D), cache, table, torch.tensor([L], dtype=torch.int32).cuda(), scale))
        assert (np.abs(out - c) <= (2.0 ** -8 + 2.0 ** -10) * c).all(), (scale, out.min(), out.max())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("qpk", [1, 5, 16])
@pytest.mark.parametrize("L", [31, 4736])
@pytest.mark.parametrize("sv", [2.0 ** 120, 2.0 ** 90, 2.0 ** -60, 2.0 ** -100])
def test_equal_values_near_the_ends_of_the_range(kind, qpk, L, sv):
    """Every token has the same V, 100 times a scale that puts it near the largest
    bf16 or far below one: the output is V (its rounding 2^-8, weights and sums 2^-10)."""
    import torch
    import top_sparse_decode_paged_b200 as sd
    rng = np.random.default_rng(L)
    D, P, G = 64, 16, 4
    c, n = CODE[kind], -(-L // P)
    k, v = np.zeros((n, P, G, D), np.float32), np.full((n, P, G, D), c, np.float32)
    k[..., 0] = rng.integers(-30, 31, (n, P, G))
    cache = sd.KvCache(_pool(k, kind), _pool(v, kind), torch.ones((n, 1, G), device="cuda"), torch.full((n, 1, G), sv, device="cuda"))
    table = torch.arange(n, dtype=torch.int32)[None].cuda()
    lse = torch.empty((1, G * qpk), device="cuda")
    out = f64(sd.sd_kv_attn(_first_dim_queries(1, G * qpk, D), cache, table, torch.tensor([L], dtype=torch.int32).cuda(), 0.1, lse=lse))
    want = c * sv
    assert (np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -10) * want).all(), (out.min() / want, out.max() / want)
    z = 0.1 * f64(cache.k_pages)[..., 0].reshape(-1, G)[:L]
    ref = np.repeat(np.log(np.exp(z).sum(0)), qpk)
    # logits of up to 20 + log2 sv in base 2, a few roundings of 2^-24 each
    assert (np.abs(f64(lse)[0] - ref) <= 2.0 ** -14).all()
