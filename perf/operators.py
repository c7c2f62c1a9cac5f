"""Cases and plain forms of the blocked-cache operators: the store with its
norm and rotation, decode attention over the 8-bit cache, and attention over
blocks that a bound on the scores selects.

A cache here is one layer's pools ``[pages, page, G, D]`` cut into blocks of
``bs`` tokens (``bs`` divides the page): an 8-bit pool has one fp32 scale per
(block, KV head) for K and one for V, and each (block, KV head) has the
smallest and largest key of every dimension, in bf16.

    store   y = x * rsqrt(mean(x^2) + eps) * w, rotated by position * inv_freq;
            s = max(amax(new rows), s of the block's earlier rows), rows coded
            as round(y / s), earlier rows coded anew when s grew
    attn8   o = sum_j softmax_j(scale * sk_j * q.k8_j) * sv_j * v8_j
    blocks  bound_c = max over the group's heads of
            sum_d max(q_d * kmin_cd, q_d * kmax_cd); the first and the last
            blocks and the best others, ties to the lower block

``run`` computes them with elementary torch operations, or with the
framework's calls where ``own`` is true.
"""
import math

import torch

own = False

EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}
SMIN = 2.0 ** -100  # no scale is smaller


# ---------------------------------------------------------------- the cases
def listed():
    # The attention shape is that of the per-head selection workload (32 query
    # heads over 8 KV heads of 128), unless a case says otherwise.
    gqa = dict(H=32, G=8, D=128)
    store = dict(op="store", norm=True, rot=128, interleaved=False)
    attn = dict(op="attn", k=0, index_block=1)
    return [
        # one user's next token: the call's latency
        dict(store, name="store_1_token_e4m3", kind="e4m3", B=1, lo=4001, hi=4001, new_lo=1, new_hi=1, page=32, bs=32, **gqa),
        # a decode step of a batch: a row is added to a block that is partly full
        dict(store, name="store_64_tokens_int8", kind="int8", B=64, lo=1, hi=8192, new_lo=1, new_hi=1, page=32, bs=32, **gqa),
        # prompts of odd lengths, read from a packed q, k, v projection
        dict(store, name="store_prompts_int8", kind="int8", B=4, lo=1000, hi=4000, new_lo=1000, new_hi=4000, page=64, bs=64, **gqa),
        # a chunk of each prompt after cached tokens; 64-wide heads, half of them rotated, pairs side by side
        dict(op="store", name="store_chunks_d64_e4m3", kind="e4m3", B=9, lo=700, hi=3000, new_lo=1, new_hi=600, page=48, bs=16,
             norm=False, rot=32, interleaved=True, H=14, G=2, D=64),
        # the cache of a bf16 pool, whose rows the bf16 attention reads
        dict(store, name="store_prompts_bf16", kind="bf16", B=3, lo=2000, hi=5000, new_lo=500, new_hi=3000, page=32, bs=32, **gqa),
        # one user, a short context: latency
        dict(attn, name="attn8_1x1000_int8", kind="int8", B=1, lo=1000, hi=1000, page=32, bs=32, **gqa),
        # a batch after an eviction: ragged lengths
        dict(attn, name="attn8_ragged_e4m3", kind="e4m3", B=16, lo=1040, hi=9232, page=32, bs=16, **gqa),
        # the whole per-head selection cache, every token attended
        dict(attn, name="attn8_16x32768_int8", kind="int8", B=16, lo=32768, hi=32768, page=32, bs=32, **gqa),
        # the tokens that the per-head indexer selects, 1024 for each KV head
        dict(op="attn", name="attn8_top1024_e4m3", kind="e4m3", B=16, lo=32768, hi=32768, page=32, bs=32, k=1024, index_block=1, **gqa),
        # one user's decode step with selected blocks: latency
        dict(op="blocks", name="blocks_1x8192_int8", kind="int8", B=1, lo=8192, hi=8192, page=32, bs=32, n=32, first=1, last=2, **gqa),
        # a batch with long contexts, an eighth of each attended
        dict(op="blocks", name="blocks_16x32768_e4m3", kind="e4m3", B=16, lo=32768, hi=32768, page=32, bs=32, n=128, first=1, last=4, **gqa),
        # ragged, 64-wide heads, few query heads for each KV head, blocks of two to a page
        dict(op="blocks", name="blocks_ragged_d64_int8", kind="int8", B=7, lo=100, hi=20000, page=64, bs=32, n=48, first=1, last=1, H=10, G=5, D=64),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["store", "attn", "attn", "blocks"])
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 8])
    H = G * rng.choice([1, 2, 4, 5, 7, 8, 16] if op != "blocks" else [1, 2, 4, 7, 8])
    page = rng.choice([16, 24, 32, 64, 128])
    bs = rng.choice([b for b in (8, 12, 16, 32, 64, 128) if page % b == 0])
    c = dict(op=op, H=H, G=G, D=D, page=page, bs=bs)
    if op == "store":
        c.update(kind=rng.choice(["int8", "e4m3", "bf16"]), norm=rng.random() < 0.7, rot=rng.choice([D, D, D // 2]), interleaved=rng.random() < 0.3)
        if rng.random() < 0.5:  # a decode step
            c.update(B=_spread(rng, 1, 256), lo=1, hi=_spread(rng, 2, 4096), new_lo=1, new_hi=1)
        else:  # prompts or chunks of them
            hi = _spread(rng, 16, 4096)
            c.update(B=_spread(rng, 1, max(1, 8192 // hi)), lo=hi, hi=hi + _spread(rng, 1, 2048), new_lo=1 + hi // 4, new_hi=hi)
        return c
    c["kind"] = rng.choice(["int8", "e4m3"])
    hi = _spread(rng, 1 if op == "attn" else 64, 65536)
    most = (1 << 28) // (hi * G * D)
    B = _spread(rng, 1, max(1, min(64, most)))
    c.update(B=B, lo=max(1, hi // rng.choice([1, 1, 2, 10])), hi=hi)
    if op == "attn":
        k, ib = 0, 1
        if rng.random() < 0.4:
            ib = rng.choice([1, 1, bs])
            k = _spread(rng, 1, max(1, 2048 // ib))
        c.update(k=k, index_block=ib)
    else:
        n = _spread(rng, 3, 192)
        c.update(n=n, first=rng.choice([0, 1]), last=rng.choice([1, 2]))
    return c


def _between(case, lo, hi, salt):
    """B whole numbers spread over [lo, hi] (over their logarithm), from the case alone; the last is hi."""
    g = torch.Generator().manual_seed(1000003 * salt + 31 * case["B"] + lo + hi)
    u = torch.rand(case["B"], generator=g, dtype=torch.float64)
    v = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round().long().clamp(lo, hi)
    v[-1] = hi
    return v


def _lengths(case):
    return _between(case, case["lo"], case["hi"], 1)


def _new_tokens(case):
    return torch.minimum(_between(case, case["new_lo"], case["new_hi"], 2), _lengths(case))


# ---------------------------------------------------------------- the inputs
def _table(case, lens, g, dev):
    """Pages in a shuffled order, with two that belong to nobody; entries behind a request's last page are -1."""
    P = case["page"]
    pages = (lens + P - 1) // P
    total = int(pages.sum()) + 2
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    width = int(pages.max())
    start = (torch.cumsum(pages, 0) - pages).to(dev)
    j = torch.arange(width, device=dev)
    at = start[:, None] + j[None, :]
    table = torch.where(j[None, :] < pages.to(dev)[:, None], perm[at.clamp(max=total - 1)], torch.full_like(perm[:1], -1))
    return table.contiguous(), total


def _encode(y, s, kind):
    z = y / s
    if kind == "int8":
        return z.round().clamp(-127, 127).to(torch.int8)
    return z.clamp(-448, 448).to(torch.float8_e4m3fn)


def _random_pool(case, total, g, dev):
    """A filled pool: keys of one block share a part, as neighbouring tokens' keys do."""
    P, bs, G, D = case["page"], case["bs"], case["G"], case["D"]
    nb = total * (P // bs)
    k = torch.randn(nb, bs, G, D, generator=g, device=dev)
    k += 0.8 * torch.randn(nb, 1, G, D, generator=g, device=dev)
    bounds = torch.stack([k.amin(1), k.amax(1)], 2).to(torch.bfloat16)
    v = torch.randn(nb, bs, G, D, generator=g, device=dev)
    out = []
    for x in (k, v):
        if case["kind"] == "bf16":
            out += [x.to(torch.bfloat16).reshape(total, P, G, D), None]
            continue
        s = (x.abs().amax((1, 3)) / QMAX[case["kind"]]).clamp(min=SMIN)
        out += [_encode(x, s[:, None, :, None], case["kind"]).reshape(total, P, G, D), s.reshape(total, P // bs, G)]
    return out[0], out[2], out[1], out[3], bounds.reshape(total, P // bs, G, 2, D)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    lens = _lengths(case)
    B, H, G, D = case["B"], case["H"], case["G"], case["D"]
    table, total = _table(case, lens, g, dev)
    st = dict(case=case, table=table, seqlens=lens.to(dev, torch.int32), max_seqlen=int(lens.max()))
    kp, vp, ks, vs, bounds = _random_pool(case, total, g, dev)
    st.update(k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, bounds=bounds)
    if case["op"] == "store":
        new = _new_tokens(case)
        T = int(new.sum())
        st["tok_start"] = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(new, 0)]).to(dev, torch.int32)
        st["T"] = T
        st["qkv"] = (torch.randn(T, (H + 2 * G) * D, generator=g, device=dev) * 1.5).to(torch.bfloat16)
        st["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
        st["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if case["norm"] else None
        st["out"] = [torch.empty(T, n, D, dtype=torch.bfloat16, device=dev) for n in (H, G, G)]
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])).float()
    else:
        st["q"] = (1.5 * torch.randn(B, H, D, generator=g, device=dev)).to(torch.bfloat16)
        st["scale"] = D ** -0.5
        st["out"] = torch.empty(B, H, D, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty(B, H, dtype=torch.float32, device=dev)
        if case["op"] == "attn" and case["k"]:
            ib = case["index_block"]
            units = (lens + ib - 1) // ib
            pick = torch.rand(B, G, int(units.max()), generator=g, device=dev)
            pick.masked_fill_((torch.arange(pick.shape[2], device=dev) >= units.to(dev)[:, None])[:, None], 2.0)
            n = min(case["k"], pick.shape[2])
            at = torch.topk(pick, n, dim=2, largest=False).indices
            at = torch.where(torch.gather(pick, 2, at) > 1.0, torch.full_like(at, 1 << 40), at).sort(-1).values
            at = torch.where(at >= 1 << 40, torch.full_like(at, -1), at)
            idx = torch.full((B, G, case["k"]), -1, dtype=torch.int32, device=dev)
            idx[:, :, :n] = at
            st["indices"] = idx
        elif case["op"] == "blocks":
            st["indices"] = torch.empty(B, G, case["n"], dtype=torch.int32, device=dev)
    if own:
        import top_sparse_decode_paged_b200 as sd
        st["cache"] = sd.KvCache(kp, vp, ks, vs, bounds, case["bs"])
        if case["op"] == "attn":
            st["workspace"] = sd.alloc_kv_attn_workspace(B, G, H, D)
        elif case["op"] == "blocks":
            st["workspace"] = sd.alloc_block_step_workspace(B, G, H, D, st["max_seqlen"], case["bs"])
    return st


# ---------------------------------------------------------------- the calls
def run(st):
    case = st["case"]
    if own:
        import top_sparse_decode_paged_b200 as sd
        if case["op"] == "store":
            H, G, D = case["H"], case["G"], case["D"]
            q, k, v = st["qkv"].view(st["T"], H + 2 * G, D).split([H, G, G], 1)
            q_out, k_out, v_out = st["out"]
            sd.sd_kv_store(q, k, v, st["cache"], st["table"], st["seqlens"], st["tok_start"], st["inv_freq"], q_weight=st["q_weight"],
                           k_weight=st["k_weight"], eps=EPS, interleaved=case["interleaved"], q_out=q_out)
            sd.sd_kv_load(st["cache"], st["table"], st["seqlens"], st["tok_start"], st["T"], k_out=k_out, v_out=v_out)
            return _stored(st, q_out, k_out, v_out)
        if case["op"] == "attn":
            sd.sd_kv_attn(st["q"], st["cache"], st["table"], st["seqlens"], st["scale"], indices=st.get("indices"), index_block=case["index_block"],
                          out=st["out"], lse=st["lse"], workspace=st["workspace"])
            return dict(out=st["out"], lse=st["lse"])
        sd.sd_kv_block_step(st["q"], st["cache"], st["table"], st["seqlens"], case["n"], st["max_seqlen"], st["scale"], n_first=case["first"],
                            n_last=case["last"], indices=st["indices"], out=st["out"], lse=st["lse"], workspace=st["workspace"])
        return dict(indices=st["indices"], out=st["out"], lse=st["lse"])
    if case["op"] == "store":
        return _store(st)
    if case["op"] == "attn":
        if case["k"]:
            tok, ok = _listed_tokens(st["indices"], case["index_block"], st["seqlens"])
        else:
            tok, ok = _all_tokens(st)
        return _attend(st, tok, ok)
    indices = _select(st)
    tok, ok = _listed_tokens(indices, case["bs"], st["seqlens"])
    return dict(indices=indices, **_attend(st, tok, ok))


def _stored(st, q, k, v):
    r = dict(q=q, k=k, v=v, bounds=st["bounds"])
    if st["case"]["kind"] != "bf16":
        r.update(k_scales=st["k_scales"], v_scales=st["v_scales"])
    return r


def _normed_rotated(x, w, pos, inv_freq, interleaved, norm):
    """fp32 [T, heads, D]: the norm of each head, then the rotation; angles in 64 bits."""
    x = x.float()
    if norm:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    R = 2 * inv_freq.numel()
    angle = pos.double()[:, None] * inv_freq.double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : R // 2], x[..., R // 2:R]
        y[..., : R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return y


def _store(st):
    case = st["case"]
    H, G, D, P, bs = case["H"], case["G"], case["D"], case["page"], case["bs"]
    q, k, v = st["qkv"].view(st["T"], H + 2 * G, D).split([H, G, G], 1)
    start, L = st["tok_start"].long(), st["seqlens"].long()
    row = torch.arange(st["T"], device=L.device)
    b = torch.searchsorted(start, row, right=True) - 1
    n = start[1:] - start[:-1]
    pos = L[b] - n[b] + row - start[b]
    q_out = _normed_rotated(q, st["q_weight"], pos, st["inv_freq"], case["interleaved"], case["norm"]).to(torch.bfloat16)
    k = _normed_rotated(k, st["k_weight"], pos, st["inv_freq"], case["interleaved"], case["norm"])
    v = v.float()
    table = st["table"].long()
    slot = table[b, pos // P] * P + pos % P                   # pool row of each new token
    blk = slot // bs                                          # a page holds whole blocks
    first = L - n                                             # the first new position of each request
    joined = pos - pos % bs < first[b]                        # whose block holds earlier rows too
    unit = torch.cumsum((pos % bs == 0) | (pos == first[b]), 0) - 1   # which touched block, counted over all requests
    # the smallest and largest key of each touched block
    bounds = st["bounds"].view(-1, G, 2, D)
    kb = k.to(torch.bfloat16).float()
    at = unit[:, None, None].expand(-1, G, D)
    lo = torch.full_like(kb, float("inf")).scatter_reduce_(0, at, kb, "amin")[unit]
    hi = torch.full_like(kb, float("-inf")).scatter_reduce_(0, at, kb, "amax")[unit]
    old = bounds[blk].float()
    with_old = torch.stack([torch.minimum(lo, old[:, :, 0]), torch.maximum(hi, old[:, :, 1])], 2)
    bounds[blk] = torch.where(joined[:, None, None, None], with_old, torch.stack([lo, hi], 2)).to(torch.bfloat16)
    if case["kind"] == "bf16":
        out = []
        for x, pool in ((k, st["k_pages"]), (v, st["v_pages"])):
            rows = pool.view(-1, G, D)
            rows[slot] = x.to(torch.bfloat16)
            out.append(rows[slot])
        return _stored(st, q_out, *out)
    kind = case["kind"]
    # the block that each request's first new token falls in, and its earlier rows
    head = (table[torch.arange(case["B"], device=L.device), first // P] * P + first % P) // bs
    head_rows = head[:, None] * bs + torch.arange(bs, device=L.device)
    earlier = (torch.arange(bs, device=L.device)[None, :] < (first % bs)[:, None])[:, :, None, None]
    out = []
    for x, pool, scales in ((k, st["k_pages"], st["k_scales"]), (v, st["v_pages"], st["v_scales"])):
        rows, s = pool.view(torch.uint8).view(-1, G, D), scales.view(-1, G)
        amax = torch.zeros(st["T"], G, device=L.device).scatter_reduce_(0, unit[:, None].expand(-1, G), x.abs().amax(-1), "amax")[unit]
        s_new = (amax / QMAX[kind]).clamp(min=SMIN)
        s_new = torch.where(joined[:, None], torch.maximum(s_new, s[blk]), s_new)
        s_head = s[head]
        s[blk] = s_new
        ratio = (s_head / s[head])[:, None, :, None]
        old = rows[head_rows]                                                            # [requests, bs, G, D]
        again = _encode(old.view(pool.dtype).float() * torch.where(earlier, ratio, torch.ones_like(ratio)), torch.ones_like(ratio), kind)
        rows[head_rows] = torch.where(earlier, again.view(torch.uint8), old)
        rows[slot] = _encode(x, s_new[..., None], kind).view(torch.uint8)
        out.append((rows[slot].view(pool.dtype).float() * s_new[..., None]).to(torch.bfloat16))
    return _stored(st, q_out, *out)


def _all_tokens(st):
    tok = torch.arange(st["max_seqlen"], device=st["seqlens"].device)[None, None, :]
    ok = tok < st["seqlens"].long()[:, None, None]
    return torch.where(ok, tok, torch.zeros_like(tok)), ok


def _listed_tokens(indices, ib, seqlens):
    """Tokens [B, G, n * ib] of the listed blocks, and which of them exist."""
    i = indices.long()
    tok = (i[..., None] * ib + torch.arange(ib, device=i.device)).flatten(2)
    ok = (i >= 0)[..., None].expand(*i.shape, ib).flatten(2) & (tok < seqlens.long()[:, None, None])
    return torch.where(ok, tok, torch.zeros_like(tok)), ok


def _attend(st, tok, ok):
    case = st["case"]
    B, H, G, D, P, bs = case["B"], case["H"], case["G"], case["D"], case["page"], case["bs"]
    b = torch.arange(B, device=tok.device)[:, None, None]
    row = torch.where(ok, st["table"].long()[b, tok // P] * P + tok % P, torch.zeros_like(tok))   # [B, 1 or G, n]
    g = torch.arange(G, device=tok.device)[None, :, None]
    keep = ok[..., None]
    k = st["k_pages"].view(-1, G, D)[row, g].float().masked_fill_(~keep, 0.0)                     # [B, G, n, D]
    sk = st["k_scales"].view(-1, G)[row // bs, g]
    q = st["q"].float().view(B, G, H // G, D)
    z = (q @ k.transpose(2, 3)) * (st["scale"] * sk)[:, :, None, :]
    del k
    z = z.masked_fill(~ok[:, :, None, :], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    v = st["v_pages"].view(-1, G, D)[row, g].float().masked_fill_(~keep, 0.0)
    sv = st["v_scales"].view(-1, G)[row // bs, g]
    out = (p * torch.where(ok, sv, torch.zeros_like(sv))[:, :, None, :]) @ v
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return dict(out=out.reshape(B, H, D).to(torch.bfloat16), lse=(m + torch.log(total)).reshape(B, H))


def _bounds_of_blocks(st, dtype):
    """The bound of each block, [B, G, blocks], -inf behind the request's last block; and how many blocks each request has."""
    case = st["case"]
    B, H, G, D, P, bs = case["B"], case["H"], case["G"], case["D"], case["page"], case["bs"]
    L = st["seqlens"].long()
    count = (L + bs - 1) // bs
    c = torch.arange(int((st["max_seqlen"] + bs - 1) // bs), device=L.device)
    ok = c[None, :] < count[:, None]
    page = st["table"].long()[:, (c * bs // P).clamp(max=st["table"].shape[1] - 1)]
    at = torch.where(ok, page * (P // bs) + (c * bs % P) // bs, torch.zeros_like(page))
    kb = st["bounds"].view(-1, G, 2, D)[at].to(dtype)                       # [B, blocks, G, 2, D]
    q = st["q"].to(dtype).view(B, G, H // G, D)
    up = torch.einsum("bgqd,bcgd->bgqc", q.clamp(min=0), kb[:, :, :, 1]) + torch.einsum("bgqd,bcgd->bgqc", q.clamp(max=0), kb[:, :, :, 0])
    return up.amax(2).masked_fill(~ok[:, None], float("-inf")), count


def _select(st):
    """[B, G, n] blocks in ascending order, -1 behind them: the first, the last, and the best others."""
    case = st["case"]
    score, count = _bounds_of_blocks(st, torch.float64)                     # values next to the border decide
    score = score.float()
    c = torch.arange(score.shape[2], device=score.device)
    forced = (c[None, :] < case["first"]) | (c[None, :] >= count[:, None] - case["last"])
    score = torch.where((forced & (c[None, :] < count[:, None]))[:, None], torch.full_like(score, float("inf")), score)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    n = min(case["n"], score.shape[2])
    pick = order[..., :n]
    pick = torch.where(pick < count[:, None, None], pick, torch.full_like(pick, 1 << 40)).sort(-1).values
    pick = torch.where(pick >= 1 << 40, torch.full_like(pick, -1), pick).to(torch.int32)
    if n < case["n"]:
        pick = torch.nn.functional.pad(pick, (0, case["n"] - n), value=-1)
    return pick.contiguous()


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    B, H, G, D, bs = case["B"], case["H"], case["G"], case["D"], case["bs"]
    L = _lengths(case)
    size = 2 if case["kind"] == "bf16" else 1
    scale = 0 if case["kind"] == "bf16" else 8
    if case["op"] == "store":
        n = _new_tokens(case)
        T = int(n.sum())
        touched = int(((L + bs - 1) // bs - (L - n) // bs).sum())
        joined = int(((L - n) % bs != 0).sum())
        # q in and out, k and v in, their codes out and read back for the caller, scales and bounds of the touched blocks
        b = T * (2 * H * D * 2 + 2 * G * D * 2 + 2 * G * D * size) + T * 2 * G * D * (size + 2)
        b += (touched + joined) * G * (scale + 4 * D) + 4 * (3 * B + 1)
        return dict(bytes=b, flops=T * (H + G) * D * 8 + T * G * D * 4)
    if case["op"] == "attn":
        tokens = int(L.sum()) if not case["k"] else int(torch.minimum(L, torch.full_like(L, case["k"] * case["index_block"])).sum())
        b = tokens * G * 2 * D + 2 * B * H * D * 2 + 4 * B * H
        b += (B * G * case["k"] * 4 + tokens // case["index_block"] * G * 8) if case["k"] else (tokens // bs) * G * 8
        return dict(bytes=b, flops=tokens * H * D * 4)
    blocks = (L + bs - 1) // bs
    kept = torch.minimum(blocks, torch.full_like(blocks, case["n"]))
    tokens = int(torch.minimum(kept * bs, L).sum())
    b = int(blocks.sum()) * G * 4 * D + tokens * G * 2 * D + int(kept.sum()) * G * 8 + 2 * B * H * D * 2 + 4 * B * H + 4 * B * G * case["n"]
    return dict(bytes=b, flops=int(blocks.sum()) * H * D * 4 + tokens * H * D * 4)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(st)
    if case["op"] == "attn" and not case["k"]:
        return _exact_attention(st, None, 1)
    if case["op"] == "attn":
        return _exact_attention(st, st["indices"], case["index_block"])
    picked = _exact_selection(st)
    r = _exact_attention(st, picked, case["bs"])
    return dict(indices=None, **r)


def _exact_attention(st, picked, ib):
    """One request and KV head after the other."""
    case = st["case"]
    B, H, G, D, P, bs = case["B"], case["H"], case["G"], case["D"], case["page"], case["bs"]
    per = H // G
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(st["seqlens"][b])
        pages = st["table"][b].long()
        for g in range(G):
            if picked is None:
                t = torch.arange(L, device="cuda")
            else:
                i = picked[b, g].long()
                i = i[i >= 0]
                t = (i[:, None] * ib + torch.arange(ib, device="cuda")).flatten()
                t = t[t < L]
            if not t.numel():
                continue
            page, slot = pages[t // P], t % P
            k = st["k_pages"][page, slot, g].double() * st["k_scales"][page, slot // bs, g].double()[:, None]
            v = st["v_pages"][page, slot, g].double() * st["v_scales"][page, slot // bs, g].double()[:, None]
            h = slice(g * per, g * per + per)
            z = st["scale"] * (st["q"][b, h].double() @ k.T)
            lse[b, h] = torch.logsumexp(z, -1)
            out[b, h] = torch.softmax(z, -1) @ v
    return dict(out=out, lse=lse)


def _exact_selection(st):
    case = st["case"]
    B, H, G, D, P, bs = case["B"], case["H"], case["G"], case["D"], case["page"], case["bs"]
    per = H // G
    picked = torch.full((B, G, case["n"]), -1, dtype=torch.long, device="cuda")
    for b in range(B):
        count = -(-int(st["seqlens"][b]) // bs)
        c = torch.arange(count, device="cuda")
        page, at = st["table"][b].long()[c * bs // P], (c * bs % P) // bs
        q = st["q"][b].double()
        for g in range(G):
            kb = st["bounds"][page, at, g].double()                          # [count, 2, D]
            best = torch.stack([torch.maximum(q[h] * kb[:, 0], q[h] * kb[:, 1]).sum(-1) for h in range(g * per, g * per + per)]).amax(0)
            best[: case["first"]] = float("inf")
            best[max(0, count - case["last"]):] = float("inf")
            take = torch.argsort(best, descending=True, stable=True)[: case["n"]]
            picked[b, g, : take.numel()] = take.sort().values
    return picked


def _exact_store(st):
    case = st["case"]
    H, G, D, P, bs, kind = case["H"], case["G"], case["D"], case["page"], case["bs"], case["kind"]
    T, half = st["T"], case["rot"] // 2
    x = st["qkv"].double().view(T, H + 2 * G, D)
    starts, lens = st["tok_start"].tolist(), st["seqlens"].tolist()
    pos = torch.cat([torch.arange(lens[b] - (starts[b + 1] - starts[b]), lens[b], device="cuda") for b in range(case["B"])])
    turn = pos.double()[:, None, None] * st["inv_freq"].double()
    heads = []
    for part, w in ((x[:, :H], st["q_weight"]), (x[:, H:H + G], st["k_weight"])):
        if case["norm"]:
            part = part / torch.sqrt(part.pow(2).mean(-1, keepdim=True) + EPS) * w.double()
        r = part[..., : 2 * half]
        pair = torch.view_as_complex(r.unflatten(-1, (half, 2)).contiguous() if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2).contiguous())
        pair = torch.view_as_real(pair * torch.polar(torch.ones_like(turn), turn))
        r = pair.flatten(-2) if case["interleaved"] else pair.transpose(-1, -2).flatten(-2)
        heads.append(torch.cat([r, part[..., 2 * half:]], -1))
    res = dict(q=heads[0])
    bounds = st["bounds"].double()
    scales = {"k": st["k_scales"], "v": st["v_scales"]}
    new = {"k": heads[1], "v": x[:, H + G:]}
    got = {n: torch.empty(T, G, D, dtype=torch.float64, device="cuda") for n in new}
    if kind != "bf16":
        scales = {n: s.double().clone() for n, s in scales.items()}
    for b in range(case["B"]):
        p0, p1 = lens[b] - (starts[b + 1] - starts[b]), lens[b]
        for c in range(p0 // bs, -(-p1 // bs)):                              # each touched block
            lo, hi = max(p0, c * bs), min(p1, c * bs + bs)
            if lo >= hi:
                continue
            rows = slice(starts[b] + lo - p0, starts[b] + hi - p0)
            page, at = int(st["table"][b, c * bs // P]), (c * bs % P) // bs
            earlier = lo > c * bs
            kk = new["k"][rows]
            ends = torch.stack([kk.amin(0), kk.amax(0)], 1)
            if earlier:
                o = bounds[page, at]
                ends = torch.stack([torch.minimum(ends[:, 0], o[:, 0]), torch.maximum(ends[:, 1], o[:, 1])], 1)
            bounds[page, at] = ends
            for n, y in new.items():
                if kind == "bf16":
                    got[n][rows] = y[rows]
                    continue
                s = (y[rows].abs().amax((0, 2)) / QMAX[kind]).clamp(min=SMIN)
                if earlier:
                    s = torch.maximum(s, scales[n][page, at])
                scales[n][page, at] = s
                z = y[rows] / s[:, None]
                z = z.round().clamp(-127, 127) if kind == "int8" else z.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                got[n][rows] = z * s[:, None]
    res.update(got, bounds=bounds)
    if kind != "bf16":
        res.update(k_scales=scales["k"], v_scales=scales["v"])
    return res
