"""Plain fp64 restatement of the blocked-cache calls (test infrastructure only).

Loops over requests, blocks and heads; numpy only. A cache is a dict of arrays:
``k``, ``v`` codes as float64 values [num_pages, P, G, D] (bf16 pools: the
values themselves), ``ks``, ``vs`` scales [num_pages, P // bs, G] (ones for bf16
pools) and ``bs``.
"""
import numpy as np


def norm_rotate(x, w, eps, inv_freq, interleaved, pos):
    """x [heads, D] float64 of one token: norm of every head (w None: none),
    then the rotation of its first 2 * len(inv_freq) dims at ``pos``."""
    x = np.array(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    n = 0 if inv_freq is None else len(inv_freq)
    y = x.copy()
    for i in range(n):
        ang = float(pos) * float(inv_freq[i])
        c, s = np.cos(ang), np.sin(ang)
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        y[:, p] = x[:, p] * c - x[:, q] * s
        y[:, q] = x[:, q] * c + x[:, p] * s
    return y


def token_slot(block_table, P, b, t):
    """(page, slot) of token t of request b."""
    return int(block_table[b, t // P]), t % P


def new_tokens(tok_start, seqlens):
    """For every request: (b, row, position) of each of its new tokens."""
    for b in range(len(seqlens)):
        n = int(tok_start[b + 1] - tok_start[b])
        for i in range(n):
            yield b, int(tok_start[b]) + i, int(seqlens[b]) - n + i


def attend(q, cache, block_table, P, seqlens, scale, picked=None, index_block=1):
    """out [B, H, D], lse [B, H], and for error bounds the weighted sum of |v|
    [B, H, D], the largest |v| and the largest scale * sum |q k| [B, H].``picked`` [B, G, n] lists blocks of
    ``index_block`` tokens; only the first min(n, ceil(L / index_block)) count."""
    B, H, D = q.shape
    G, bs = cache["k"].shape[2], cache["bs"]
    per = H // G
    out = np.zeros((B, H, D))
    mass = np.zeros((B, H, D))
    lse = np.full((B, H), -np.inf)
    vmax = np.zeros((B, H))
    zabs = np.zeros((B, H))
    for b in range(B):
        L = int(seqlens[b])
        for g in range(G):
            toks = list(range(L))
            if picked is not None:
                toks = []
                for e in picked[b, g][: -(-L // index_block)]:
                    if e >= 0:
                        toks += [t for t in range(int(e) * index_block, int(e) * index_block + index_block) if t < L]
            if not toks:
                continue
            t = np.asarray(toks)
            page, slot = block_table[b, t // P], t % P
            ks, vs = cache["ks"][page, slot // bs, g], cache["vs"][page, slot // bs, g]
            k = cache["k"][page, slot, g] * ks[:, None]
            v = cache["v"][page, slot, g] * vs[:, None]
            for h in range(g * per, (g + 1) * per):
                z = scale * (k @ q[b, h])
                m = z.max()
                p = np.exp(z - m)
                out[b, h] = (p @ v) / p.sum()
                mass[b, h] = (p @ np.abs(v)) / p.sum()
                lse[b, h] = m + np.log(p.sum())
                vmax[b, h] = np.abs(v).max()
                zabs[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
    return out, lse, mass, vmax, zabs


def block_scores(q, bounds, block_table, P, bs, b, g, per, count):
    """fp32 roundings of the bounds of request b's blocks under KV head g; a
    head whose sum is not a number (infinities of both signs) is left out."""
    s = np.empty(count, dtype=np.float32)
    for c in range(count):
        page, slot = token_slot(block_table, P, b, c * bs)
        lo, hi = bounds[page, slot // bs, g]
        sums = [np.maximum(q[b, h] * lo, q[b, h] * hi).sum() for h in range(g * per, (g + 1) * per)]
        s[c] = np.float32(max(-np.inf if np.isnan(x) else x for x in sums))
    return s


def block_topk(q, bounds, block_table, P, bs, seqlens, n, n_first, n_last):
    """[B, G, n] ascending, -1 padded."""
    B, H, D = q.shape
    G = bounds.shape[2]
    out = np.full((B, G, n), -1, dtype=np.int32)
    for b in range(B):
        count = -(-int(seqlens[b]) // bs)
        for g in range(G):
            s = block_scores(q, bounds, block_table, P, bs, b, g, H // G, count)
            c = np.arange(count)
            forced = (c < n_first) | (c >= count - n_last)
            order = np.lexsort((c, -s.astype(np.float64), ~forced))
            take = np.sort(order[: min(n, count)])
            out[b, g, : len(take)] = take
    return out
