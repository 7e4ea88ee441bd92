"""The 8-bit key/value cache and attention over it.  Test infrastructure only.

The cache is kept here as the library lays it out: k_codes [blocks, h, block,
d] and v_codes [blocks, h, d, block] of uint8 e4m3 codes, scales [blocks, h]
float32, and a block table per sequence.  Everything is done one block, head
and token at a time in float64; codes and scales are decided exactly (powers
of two).
"""

import math

import numpy as np

from . import e4m3

AMAX_FLOOR = float(np.float32(1e-4))


def pow2_scale(amax):
    """Smallest power of two s with amax <= 448 s."""
    s = 2.0 ** math.floor(math.log2(max(amax, AMAX_FLOOR) / 448.0))
    while s * 448.0 < max(amax, AMAX_FLOOR):
        s *= 2
    return s


def page_of(table, num_blocks, seq, token, block):
    j = token // block
    if j >= table.shape[1] or not 0 <= table[seq, j] < num_blocks:
        return None
    return int(table[seq, j])


def append_ref(k, v, cache, table, ctx, cu):
    """A copy of the cache after k, v [total, h, d] joined it."""
    kc, vc, ks, vs = (np.array(x) for x in cache)
    blocks, heads, block, _ = kc.shape
    for seq in range(table.shape[0]):
        n, c0 = int(cu[seq + 1] - cu[seq]), int(ctx[seq])
        for j in range(c0 // block, -(-(c0 + n) // block) if n else 0):
            page = page_of(table, blocks, seq, j * block, block)
            if page is None:
                continue
            lo, hi = max(j * block, c0), min((j + 1) * block, c0 + n)
            old = max(c0 - j * block, 0)
            rows = slice(int(cu[seq]) + lo - c0, int(cu[seq]) + hi - c0)
            for head in range(heads):
                for x, codes, scales in ((k, kc[page, head], ks), (v, vc[page, head].T, vs)):
                    new = np.asarray(x[rows, head], np.float64)
                    size = np.abs(new[np.isfinite(new)])
                    s = pow2_scale(float(size.max()) if size.size else 0.0)
                    if old:
                        was = float(scales[page, head])
                        s = max(s, was)
                        if s > was:
                            codes[:old] = e4m3.encode(e4m3.decode(codes[:old]) * (was / s))
                    codes[lo - j * block:hi - j * block] = e4m3.encode(new / s)
                    scales[page, head] = s
    return kc, vc, ks, vs


def gather(cache, table, seq, head, length):
    """(keys, values, there) [length, d] float64 of one head; `there` marks tokens the table has."""
    kc, vc, ks, vs = cache
    blocks, _, block, d = kc.shape
    keys, vals, there = np.zeros((length, d)), np.zeros((length, d)), np.zeros(length, bool)
    for j in range(-(-length // block)):
        page = page_of(table, blocks, seq, j * block, block)
        if page is None:
            continue
        n = min(block, length - j * block)
        at = slice(j * block, j * block + n)
        keys[at] = e4m3.decode(kc[page, head, :n]) * float(ks[page, head])
        vals[at] = e4m3.decode(vc[page, head, :, :n].T) * float(vs[page, head])
        there[at] = True
    return keys, vals, there


def attention_ref(q, cache, table, kv_lens, cu, scale, causal=True, window=0):
    """(out [total, h_q, d], lse [total, h_q]) in float64, row by row over the keys it sees.

    Queries stand where the lengths say; tokens past the table's room are seen by none."""
    total, hq, d = q.shape
    heads = cache[0].shape[1]
    room = table.shape[1] * cache[0].shape[2]
    out, lse = np.zeros((total, hq, d)), np.full((total, hq), -np.inf)
    for seq in range(table.shape[0]):
        n, length = int(cu[seq + 1] - cu[seq]), max(int(kv_lens[seq]), 0)
        kv = min(length, room)
        for head in range(heads):
            keys, vals, there = gather(cache, table, seq, head, kv)
            for i in range(n):
                pos = length - n + i
                hi = min(max(pos + 1, 0), kv) if causal else kv
                lo = max(pos - window + 1, 0) if window else 0
                see = [j for j in range(lo, hi) if there[j]]
                if not see:
                    continue
                for h in range(head * hq // heads, (head + 1) * hq // heads):
                    x = scale * (keys[see] @ np.asarray(q[cu[seq] + i, h], np.float64))
                    top = x.max()
                    p = np.exp(x - top)
                    out[cu[seq] + i, h] = (p @ vals[see]) / p.sum()
                    lse[cu[seq] + i, h] = top + np.log(p.sum())
    return out, lse
