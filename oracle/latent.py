"""Latent attention, its paged cache and the rotation of rope parts.  Test infrastructure only.

The cache is (latent, rope, scales) as the library lays it out, with latent
[blocks, block, L] as float values (bf16 caches, scales None) or uint8 e4m3
codes, rope [blocks, block, L/8] as float values, scales [blocks, block, L/128]
float32.  Everything is float64; nothing is rounded but codes.
"""

import numpy as np

from . import e4m3
from .kv8 import page_of, pow2_scale


def rotate(x, angles, interleaved):
    """x [..., P] turned by angles [..., P] = cosines | sines (broadcast over heads)."""
    half = x.shape[-1] // 2
    c, s = np.asarray(angles[..., :half], np.float64), np.asarray(angles[..., half:], np.float64)
    x = np.asarray(x, np.float64)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y = np.empty_like(x)
    turned = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0::2], y[..., 1::2] = turned
    else:
        y[..., :half], y[..., half:] = turned
    return y


def normalise(c, norm, eps):
    c = np.asarray(c, np.float64)
    return c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)


def quantise(y):
    """[L] -> (codes, scales [L/128])."""
    codes, scales = np.empty(y.shape, np.uint8), []
    for g in range(0, y.shape[0], 128):
        size = np.abs(y[g:g + 128][np.isfinite(y[g:g + 128])])
        s = pow2_scale(float(size.max()) if size.size else 0.0)
        codes[g:g + 128] = e4m3.encode(y[g:g + 128] / s)
        scales.append(s)
    return codes, np.array(scales, np.float32)


def append_ref(latent, rope, cache, table, ctx, cu, angles, norm=None, eps=1e-6, q=None, interleaved=True):
    """(cache after the new tokens joined it, with bf16 latents and rope parts not
    rounded; q turned, rows that are no token's NaN)."""
    lat, rop = np.array(cache[0], np.float64 if cache[2] is None else np.uint8), np.array(cache[1], np.float64)
    scl = None if cache[2] is None else np.array(cache[2])
    blocks, block, _ = lat.shape
    turned = None if q is None else np.full(q.shape, np.nan)
    for seq in range(table.shape[0]):
        for i in range(int(cu[seq + 1] - cu[seq])):
            row, pos = int(cu[seq]) + i, int(ctx[seq]) + i
            if not 0 <= pos < angles.shape[0]:
                continue
            if q is not None:
                turned[row] = rotate(q[row], angles[pos], interleaved)
            page = page_of(table, blocks, seq, pos, block)
            if page is None:
                continue
            y = np.asarray(latent[row], np.float64) if norm is None else normalise(latent[row], norm, eps)
            if scl is None:
                lat[page, pos % block] = y
            else:
                lat[page, pos % block], scl[page, pos % block] = quantise(y)
            rop[page, pos % block] = rotate(rope[row], angles[pos], interleaved)
    return (lat, rop, scl), turned


def tokens_of(cache, table, seq, first, count):
    """(latents, rope parts, there) of tokens first .. first + count - 1 of one sequence."""
    latent, rope, scales = cache
    blocks, block, L = latent.shape
    c, r, there = np.zeros((count, L)), np.zeros((count, rope.shape[2])), np.zeros(count, bool)
    for i in range(count):
        page = page_of(table, blocks, seq, first + i, block) if first + i >= 0 else None
        if page is None:
            continue
        at = (page, (first + i) % block)
        c[i] = latent[at] if scales is None else e4m3.decode(latent[at]) * np.repeat(scales[at].astype(np.float64), 128)
        r[i] = rope[at]
        there[i] = True
    return c, r, there


def _softmax(x, v):
    """(weighted mean of v, of |v|, log of the sum of exponentials)."""
    top = x.max()
    p = np.exp(x - top)
    return (p @ v) / p.sum(), (p @ np.abs(v)) / p.sum(), top + np.log(p.sum())


def attention_ref(q, q_rope, cache, table, kv_lens, cu, scale, causal=True):
    """Absorbed: (out [total, h, L], the same means of |c|, lse [total, h]), row by row over the tokens it sees."""
    total, heads, L = q.shape
    room = table.shape[1] * cache[0].shape[1]
    out, size, lse = np.zeros((total, heads, L)), np.zeros((total, heads, L)), np.full((total, heads), -np.inf)
    for seq in range(table.shape[0]):
        n, length = int(cu[seq + 1] - cu[seq]), max(int(kv_lens[seq]), 0)
        kv = min(length, room)
        c, r, there = tokens_of(cache, table, seq, 0, kv)
        for i in range(n):
            hi = min(max(length - n + i + 1, 0), kv) if causal else kv
            see = np.flatnonzero(there[:hi])
            for h in range(heads if see.size else 0):
                row = int(cu[seq]) + i
                x = scale * (c[see] @ np.asarray(q[row, h], np.float64) + r[see] @ np.asarray(q_rope[row, h], np.float64))
                out[row, h], size[row, h], lse[row, h] = _softmax(x, c[see])
    return out, size, lse


def expanded_ref(q, kv, k_rope, cu_q, cu_kv, scale, causal=True):
    """Expanded: (out [total, h, D], the same means of |v|, lse [total, h]) of q [total, h, 3 D / 2], kv [total_kv, h, 2 D]."""
    total, heads, _ = q.shape
    D = kv.shape[2] // 2
    out, size, lse = np.zeros((total, heads, D)), np.zeros((total, heads, D)), np.full((total, heads), -np.inf)
    q, kv, k_rope = (np.asarray(x, np.float64) for x in (q, kv, k_rope))
    for seq in range(len(cu_q) - 1):
        n, m, first = int(cu_q[seq + 1] - cu_q[seq]), int(cu_kv[seq + 1] - cu_kv[seq]), int(cu_kv[seq])
        for i in range(n):
            hi = min(max(m - n + i + 1, 0), m) if causal else m
            see = slice(first, first + hi)
            for h in range(heads if hi else 0):
                row = int(cu_q[seq]) + i
                x = scale * (kv[see, h, :D] @ q[row, h, :D] + k_rope[see] @ q[row, h, D:])
                out[row, h], size[row, h], lse[row, h] = _softmax(x, kv[see, h, D:])
    return out, size, lse
