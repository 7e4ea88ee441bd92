"""Latent attention, its cache and the rotation on the GPU against the oracle.

Bounds, for bf16 half steps of 2^-8 relative:

  rotation   a cos - b sin in fp32 (three roundings of 2^-24 of |a cos| + |b sin|) and one to bf16:
             2^-8 |r| + 2^-22 (|a cos| + |b sin|), with both terms below 2^4 here
  norm       sums and quotients in fp32 (about 20 roundings of 2^-24), one to bf16: 2^-8 |r| (1 + 2^-10)
  codes      without a norm decided exactly: bit for bit
  out        its rounding, 2^-8 |r|; each probability's rounding to bf16, 2^-8 of the mean W of |v|
             (2^-16 where all steps end the sequence or have masks: two pieces); scores off by e change weights by e:
             e <= 50 roundings (18 products of 32 and their tree) of 2^-24 of scale sum |q||k| < 80
             here, so 2 e < 2^-11, of W
  lse        e, and a few roundings of itself: 2^-12 + 2^-20 |r|
"""

import ctypes

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
import oracle
from oracle import latent as R
from tests import gpu_harness as H
from tests.test_gpu_kv8 import bf16, i32, pages, running

pytestmark = pytest.mark.gpu


class OwnStream(torch.cuda.ExternalStream):
    """A new stream.  torch's own come from a pool of 32 and are handed out again,
    with the workspaces that other tests have made them."""

    def __new__(cls):
        at = ctypes.c_void_p()
        assert dg.lib().hipStreamCreate(ctypes.byref(at)) == 0
        return super().__new__(cls, at.value)


def dev_bf16(x, dev):
    return H.f32_to_device(x, dev).bfloat16()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def blank(blocks, block, L, f8):
    """A pool full of NaN."""
    return (np.full((blocks, block, L), 0x7F, np.uint8) if f8 else np.full((blocks, block, L), np.nan, np.float32),
            np.full((blocks, block, L // 8), np.nan, np.float32),
            np.full((blocks, block, L // 128), np.nan, np.float32) if f8 else None)


def upload(cache, dev):
    latent, rope, scales = cache
    return (torch.from_numpy(latent).to(dev).view(torch.float8_e4m3fn) if scales is not None else dev_bf16(latent, dev),
            dev_bf16(rope, dev), None if scales is None else H.f32_to_device(scales, dev))


def filled(rng, lens, block, L, f8, max_blocks=None):
    """(cache, table) holding random tokens of every sequence, NaN everywhere else; entries without tokens are junk."""
    table, blocks = pages(rng, lens, block, max_blocks)
    latent, rope, scales = blank(blocks, block, L, f8)
    for i, n in enumerate(lens):
        for t in range(n):
            at = (table[i, t // block], t % block)
            c = bf16(rng.standard_normal(L) * np.exp2(rng.integers(-2, 2)))
            rope[at] = bf16(rng.standard_normal(L // 8))
            if f8:
                latent[at], scales[at] = R.quantise(c)
            else:
                latent[at] = c
    return (latent, rope, scales), table


def angles(rng, positions, P):
    a = rng.uniform(-np.pi, np.pi, (positions, P // 2))
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def check_out(out, lse, want, rest=2.0 ** -8):
    r, w, l = want
    got, got_lse = host(out), lse.cpu().numpy().astype(np.float64)
    bound = 2.0 ** -8 * np.abs(r) + (rest + 2.0 ** -11) * w
    assert np.array_equal(np.isnan(got), np.isnan(r)) and np.array_equal(np.isnan(got_lse), np.isnan(l))
    known = ~np.isnan(r)
    off = np.abs(got - r)[known]
    assert (off <= bound[known]).all(), f"{np.max(off / np.maximum(bound[known], 1e-30))} of the bound"
    seen, none = np.isfinite(l), l == -np.inf
    assert (np.abs(got_lse[seen] - l[seen]) <= 2.0 ** -12 + 2.0 ** -20 * np.abs(l[seen])).all()
    assert (got_lse[none] == -np.inf).all()


APPEND = [
    # L, e4m3, block, heads, lengths before, new tokens, interleaved, norm
    (512, False, 64, 16, [0], [1], True, True),
    (512, True, 16, 3, [5, 0, 31], [1, 16, 2], True, False),
    (256, False, 32, 33, [7, 1, 0], [2, 0, 70], False, True),
    (256, True, 128, 1, [0, 100], [129, 29], False, False),
    (512, False, 16, 128, [63, 64], [3, 5], False, False),
    (512, True, 64, 0, list(range(70)), [1] * 70, True, False),
    (256, True, 16, 5, [3], [40], True, True),
]


@pytest.mark.parametrize("L,f8,block,heads,ctx,new,pairs,norm", APPEND)
def test_append(gpu, L, f8, block, heads, ctx, new, pairs, norm):
    print(f"[case] latent append {L} {f8} {block} {heads} {len(ctx)}", flush=True)
    rng = np.random.default_rng(L + block + heads)
    P, total = L // 8, sum(new)
    table, blocks = pages(rng, [a + b for a, b in zip(ctx, new)], block)
    before = blank(blocks, block, L, f8)
    wide = bf16(rng.standard_normal((total + 2, 64 + L + P + 8)) * 4)       # two rows behind the last sequence
    q = bf16(rng.standard_normal((total + 2, max(heads, 1), 2 * P)))
    w = bf16(rng.uniform(0.5, 1.5, L)) if norm else None
    an = angles(rng, max(a + b for a, b in zip(ctx, new)), P)
    x, qd = dev_bf16(wide, gpu), dev_bf16(q, gpu)
    cache = upload(before, gpu)
    qo = torch.full((total + 2, max(heads, 1), P), float("nan"), dtype=torch.bfloat16, device=gpu)
    dg.latent_append(x[:, 64:64 + L], x[:, 64 + L:64 + L + P], cache, i32(table, gpu), i32(ctx, gpu), i32(running(new), gpu),
                     max(new), H.f32_to_device(an, gpu), None if w is None else dev_bf16(w, gpu),
                     q_rope=qd[..., P:] if heads else None, q_out=qo if heads else None, interleaved=pairs)
    want, q_want = R.append_ref(wide[:, 64:64 + L], wide[:, 64 + L:64 + L + P], before, table, ctx, running(new), an, w,
                                q=q[..., P:] if heads else None, interleaved=pairs)
    for got, r in [(host(cache[1]), want[1])] + ([(host(qo), q_want)] if heads else []):
        assert np.array_equal(np.isnan(got), np.isnan(r))
        assert (np.abs(got - r)[~np.isnan(r)] <= (2.0 ** -8 * np.abs(r) + 2.0 ** -17)[~np.isnan(r)]).all()
    if not f8:
        got, r = host(cache[0]), want[0]
        assert np.array_equal(np.isnan(got), np.isnan(r))
        ok = ~np.isnan(r)
        assert (np.abs(got - r)[ok] <= 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(r)[ok]).all() if norm else np.array_equal(got[ok], r[ok])
    elif not norm:
        assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), want[0])
        assert np.array_equal(cache[2].cpu().numpy(), want[2], equal_nan=True)
    else:
        # a value next to a border may go either way: half a step of the oracle's, and what the norm is off by
        here = np.isfinite(want[2])
        assert np.array_equal(cache[2].cpu().numpy()[here], want[2][here])
        written = np.repeat(here, 128, -1)
        got = oracle.decode(cache[0].view(torch.uint8).cpu().numpy()).astype(np.float64)
        scale = np.repeat(want[2].astype(np.float64), 128, -1)
        y = np.full(got.shape, np.nan)
        for s in range(len(ctx)):
            for i in range(new[s]):
                pos = ctx[s] + i
                y[table[s, pos // block], pos % block] = R.normalise(wide[running(new)[s] + i, 64:64 + L], w, 1e-6)
        bound = np.maximum(2.0 ** -4 * np.abs(y / scale), 2.0 ** -10) * (1 + 2.0 ** -10)
        assert (np.abs(got - y / scale)[written] <= bound[written]).all()


def test_append_in_place_and_beside_the_table(gpu):
    rng = np.random.default_rng(3)
    L, P, block = 256, 32, 16
    # sequence 0: block 1 missing; 1: entry past the pool; 2: runs out of the table, and of the angles
    table = np.array([[0, -1, 1], [2, 1000, 3], [4, 5, 6]], np.int32)
    before, new, ctx = blank(8, block, L, True), [40, 20, 30], [0, 5, 30]
    an, total = angles(rng, 56, P), 90
    wide, q = bf16(rng.standard_normal((total, L + P))), bf16(rng.standard_normal((total, 4, P)))
    x, qd = dev_bf16(wide, gpu), dev_bf16(q, gpu)
    cache = upload(before, gpu)
    dg.latent_append(x[:, :L], x[:, L:], cache, i32(table, gpu), i32(ctx, gpu), i32(running(new), gpu), 40,
                     H.f32_to_device(an, gpu), q_rope=qd)
    want, q_want = R.append_ref(wide[:, :L], wide[:, L:], before, table, ctx, running(new), an, q=q)
    assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), want[0])
    assert np.array_equal(np.isnan(host(cache[1])), np.isnan(want[1]))
    got = host(qd)
    ignored = np.isnan(q_want)
    assert ignored.any() and np.array_equal(got[ignored], q[ignored])       # positions past the angles
    assert (np.abs(got - q_want)[~ignored] <= 2.0 ** -8 * np.abs(q_want)[~ignored] + 2.0 ** -17).all()


def test_append_more_tokens_than_the_longest(gpu):
    rng = np.random.default_rng(4)
    L, P, block = 512, 64, 32
    table, blocks = pages(rng, [10, 10], block)
    before, an = blank(blocks, block, L, False), angles(rng, 16, P)
    wide = bf16(rng.standard_normal((20, L + P)))
    cache = upload(before, gpu)
    x = dev_bf16(wide, gpu)
    dg.latent_append(x[:, :L], x[:, L:], cache, i32(table, gpu), i32([0, 0], gpu), i32([0, 10, 20], gpu), 7,
                     H.f32_to_device(an, gpu), interleaved=False)
    got = host(cache[0])
    for s in range(2):
        assert np.array_equal(got[table[s, 0], :7], wide[10 * s:10 * s + 7, :L]) and np.isnan(got[table[s, 0], 7:]).all()


def test_append_non_finite(gpu):
    L, P, block = 256, 32, 16
    c = np.zeros((4, L), np.float32)
    c[0, :4] = [np.inf, -np.inf, np.nan, 1.0]
    c[1, :2] = [1e38, -1.0]
    c[1, 128:130] = [1e-30, 448.0]
    c[3] = 1e-39
    c = bf16(c)
    table = np.array([[1]], np.int32)
    before, an = blank(2, block, L, True), angles(np.random.default_rng(0), 4, P)
    cache = upload(before, gpu)
    rope = np.ones((4, P), np.float32)
    dg.latent_append(dev_bf16(c, gpu), dev_bf16(rope, gpu), cache, i32(table, gpu), i32([0], gpu), i32([0, 4], gpu), 4,
                     H.f32_to_device(an, gpu))
    want, _ = R.append_ref(c, rope, before, table, [0], [0, 4], an)
    assert np.array_equal(oracle.decode(cache[0].view(torch.uint8).cpu().numpy()), oracle.decode(want[0]), equal_nan=True)
    assert np.array_equal(cache[2].cpu().numpy(), want[2], equal_nan=True)


@pytest.mark.parametrize("L,f8,block,starts,lens", [
    (512, True, 64, [0, 3, 100], [1, 70, 129]), (256, False, 16, [0, 0], [33, 0]), (512, False, 128, [17], [200]),
    (256, True, 32, [1, 2], [5, 65])])
def test_gather(gpu, L, f8, block, starts, lens):
    print(f"[case] latent gather {L} {f8} {block}", flush=True)
    rng = np.random.default_rng(L + block)
    cache, table = filled(rng, [a + b for a, b in zip(starts, lens)], block, L, f8)
    table = np.concatenate((table, np.full((len(lens), 1), -1, np.int32)), 1)
    on = upload(cache, gpu)
    total = sum(lens) + 3                                                    # three rows behind the last sequence
    rows = torch.full((total, L), float("nan"), dtype=torch.bfloat16, device=gpu)
    rope = torch.full((total, L // 8), float("nan"), dtype=torch.bfloat16, device=gpu)
    dg.latent_gather(on, i32(table, gpu), i32(running(lens), gpu), rows, rope, starts=i32(starts, gpu))
    at = 0
    for s, (a, n) in enumerate(zip(starts, lens)):
        c, r, there = R.tokens_of(cache, table, s, a, n)
        assert there.all() and np.array_equal(host(rows)[at:at + n], c) and np.array_equal(host(rope)[at:at + n], r)
        at += n
    assert np.isnan(host(rows)[at:]).all() and np.isnan(host(rope)[at:]).all()


def test_gather_leaves_what_the_table_does_not_have(gpu):
    rng = np.random.default_rng(5)
    cache, table = filled(rng, [48], 16, 256, True)
    table[0, 1] = 999
    rows = torch.full((80, 256), 7.0, dtype=torch.bfloat16, device=gpu)
    rope = torch.full((80, 32), 7.0, dtype=torch.bfloat16, device=gpu)
    dg.latent_gather(upload(cache, gpu), i32(table, gpu), i32([0, 80], gpu), rows, rope)
    c, r, there = R.tokens_of(cache, table, 0, 0, 48)
    assert np.array_equal(host(rows)[:48][there], c[there]) and (host(rows)[:48][~there] == 7).all()
    assert (host(rows)[48:] == 7).all() and (host(rope)[16:32] == 7).all()


ABSORBED = [
    # L, e4m3, block, heads, new tokens, lengths
    (512, False, 64, 16, [1], [1]),
    (512, False, 64, 16, [1], [64]),
    (512, True, 16, 8, [1, 1, 1], [65, 17, 300]),
    (256, False, 16, 8, [1], [777]),
    (256, True, 32, 128, [1, 1], [150, 40]),
    (512, True, 64, 128, [1, 1], [200, 129]),
    (512, False, 128, 128, [1], [515]),
    (512, True, 32, 20, [3, 1, 2], [100, 1, 258]),
    (256, False, 64, 5, [40, 7, 0, 66], [40, 90, 31, 200]),
    (512, False, 16, 1, [1, 3], [130, 3]),
    (512, False, 32, 31, [1, 1], [70, 300]),
    (256, True, 128, 33, [2, 5], [64, 140]),
    (512, True, 16, 40, [9], [130]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("L,f8,block,heads,new,lens", ABSORBED)
def test_absorbed(gpu, L, f8, block, heads, new, lens, causal):
    print(f"[case] absorbed {L} {f8} {block} {heads} {new} {lens} {causal}", flush=True)
    rng = np.random.default_rng(L + block + heads + sum(lens))
    cache, table = filled(rng, lens, block, L, f8)
    total = sum(new)
    q, qr = bf16(rng.standard_normal((total, heads, L))), bf16(rng.standard_normal((total, heads, L // 8)))
    out = torch.full((total + 2, heads, L), float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full((total + 2, heads), float("nan"), device=gpu)
    pad = lambda x: dev_bf16(np.concatenate((x, x[:1], x[:1])), gpu)  # noqa: E731  (two rows behind the last sequence)
    dg.latent_attention(pad(q), pad(qr), upload(cache, gpu), i32(table, gpu), i32(lens, gpu), i32(running(new), gpu), max(new),
                        out, lse, causal=causal)
    want = R.attention_ref(q, qr, cache, table, lens, running(new), (L * 3 / 8) ** -0.5, causal)
    strict = max(lens) < 64  # 64 tokens are a step that all rows see wholly: one piece
    check_out(out[:total], lse[:total], want, 2.0 ** -16 if strict else 2.0 ** -8)
    assert torch.isnan(out[total:]).all() and torch.isnan(lse[total:]).all()


EXPANDED = [
    # D, heads, queries, tokens
    (128, 2, [1], [1]),
    (128, 3, [5, 64], [5, 64]),
    (64, 5, [150, 40, 7], [150, 40, 7]),
    (128, 1, [130, 0, 3], [200, 20, 300]),
    (64, 8, [1, 17], [129, 500]),
    (128, 4, [257], [257]),
    (64, 1, [70, 70], [65, 0]),                                              # queries before the first token
    (128, 2, [20], [3]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,heads,new,lens", EXPANDED)
def test_expanded(gpu, D, heads, new, lens, causal):
    print(f"[case] expanded {D} {heads} {new} {lens} {causal}", flush=True)
    rng = np.random.default_rng(D + heads + sum(lens))
    total, keys = sum(new), sum(lens)
    q = bf16(rng.standard_normal((total, heads, D + D // 2)))
    kv = bf16(rng.standard_normal((keys, heads, 2 * D)))
    r = bf16(rng.standard_normal((keys, D // 2)))
    out = torch.full((total + 2, heads, D), float("nan"), dtype=torch.bfloat16, device=gpu)
    lse = torch.full((total + 2, heads), float("nan"), device=gpu)
    q_on = dev_bf16(np.concatenate((q, q[:1], q[:1])), gpu)
    # keys and values as a part of a wider row, behind them tokens that are no sequence's
    kv_on = torch.full((keys + 70, heads * 2 * D + 24), float("nan"), dtype=torch.bfloat16, device=gpu)
    kv_on[:keys, 8:8 + heads * 2 * D] = dev_bf16(kv, gpu).flatten(1)
    r_on = torch.full((keys + 70, D), float("nan"), dtype=torch.bfloat16, device=gpu)
    r_on[:keys, D // 2:] = dev_bf16(r, gpu)
    dg.latent_expanded_attention(q_on, kv_on[:, 8:8 + heads * 2 * D].unflatten(1, (heads, 2 * D)), r_on[:, D // 2:],
                                 i32(running(new), gpu), i32(running(lens), gpu), max(new), out, lse, causal=causal)
    want = R.expanded_ref(q, kv, r, running(new), running(lens), (D * 3 / 2) ** -0.5, causal)
    strict = max(lens) < 64  # 64 tokens are a step that all rows see wholly: one piece
    check_out(out[:total], lse[:total], want, 2.0 ** -16 if strict else 2.0 ** -8)
    assert torch.isnan(out[total:]).all() and torch.isnan(lse[total:]).all()
