"""The 8-bit key/value cache and its attention on the GPU against the oracle.

Caches are compared bit for bit: scales are powers of two, so codes are
decided exactly.  Attention outputs are held to the oracle's acceptance rule
(8e-3 |r| + 1e-3 rms): half an ulp of the bf16 output is 1.95e-3 |r|, and the
probabilities' rounding to fp16 (2^-12 each, independent) adds about
2^-12 rms.  Log-sums are held to 1e-4 + 1e-6 |r|: an fp32 score of d <= 256
products of unit-size factors is off by at most (d + 8) 2^-24 of their
absolute sum, which is below 6 here.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
import oracle
from oracle import kv8
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def bf16(x):
    return oracle.bf16_round(x)


def pages(rng, lens, block, max_blocks=None, spare=2, junk=True):
    """A block table in random order; entries that no token needs hold junk."""
    need = [-(-t // block) for t in lens]
    most = max(need + [1]) if max_blocks is None else max_blocks
    order = list(rng.permutation(sum(need) + spare))
    table = np.full((len(lens), most), 2 ** 30 if junk else -1, np.int32)
    table[:, 1::2] = -7
    for i, n in enumerate(need):
        table[i, :n] = [order.pop() for _ in range(n)]
    return table, sum(need) + spare


def blank(blocks, h, block, d):
    """A pool full of NaN codes and NaN scales."""
    return (np.full((blocks, h, block, d), 0x7F, np.uint8), np.full((blocks, h, d, block), 0xFF, np.uint8),
            np.full((blocks, h), np.nan, np.float32), np.full((blocks, h), np.nan, np.float32))


def to_device(cache, dev):
    return tuple(torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in cache)


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def running(lens):
    return np.concatenate(([0], np.cumsum(lens))).astype(np.int32)


def same_cache(got, want):
    for x, y, name in zip(got, want, ("k_codes", "v_codes", "k_scales", "v_scales")):
        assert np.array_equal(x.cpu().numpy(), y, equal_nan=y.dtype == np.float32), name


def values(rng, shape, spread=6):
    """bf16 values over several binades, so that scales differ and grow."""
    return bf16(rng.standard_normal(shape) * np.exp2(rng.integers(-spread, spread, shape[:-2] + (1, 1))))


APPEND = [
    # block, h_kv, d, lengths before, new tokens
    (16, 1, 64, [0], [1]),
    (16, 2, 64, [5, 0, 31], [1, 16, 2]),
    (64, 3, 128, [63, 64, 1, 200], [1, 1, 130, 0]),
    (128, 2, 256, [0, 100], [129, 29]),
    (32, 1, 128, [7], [200]),
    (64, 8, 128, [1500, 3], [1, 1]),
]


@pytest.mark.parametrize("block,h,d,ctx,new", APPEND)
def test_append(gpu, block, h, d, ctx, new):
    print(f"[case] append block {block} h {h} d {d} {ctx} {new}", flush=True)
    rng = np.random.default_rng(block + h + d)
    table, blocks = pages(rng, [a + b for a, b in zip(ctx, new)], block)
    before, cu0, cu = blank(blocks, h, block, d), running(ctx), running(new)
    if cu0[-1]:
        before = kv8.append_ref(values(rng, (cu0[-1], h, d)), values(rng, (cu0[-1], h, d)), before, table,
                                [0] * len(ctx), cu0)
    # keys and values as slices of one wider projection
    wide = values(rng, (cu[-1], 2 * h + 1, d))
    x = H.f32_to_device(wide, gpu).bfloat16()
    cache = to_device(before, gpu)
    dg.kv8_append(x[:, 1:h + 1], x[:, h + 1:], cache, i32(table, gpu), i32(ctx, gpu), i32(cu, gpu), max(new))
    same_cache(cache, kv8.append_ref(wide[:, 1:h + 1], wide[:, h + 1:], before, table, ctx, cu))


def test_append_token_by_token_with_growing_scales(gpu):
    rng = np.random.default_rng(11)
    h, d, block, n = 2, 64, 32, 70
    k = bf16(rng.standard_normal((n, h, d)) * np.exp2(np.arange(n) % 9)[:, None, None])
    v = bf16(rng.standard_normal((n, h, d)) * np.exp2(-4.0 + np.arange(n) // 7)[:, None, None])
    table, blocks = pages(rng, [n], block)
    want = blank(blocks, h, block, d)
    cache = to_device(want, gpu)
    kd, vd = H.f32_to_device(k, gpu).bfloat16(), H.f32_to_device(v, gpu).bfloat16()
    for i in range(n):
        dg.kv8_append(kd[i:i + 1], vd[i:i + 1], cache, i32(table, gpu), i32([i], gpu), i32([0, 1], gpu), 1)
        want = kv8.append_ref(k[i:i + 1], v[i:i + 1], want, table, [i], [0, 1])
    same_cache(cache, want)


def test_append_non_finite_and_extreme(gpu):
    h, d, block = 1, 64, 16
    k = np.zeros((5, h, d), np.float32)
    k[0, 0, :4] = [np.inf, -np.inf, np.nan, 1.0]
    k[1, 0, :2] = [3e38, -1.0]                     # the scale leaps: older codes vanish but NaN and infinities do not
    k[2, 0, :2] = [1e-30, 448.0]
    k[4] = 1e-39
    k = bf16(k)
    table = np.array([[1, 0]], np.int32)
    want = blank(3, h, block, d)
    cache = to_device(want, gpu)
    kd = H.f32_to_device(k, gpu).bfloat16()
    for lo, hi in ((0, 1), (1, 2), (2, 5)):
        dg.kv8_append(kd[lo:hi], kd[lo:hi], cache, i32(table, gpu), i32([lo], gpu), i32([0, hi - lo], gpu), hi - lo)
        want = kv8.append_ref(k[lo:hi], k[lo:hi], want, table, [lo], [0, hi - lo])
    for x, y in zip(cache, want):
        x = x.cpu().numpy()
        if y.dtype == np.uint8:                    # a NaN's sign is not defined
            assert np.array_equal(oracle.decode(x), oracle.decode(y), equal_nan=True)
        else:
            assert np.array_equal(x, y, equal_nan=True)


def test_append_ignores_what_the_table_does_not_have(gpu):
    rng = np.random.default_rng(12)
    h, d, block = 2, 64, 16
    x = values(rng, (60, h, d))
    # sequence 0: block 1 missing; 1: entry past the pool; 2: runs out of the table's width
    table = np.array([[0, -1, 1], [2, 1000, 3], [4, 5, 6]], np.int32)
    before = blank(8, h, block, d)
    new, ctx = [20, 20, 20], [0, 0, 40]
    cache = to_device(before, gpu)
    xd = H.f32_to_device(x, gpu).bfloat16()
    dg.kv8_append(xd, xd, cache, i32(table, gpu), i32(ctx, gpu), i32(running(new), gpu), 20)
    # the last sequence's block 6 gets its tokens 40..47 without the 8 older ones' scale: start it from a defined one
    want = before
    want[2][6], want[3][6] = np.nan, np.nan
    want = kv8.append_ref(x[:40], x[:40], want, table, ctx, [0, 20, 40, 40])
    got = [y.cpu().numpy() for y in cache]
    for i in (0, 1, 2, 3, 5, 7):
        for a, b in zip(got, want):
            assert np.array_equal(a[i], b[i], equal_nan=b.dtype == np.float32), i


def make_cache(rng, lens, block, h, d, **kw):
    table, blocks = pages(rng, lens, block, **kw)
    cu = running(lens)
    k = bf16(rng.standard_normal((cu[-1], h, d)) + 2.0 * (np.arange(d) % 32 == 5))
    v = values(rng, (cu[-1], h, d), 3)
    return kv8.append_ref(k, v, blank(blocks, h, block, d), table, [0] * len(lens), cu), table


def attend(gpu, q, cache, table, kv, cu, lse=True, **kw):
    total, hq, d = q.shape
    out, flat = H.sentinel_bf16((total, hq, d), gpu, 256)
    sums = torch.full((total, hq), 7.0, device=gpu) if lse else None
    dg.kv8_attention(H.f32_to_device(q, gpu).bfloat16(), to_device(cache, gpu), i32(table, gpu), i32(kv, gpu),
                     i32(cu, gpu), int(np.max(np.diff(cu), initial=0)), out, sums, **kw)
    torch.cuda.synchronize()
    assert H.guard_untouched(flat, total * hq * d)
    return H.d_float(out), None if sums is None else sums.cpu().numpy().astype(np.float64)


def hold(got, want):
    out, lse = got
    res = oracle.tolerance_check(out, want[0])
    assert res["ok"], res
    empty = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(lse), empty) and np.all(out[empty] == 0)
    assert np.all(np.abs(lse[~empty] - want[1][~empty]) <= 1e-4 + 1e-6 * np.abs(want[1][~empty]))


ATTN = [
    # block, h_q, h_kv, d, queries, tokens in the cache, window
    (16, 1, 1, 64, [1], [1], 0),
    (16, 8, 1, 64, [1], [777], 0),
    (64, 4, 4, 128, [1, 1, 1], [1, 64, 65], 0),
    (128, 16, 2, 128, [1, 1], [1000, 129], 0),
    (32, 10, 2, 256, [1, 1, 1], [33, 500, 0], 0),        # a sequence without tokens
    (64, 32, 8, 128, [1] * 5, [300, 64, 5, 128, 1], 0),
    (16, 6, 2, 64, [3, 1, 5], [40, 17, 5], 0),            # several tokens, one sequence all new
    (64, 8, 2, 128, [70, 33], [70, 200], 0),              # prompts, one behind a prefix
    (128, 4, 1, 128, [130], [130], 0),
    (64, 20, 1, 64, [9], [150], 0),                       # 20 heads a group: rows of a tile split a query's heads
    (32, 4, 2, 256, [40], [100], 0),
    (64, 4, 2, 64, [5, 0, 2], [3, 10, 2], 0),             # more queries than tokens; no queries
    (64, 8, 2, 128, [1, 1], [700, 70], 100),
    (16, 4, 4, 64, [50], [300], 7),
    (128, 8, 4, 128, [66, 1], [200, 64], 64),
    (64, 2, 1, 128, [1], [9000], 0),                      # one sequence over many workgroups
    (64, 16, 4, 128, [150, 90, 1], [150, 400, 333], 0),
]


@pytest.fixture(params=["", "kv8_split", "kv8_prompt"])
def way(request, monkeypatch):
    """The library's own choice between its two ways of a call, and each of them."""
    if request.param:
        monkeypatch.setenv("DG_FORCE_CONFIG", request.param)
    return request.param


@pytest.mark.parametrize("block,hq,h,d,new,kv,window", ATTN)
def test_attention(way, gpu, block, hq, h, d, new, kv, window):
    print(f"[case] attention block {block} heads {hq}/{h} d {d} {new} {kv} window {window}", flush=True)
    rng = np.random.default_rng(block + hq + d + len(kv))
    cache, table = make_cache(rng, kv, block, h, d)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], hq, d)))
    want = kv8.attention_ref(q, cache, table, kv, cu, d ** -0.5, window=window)
    got = attend(gpu, q, cache, table, kv, cu, window=window)
    hold(got, want)
    again = attend(gpu, q, cache, table, kv, cu, window=window)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


@pytest.mark.parametrize("new,kv,hq", [([1, 1], [100, 3], 4), ([20, 7], [200, 7], 8)])
def test_attention_not_causal_and_without_lse(way, gpu, new, kv, hq):
    rng = np.random.default_rng(21)
    cache, table = make_cache(rng, kv, 32, 2, 64)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], hq, 64)))
    hold(attend(gpu, q, cache, table, kv, cu, scale=0.3, causal=False),
         kv8.attention_ref(q, cache, table, kv, cu, 0.3, causal=False))
    out, _ = attend(gpu, q, cache, table, kv, cu, lse=False)
    assert oracle.tolerance_check(out, kv8.attention_ref(q, cache, table, kv, cu, 0.125)[0])["ok"]


def test_attention_large_scores_and_far_scales(way, gpu):
    # scores of +-200 (a one-hot softmax), value scales 2^40 apart, some blocks' values zero
    rng = np.random.default_rng(22)
    cache, table = make_cache(rng, [300], 64, 1, 64)
    cache[3][table[0, :5], 0] = np.exp2(np.array([-30, 10, -5, 0, -22], np.float32))
    q = bf16(rng.standard_normal((12, 2, 64)) * np.exp2(np.arange(12) // 2)[:, None, None])
    cu = [0, 12]
    want = kv8.attention_ref(q, cache, table, [300], cu, 1.0)
    out, lse = attend(gpu, q, cache, table, [300], cu, scale=1.0)
    # an fp32 score x is off by up to 72 2^-24 sum |q k|, and so are p and the output relative to its largest term
    for i in range(12):
        for h in range(2):
            keys, vals, _ = kv8.gather(cache, table, 0, 0, 289 + i)
            off = 72 * 2 ** -24 * float((np.abs(keys) @ np.abs(q[i, h])).max())
            size = np.abs(np.exp(keys @ q[i, h].astype(np.float64) - want[1][i, h])[:, None] * vals).sum(0)
            assert np.all(np.abs(out[i, h] - want[0][i, h]) <= 2 ** -8 * np.abs(want[0][i, h]) + (2 * off + 2 ** -10) * size)
            assert abs(lse[i, h] - want[1][i, h]) <= off + 1e-6 * abs(want[1][i, h]) + 1e-6


def nan_case(gpu, new, kv, hq, where, in_values, window=0):
    """NaN put into token `where` of the cache: rows that see it are NaN (for a value in its dimension only), others unhurt."""
    rng = np.random.default_rng(23)
    cache, table = make_cache(rng, [kv], 32, 1, 64)
    q = bf16(rng.standard_normal((new, hq, 64)))
    clean = attend(gpu, q, cache, table, [kv], [0, new], window=window)
    page, at = table[0, where // 32], where % 32
    if in_values:
        cache[1][page, 0, 5, at] = 0xFF
    else:
        cache[0][page, 0, at, 3] = 0x7F
    out, lse = attend(gpu, q, cache, table, [kv], [0, new], window=window)
    for i in range(new):
        pos = kv - new + i
        if pos >= where and (not window or pos - window < where):
            if in_values:
                assert np.isnan(out[i, :, 5]).all(), i
                rest = np.delete(out[i], 5, -1)
                assert np.array_equal(rest, np.delete(clean[0][i], 5, -1)), i
            else:
                assert np.isnan(out[i]).all() and np.isnan(lse[i]).all(), i
        else:
            assert np.array_equal(out[i], clean[0][i]) and np.array_equal(lse[i], clean[1][i]), i


@pytest.mark.parametrize("in_values", [False, True])
@pytest.mark.parametrize("new,kv,hq,where,window", [(1, 100, 4, 50, 0), (10, 100, 4, 95, 0), (40, 100, 2, 70, 0), (150, 200, 4, 100, 0),
                                                    (1, 100, 4, 20, 30), (40, 100, 2, 40, 30), (150, 200, 4, 60, 20)])
def test_attention_nan(way, gpu, new, kv, hq, where, window, in_values):
    nan_case(gpu, new, kv, hq, where, in_values, window)


def test_attention_skips_tokens_that_the_table_does_not_have(way, gpu):
    rng = np.random.default_rng(24)
    cache, table = make_cache(rng, [200, 100], 32, 2, 64)
    table[0, 2], table[1, 0] = -1, 2 ** 30
    q = bf16(rng.standard_normal((30, 4, 64)))
    hold(attend(gpu, q, cache, table, [200, 100], [0, 10, 30]),
         kv8.attention_ref(q, cache, table, [200, 100], [0, 10, 30], 0.125))
    # lengths past the table's width count up to it: the first sequence then sees blank tokens, NaN all of them
    long = np.array([table.shape[1] * 32 + 50, 100])
    got = attend(gpu, q, cache, table, long, [0, 10, 30])
    want = kv8.attention_ref(q, cache, table, long, [0, 10, 30], 0.125)
    assert np.isnan(want[0][:10]).all() and np.isnan(got[0][:10]).all() and np.isnan(got[1][:10]).all()
    hold([x[10:] for x in got], [x[10:] for x in want])


def test_attention_strided_queries_and_other_stream(way, gpu):
    rng = np.random.default_rng(25)
    cache, table = make_cache(rng, [150, 40], 64, 2, 128)
    wide = bf16(rng.standard_normal((6, 8 + 5, 128)))
    cu = [0, 1, 6]
    want = kv8.attention_ref(wide[:, 2:10], cache, table, [150, 40], cu, 128 ** -0.5)
    out = torch.empty((6, 8, 128), dtype=torch.bfloat16, device=gpu)
    lse = torch.empty((6, 8), device=gpu)
    x, c = H.f32_to_device(wide, gpu).bfloat16(), to_device(cache, gpu)
    t, kv, sums = i32(table, gpu), i32([150, 40], gpu), i32(cu, gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.kv8_attention(x[:, 2:10], c, t, kv, sums, 5, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    hold((H.d_float(out), lse.cpu().numpy().astype(np.float64)), want)


def test_attention_many_prompts(gpu):
    # enough rows for the way of prompts to be chosen, lengths of all kinds
    rng = np.random.default_rng(29)
    new = [int(x) for x in rng.integers(0, 40, 64)]
    new[5] = 48
    kv = [n + int(x) for n, x in zip(new, rng.integers(0, 90, 64))]
    cache, table = make_cache(rng, kv, 32, 4, 64)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], 8, 64)))
    hold(attend(gpu, q, cache, table, kv, cu), kv8.attention_ref(q, cache, table, kv, cu, 0.125))


def test_attention_many_sequences(gpu):
    # more sequences than one pass of a workgroup over them takes, most of them short, some empty
    rng = np.random.default_rng(26)
    kv = list(rng.integers(0, 40, 600))
    kv[300] = 3000
    cache, table = make_cache(rng, [int(x) for x in kv], 16, 1, 64)
    q = bf16(rng.standard_normal((600, 2, 64)))
    cu = np.arange(601)
    hold(attend(gpu, q, cache, table, kv, cu), kv8.attention_ref(q, cache, table, kv, cu, 0.125))


def test_attention_past_four_gib(gpu):
    # a pool whose code arrays pass 4 GiB, with the sequence in its last blocks
    rng = np.random.default_rng(27)
    h, block, d = 8, 128, 256
    blocks = (1 << 32) // (h * block * d) + 6
    small, _ = make_cache(rng, [300], block, h, d)
    pool = dg.empty_kv8_cache(blocks, h, d, block, gpu)
    take = [blocks - 1, blocks - 3, blocks - 2]
    own, table = make_cache(rng, [300], block, h, d)
    for j, page in enumerate(take):
        for x, y in zip(pool, own):
            x[page] = torch.from_numpy(np.ascontiguousarray(y[table[0, j]])).to(gpu).view(x.dtype)
    q = bf16(rng.standard_normal((1, 16, d)))
    out = torch.empty((1, 16, d), dtype=torch.bfloat16, device=gpu)
    lse = torch.empty((1, 16), device=gpu)
    dg.kv8_attention(H.f32_to_device(q, gpu).bfloat16(), pool, i32([take], gpu), i32([300], gpu), i32([0, 1], gpu), 1, out, lse)
    hold((H.d_float(out), lse.cpu().numpy().astype(np.float64)),
         kv8.attention_ref(q, own, table, [300], [0, 1], d ** -0.5))
    k = bf16(rng.standard_normal((1, h, d)))
    dg.kv8_append(H.f32_to_device(k, gpu).bfloat16(), H.f32_to_device(k, gpu).bfloat16(), pool, i32([take], gpu),
                  i32([300], gpu), i32([0, 1], gpu), 1)
    want = kv8.append_ref(k, k, own, table, [300], [0, 1])
    last = table[0, 2]
    for x, y in zip(pool, want):
        got = x[take[2]].view(torch.uint8).cpu().numpy() if y.dtype == np.uint8 else x[take[2]].cpu().numpy()
        assert np.array_equal(got, y[last], equal_nan=y.dtype == np.float32)


def test_decode_loop_in_a_graph(gpu):
    # append + attention captured once, replayed as the sequences grow
    rng = np.random.default_rng(28)
    h, hq, d, block = 2, 8, 64, 16
    kv = [30, 3]
    steps = 40
    table, blocks = pages(rng, [x + steps for x in kv], block)
    cu0 = running(kv)
    before = kv8.append_ref(values(rng, (cu0[-1], h, d)), values(rng, (cu0[-1], h, d)), blank(blocks, h, block, d), table,
                            [0, 0], cu0)
    cache, t = to_device(before, gpu), i32(table, gpu)
    ctx, lens, cu = i32(kv, gpu), i32(kv, gpu), i32([0, 1, 2], gpu)
    x = torch.zeros((2, hq + 2 * h, d), dtype=torch.bfloat16, device=gpu)
    out, lse = torch.empty((2, hq, d), dtype=torch.bfloat16, device=gpu), torch.empty((2, hq), device=gpu)

    def step():
        lens.copy_(ctx + 1)
        dg.kv8_append(x[:, hq:hq + h], x[:, hq + h:], cache, t, ctx, cu, 1)
        dg.kv8_attention(x[:, :hq], cache, t, lens, cu, 1, out, lse)
        ctx.copy_(lens)

    side = torch.cuda.Stream()
    dg.reserve_workspace(dg.kv8_attention_workspace_size(d), side)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    want = before
    for i in range(steps):
        wide = values(rng, (2, hq + 2 * h, d), 2)
        x.copy_(H.f32_to_device(wide, gpu))
        graph.replay()
        torch.cuda.synchronize()
        now = [a + i for a in kv]
        want = kv8.append_ref(wide[:, hq:hq + h], wide[:, hq + h:], want, table, now, [0, 1, 2])
        if i % 8 == 0 or i == steps - 1:
            same_cache(cache, want)
            hold((H.d_float(out), lse.cpu().numpy().astype(np.float64)),
                 kv8.attention_ref(wide[:, :hq], want, table, [a + 1 for a in now], [0, 1, 2], d ** -0.5))


def test_capture_needs_a_reserved_workspace(gpu):
    rng = np.random.default_rng(30)
    cache, table = make_cache(rng, [200], 32, 1, 64)
    q = H.f32_to_device(bf16(rng.standard_normal((1, 4, 64))), gpu).bfloat16()
    out, c, t, kv, cu = torch.empty_like(q), to_device(cache, gpu), i32(table, gpu), i32([200], gpu), i32([0, 1], gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with pytest.raises(dg.DGError) as refused:
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            dg.kv8_attention(q, c, t, kv, cu, 1, out)
    assert refused.value.status == 7
    torch.cuda.synchronize()


def test_binding_refuses(gpu):
    cache = dg.empty_kv8_cache(4, 2, 64, 16, gpu)
    t, lens, cu = i32([[0, 1]], gpu), i32([3], gpu), i32([0, 1], gpu)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=gpu)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=gpu)
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        dg.kv8_append(x, x, (cache[0], cache[0], cache[2], cache[3]), t, lens, cu, 1)     # values not turned
    with pytest.raises(ValueError):
        dg.kv8_append(x, x[:, :1], cache, t, lens, cu, 1)
    with pytest.raises(TypeError):
        dg.kv8_append(x.float(), x, cache, t, lens, cu, 1)
    with pytest.raises(ValueError):
        dg.kv8_append(x, x, cache, t, lens, i32([0, 1, 1], gpu), 1)
    with pytest.raises(ValueError):
        dg.kv8_attention(q, cache, t, lens, cu, 1, out[:, :2].contiguous())
    with pytest.raises(ValueError):
        dg.kv8_attention(q.transpose(0, 1), cache, t, lens, cu, 1, out)
    with pytest.raises(TypeError):
        dg.kv8_attention(q, cache, t.long(), lens, cu, 1, out)
    with pytest.raises(dg.DGError):
        dg.kv8_attention(q[:, :3].contiguous(), cache, t, lens, cu, 1, out[:, :3].contiguous())    # 3 heads over 2
    with pytest.raises(dg.DGError):
        dg.kv8_attention(q, cache, t, lens, cu, 1, out, window=4, causal=False)
    with pytest.raises(dg.DGError):
        dg.kv8_attention(q, cache, t, lens, cu, -1, out)
    odd = dg.empty_kv8_cache(4, 2, 96, 16, gpu)
    y = torch.zeros((1, 2, 96), dtype=torch.bfloat16, device=gpu)
    with pytest.raises(dg.DGError):
        dg.kv8_append(y, y, odd, t, lens, cu, 1)
    # nothing to do: nothing is touched
    none = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=gpu)
    assert dg.kv8_attention(none, cache, t, lens, i32([0, 0], gpu), 0, none.clone()).shape == (0, 4, 64)
