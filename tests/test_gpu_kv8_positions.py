"""Where queries stand: by the sequence's length and its number of queries,
also where the block table has no room for all tokens, or max_q says less than
there are.  Held to the definition written out here, on top of the oracle's."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import kv8
from tests import gpu_harness as H
from tests.test_gpu_kv8 import attend, bf16, hold, i32, make_cache, running, to_device, way  # noqa: F401

pytestmark = pytest.mark.gpu


def by_definition(q, cache, table, kv_lens, cu, scale, window):
    """Causal; query i of n at kv_len - n + i sees the tokens in the table up to there, the last `window` of them by position."""
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    h = cache[0].shape[1]
    room = table.shape[1] * cache[0].shape[2]
    for seq in range(len(kv_lens)):
        n = cu[seq + 1] - cu[seq]
        for head in range(q.shape[1]):
            keys, vals, there = kv8.gather(cache, table, seq, head * h // q.shape[1], min(kv_lens[seq], room))
            for i in range(n):
                pos = kv_lens[seq] - n + i
                j = np.arange(len(there))
                see = there & (j <= pos) & ((j > pos - window) if window else True)
                if see.any():
                    x = scale * keys[see] @ q[cu[seq] + i, head].astype(np.float64)
                    p = np.exp(x - x.max())
                    out[cu[seq] + i, head] = p @ vals[see] / p.sum()
                    lse[cu[seq] + i, head] = x.max() + np.log(p.sum())
    return out, lse


@pytest.mark.parametrize("window", [0, 20, 64])
@pytest.mark.parametrize("block,hq,h,d,new,over", [(16, 4, 2, 64, [9, 3], [5, 60]), (64, 2, 1, 128, [100], [70]), (32, 2, 2, 64, [1, 40], [1, 200]),
                                                   (64, 2, 2, 256, [30], [10])])
def test_lengths_past_the_table(way, gpu, block, hq, h, d, new, over, window):  # noqa: F811
    print(f"[case] {over} tokens past the table, block {block} heads {hq}/{h} d {d} {new} window {window}", flush=True)
    rng = np.random.default_rng(41)
    room = 3 * block
    cache, table = make_cache(rng, [room] * len(new), block, h, d)
    kv, cu = [room + x for x in over], running(new)
    q = bf16(rng.standard_normal((cu[-1], hq, d)))
    got = attend(gpu, q, cache, table, kv, cu, window=window)
    hold(got, by_definition(q, cache, table, kv, cu, d ** -0.5, window))
    hold(got, kv8.attention_ref(q, cache, table, kv, cu, d ** -0.5, window=window))


@pytest.mark.parametrize("window", [0, 11])
def test_rows_past_max_q_are_ignored(way, gpu, window):  # noqa: F811
    rng = np.random.default_rng(42)
    kv, new, most = [90, 200], [40, 3], 25
    cache, table = make_cache(rng, kv, 32, 2, 64)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], 4, 64)))
    out = torch.full((cu[-1], 4, 64), 7.0, dtype=torch.bfloat16, device=gpu)
    lse = torch.full((cu[-1], 4), 7.0, device=gpu)
    dg.kv8_attention(H.f32_to_device(q, gpu).bfloat16(), to_device(cache, gpu), i32(table, gpu), i32(kv, gpu), i32(cu, gpu), most,
                     out, lse, window=window)
    want = by_definition(q, cache, table, kv, cu, 0.125, window)
    got = H.d_float(out), lse.cpu().numpy().astype(np.float64)
    here = np.r_[0:most, new[0]:cu[-1]]
    hold([x[here] for x in got], [x[here] for x in want])
    assert np.all(got[0][most:new[0]] == 7.0) and np.all(got[1][most:new[0]] == 7.0)
