"""Prompts and single tokens in one attention call: each sequence is right
whichever way it goes, and long sequences do not wait behind a prompt's way of
walking their keys."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import kv8
from tests.test_gpu_kv8 import attend, bf16, hold, i32, make_cache, running

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h,d,new,kv", [
    # enough packed rows for the way of prompts: prompts, single tokens, one of just too few and one of just enough rows, empty ones
    (8, 64, [130] * 12 + [1] * 16 + [0, 70, 31, 32, 1], [150] * 12 + [int(x) for x in range(1, 400, 25)] + [90, 70, 200, 200, 0]),
    (8, 256, [3, 70, 70, 0, 1, 5] + [64] * 10, [300, 70, 90, 10, 500, 2] + [100] * 10),
])
def test_prompts_among_single_tokens(gpu, h, d, new, kv):
    print(f"[case] mixed batch h {h} d {d} {new}", flush=True)
    rng = np.random.default_rng(51)
    cache, table = make_cache(rng, kv, 32, h, d)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], 2 * h, d)))
    want = kv8.attention_ref(q, cache, table, kv, cu, d ** -0.5)
    got = attend(gpu, q, cache, table, kv, cu)
    hold(got, want)
    again = attend(gpu, q, cache, table, kv, cu)
    assert np.array_equal(got[0], again[0]) and np.array_equal(got[1], again[1])


def test_long_sequences_beside_a_prompt(gpu):
    # 8 single tokens of 65536 beside a prompt of 2048 take 3 times as long as the two alone at the very most (walked by one
    # workgroup a head each they took 6 times as long)
    h, hq, d, block, tokens = 8, 32, 128, 64, 65536
    per = tokens // block
    torch.manual_seed(5)
    blocks = 8 * per + 2048 // block
    cache = (torch.randint(0, 0x60, (blocks, h, block, d), dtype=torch.uint8, device=gpu),
             torch.randint(0, 0x60, (blocks, h, d, block), dtype=torch.uint8, device=gpu),
             torch.full((blocks, h), 2.0 ** -8, device=gpu), torch.full((blocks, h), 2.0 ** -8, device=gpu))
    table = torch.arange(9 * per, dtype=torch.int32, device=gpu).view(9, per)

    def us(new, kv, rows):
        cu, most = running(new), max(new)
        q = torch.randn((int(cu[-1]), hq, d), device=gpu).bfloat16()
        out, t = torch.empty_like(q), table[rows].contiguous()
        kv, cu = i32(kv, gpu), i32(cu, gpu)
        times = []
        for _ in range(5):
            start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(3):
                dg.kv8_attention(q, cache, t, kv, cu, most, out)
            stop.record()
            stop.synchronize()
            times.append(start.elapsed_time(stop) / 3 * 1e3)
        return min(times)

    single, prompt = us([1] * 8, [tokens] * 8, slice(0, 8)), us([2048], [2048], slice(8, 9))
    both = us([1] * 8 + [2048], [tokens] * 8 + [2048], slice(0, 9))
    print(f"single tokens {single:.0f} us, prompt {prompt:.0f} us, together {both:.0f} us", flush=True)
    assert both < 3 * (single + prompt)
