"""Every compiled form of the cache's append, and non-causal attention at every
head dimension, against the oracle; tolerances as in test_gpu_kv8."""

import numpy as np
import pytest

import fp8_block_scaled_nt_amd as dg
from oracle import kv8
from tests import gpu_harness as H
from tests.test_gpu_kv8 import (attend, bf16, blank, hold, i32, make_cache, pages, running, same_cache, to_device, values,  # noqa: F401
                                way)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
# a wave's form: up to 4 tokens, over two groups of 4 positions, over two blocks; a workgroup's: parts of blocks and whole ones
@pytest.mark.parametrize("ctx,new", [([3, 14, 0, 130], [4, 4, 2, 3]), ([5, 0, 127], [300, 5, 41])])
def test_append(gpu, block, d, ctx, new):
    print(f"[case] append block {block} d {d} {ctx} {new}", flush=True)
    rng = np.random.default_rng(block + d)
    h = 2
    table, blocks = pages(rng, [a + b for a, b in zip(ctx, new)], block)
    cu0, cu = running(ctx), running(new)
    before = kv8.append_ref(values(rng, (cu0[-1], h, d)), values(rng, (cu0[-1], h, d)), blank(blocks, h, block, d), table,
                            [0] * len(ctx), cu0)
    k, v = values(rng, (cu[-1], h, d)), values(rng, (cu[-1], h, d))
    cache = to_device(before, gpu)
    dg.kv8_append(H.f32_to_device(k, gpu).bfloat16(), H.f32_to_device(v, gpu).bfloat16(), cache, i32(table, gpu), i32(ctx, gpu),
                  i32(cu, gpu), max(new))
    same_cache(cache, kv8.append_ref(k, v, before, table, ctx, cu))


@pytest.mark.parametrize("block,hq,h,d,new,kv", [(16, 4, 2, 64, [1, 50], [100, 75]), (64, 8, 2, 128, [1, 1], [300, 64]),
                                                 (32, 4, 2, 128, [70, 3], [200, 1]), (128, 4, 1, 256, [1, 2], [257, 40]),
                                                 (64, 2, 2, 256, [90], [130])])
def test_attention_not_causal(way, gpu, block, hq, h, d, new, kv):  # noqa: F811
    print(f"[case] not causal block {block} heads {hq}/{h} d {d} {new} {kv}", flush=True)
    rng = np.random.default_rng(block + d)
    cache, table = make_cache(rng, kv, block, h, d)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], hq, d)))
    hold(attend(gpu, q, cache, table, kv, cu, causal=False),
         kv8.attention_ref(q, cache, table, kv, cu, d ** -0.5, causal=False))
