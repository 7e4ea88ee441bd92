"""Attention over the 8-bit cache where the second product's operand needs its
whole range: blocks of far apart value scales, and a token that takes nearly
all of a row's weight but holds zeros.  Every output element is held by
itself, not against the largest of its row.

An element sum_j w[j] v[j] (w the softmax weights) may be off by

  2^-8 |r|                          its own rounding to bf16 (half an ulp is 2^-9)
  (2 x + 2^-11) sum_j w[j] |v[j]|   scores off by x, and so w by that much twice (l has
                                    it too); w as fp16 or two bf16 pieces, 2^-12 or less,
                                    and fp32 sums
  2^-32 f max(w) sum_j |v[j]|       weights that fp16 holds below its normal range, to
                                    steps of 2^-31 of the largest w times value scale;
                                    f is how far value scales lie apart, 2^4 at most

with x = (d + 8) 2^-24 max_j scale |q| . |k[j]|, an fp32 sum of d products and
a few roundings.
"""

import numpy as np
import pytest

from oracle import kv8
from tests.test_gpu_kv8 import attend, bf16, blank, make_cache, pages, running, way  # noqa: F401

pytestmark = pytest.mark.gpu


def hold_each(got, q, cache, table, kv, cu, scale):
    d, hq, h = q.shape[2], q.shape[1], cache[0].shape[1]
    want, sums = kv8.attention_ref(q, cache, table, kv, cu, scale)
    worst = 0.0
    for seq in range(len(kv)):
        n = int(cu[seq + 1] - cu[seq])
        for head in range(hq):
            keys, vals, _ = kv8.gather(cache, table, seq, head * h // hq, kv[seq])
            vs = cache[3][table[seq, :-(-kv[seq] // cache[0].shape[2])], head * h // hq]
            apart = min(float(vs.max() / vs.min()), 16.0)
            for i in range(n):
                at, see = cu[seq] + i, kv[seq] - n + i + 1
                row = q[at, head].astype(np.float64)
                x = (d + 8) * 2.0 ** -24 * scale * float((np.abs(keys[:see]) @ np.abs(row)).max())
                w = np.exp(scale * (keys[:see] @ row) - sums[at, head])
                size = np.abs(vals[:see])
                bound = (2.0 ** -8 * np.abs(want[at, head]) + (2 * x + 2.0 ** -11) * (w @ size)
                         + 2.0 ** -32 * apart * w.max() * size.sum(0))
                worst = max(worst, float((np.abs(got[0][at, head] - want[at, head]) / np.maximum(bound, 1e-300)).max()))
                assert abs(got[1][at, head] - sums[at, head]) <= x + 1e-6 * abs(sums[at, head]) + 1e-6, (at, head)
    assert worst <= 1, worst


@pytest.mark.parametrize("block,hq,h,d,new,kv", [(64, 4, 2, 64, [1], [400]), (16, 4, 1, 128, [1, 3], [300, 150]),
                                                 (32, 2, 2, 64, [140], [260]), (16, 2, 1, 256, [70], [330])])
@pytest.mark.parametrize("apart", [3, 12, 16, 20, 24, 30, 60, -20])
def test_a_scale_far_from_the_others(way, gpu, block, hq, h, d, new, kv, apart):  # noqa: F811
    print(f"[case] scales 2^{apart} apart, block {block} heads {hq}/{h} d {d} {new} {kv}", flush=True)
    rng = np.random.default_rng(apart + 100)
    cache, table = make_cache(rng, kv, block, h, d)
    cache[3][np.isfinite(cache[3])] = 2.0 ** -6
    # one block in the middle and one that holds the last token: a single outlier, and nothing else that a code could show
    for seq, n in enumerate(kv):
        for j in (1, n // 64 * 64 // block - 1):
            page = table[seq, j]
            cache[1][page] = 0
            cache[1][page, :, 5, 3] = 0x7E          # 448
            cache[3][page] = 2.0 ** (apart - 6)
    cu = running(new)
    q = bf16(rng.standard_normal((cu[-1], hq, d)))
    hold_each(attend(gpu, q, cache, table, kv, cu), q, cache, table, kv, cu, d ** -0.5)


@pytest.mark.parametrize("log2w", [10, 18, 24])
@pytest.mark.parametrize("new,kv", [(1, 900), (130, 500)])
def test_a_token_of_most_weight_and_no_values(way, gpu, new, kv, log2w):  # noqa: F811
    h, d, block = 1, 64, 32
    rng = np.random.default_rng(log2w)
    k = bf16(rng.standard_normal((kv, h, d)) * 0.25)
    k[0] = 0
    k[0, 0, 7] = log2w
    v = bf16(rng.standard_normal((kv, h, d)))
    v[0] = 0
    table, blocks = pages(rng, [kv], block)
    cache = kv8.append_ref(k, v, blank(blocks, h, block, d), table, [0], [0, kv])
    q = rng.standard_normal((new, 2, d))
    q[..., 7] = np.log(2)
    q = bf16(q)
    hold_each(attend(gpu, q, cache, table, [kv], [0, new], scale=1.0), q, cache, table, [kv], [0, new], 1.0)


@pytest.mark.parametrize("new,kv", [(1, 700), (12, 300), (150, 400)])
def test_blocks_of_zeros_beside_large_and_small_values(way, gpu, new, kv):  # noqa: F811
    # scales as the append gives them: 2^-22 for blocks of zeros, and values of 2^-12, 1 and 2^10 in blocks of their own
    h, d, block = 1, 64, 64
    rng = np.random.default_rng(kv)
    k, v = bf16(rng.standard_normal((kv, h, d))), rng.standard_normal((kv, h, d))
    v *= np.array([1.0, 0.0, 2.0 ** 10, 2.0 ** -12])[np.arange(kv) // block % 4][:, None, None]
    v[np.arange(kv) // block % 4 == 2, :, 1:] = 0
    table, blocks = pages(rng, [kv], block)
    cache = kv8.append_ref(k, bf16(v), blank(blocks, h, block, d), table, [0], [0, kv])
    q = bf16(rng.standard_normal((new, 4, d)))
    hold_each(attend(gpu, q, cache, table, [kv], [0, new]), q, cache, table, [kv], [0, new], 0.125)
