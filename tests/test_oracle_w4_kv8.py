"""The oracles of the 4-bit weights and the 8-bit key/value cache, pinned by
hand-made cases and by rules that any right implementation keeps (CPU)."""

import numpy as np
import pytest

import oracle
from oracle import e4m3, kv8


def test_w4_e2m1_on_the_grid_is_exact():
    # a group whose largest value is 6 s with s a bf16 value holds every e2m1 value exactly
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -1.5, -2, -3, -4, -6, 0], np.float32)
    x = np.tile(grid, 4)[None, :] * np.float32(0.25)
    codes, s, z = oracle.quantize_w4(x, "e2m1", 32)
    assert z is None and np.all(s == 0.25) and codes.shape == (1, 32)
    assert np.array_equal(oracle.dequantize_w4(codes, s, z), x.astype(np.float64))


def test_w4_u4_by_hand():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [-3.0, 12.0, 0.4, 0.6]          # lo -3, hi 12, s = 1, z = 3
    codes, s, z = oracle.quantize_w4(x, "u4", 32)
    assert s[0, 0] == 1.0 and z[0, 0] == 3
    w = oracle.dequantize_w4(codes, s, z)
    assert list(w[0, :5]) == [-3.0, 12.0, 0.0, 1.0, 0.0]
    # all positive: the zero point is 0 and zero stays representable
    codes, s, z = oracle.quantize_w4(np.full((2, 64), 7.5, np.float32), "u4", 64)
    assert np.all(z == 0) and np.all(s == 0.5) and np.all(codes == 0xFF)


@pytest.mark.parametrize("fmt,group", [("e2m1", 32), ("u4", 64), ("u4", 128)])
def test_w4_error_is_within_a_step(fmt, group):
    x = np.random.default_rng(3).standard_normal((5, 256)).astype(np.float32)
    codes, s, z = oracle.quantize_w4(x, fmt, group)
    err = np.abs(oracle.dequantize_w4(codes, s, z) - x).reshape(5, -1, group)
    # e2m1: half of the widest step (2); u4: rounding of x and of the zero point, half a step each
    assert np.all(err <= (1.0 + 0.05) * s[..., None])
    a = np.random.default_rng(4).standard_normal((3, 256))
    loop = [[sum(a[i, j] * oracle.dequantize_w4(codes, s, z)[r, j] for j in range(256)) for r in range(5)] for i in range(3)]
    assert np.allclose(oracle.w4_gemm_ref(a, codes, s, z), loop, rtol=1e-12)


def empty_cache(blocks, h, block, d):
    return (np.full((blocks, h, block, d), 0x7F, np.uint8), np.full((blocks, h, d, block), 0x7F, np.uint8),
            np.full((blocks, h), np.nan, np.float32), np.full((blocks, h), np.nan, np.float32))


@pytest.mark.parametrize("amax,s", [(448.0, 1.0), (448.1, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7),
                                    (0.0, 2.0 ** -22)])
def test_pow2_scale(amax, s):
    assert kv8.pow2_scale(amax) == s


def test_append_token_by_token_equals_at_once_above_the_smallest_normal():
    rng = np.random.default_rng(5)
    # values whose codes stay normal in every scale that the block passes through
    k = (rng.uniform(1, 2, (40, 2, 64)) * np.where(rng.random((40, 2, 64)) < 0.5, -1, 1)).astype(np.float32)
    k *= np.float32(2.0) ** (np.arange(40) % 5)[:, None, None]
    v = k[:, ::-1].copy()
    table = np.array([[2, 0, 1]])
    at_once = kv8.append_ref(k, v, empty_cache(3, 2, 16, 64), table, [0], [0, 40])
    c = empty_cache(3, 2, 16, 64)
    for i in range(40):
        c = kv8.append_ref(k[i:i + 1], v[i:i + 1], c, table, [i], [0, 1])
    for x, y in zip(at_once, c):
        assert np.array_equal(x, y, equal_nan=x.dtype == np.float32)
    keys, vals, there = kv8.gather(at_once, table, 0, 1, 40)
    assert there.all() and np.all(np.abs(keys - k[:, 1]) <= np.abs(k[:, 1]) / 16 + 1e-12)
    assert np.all(np.abs(vals - v[:, 1]) <= np.abs(v[:, 1]) / 16 + 1e-12)


def test_append_leaves_the_rest_alone():
    k = np.ones((3, 1, 64), np.float32)
    before = empty_cache(2, 1, 16, 64)
    after = kv8.append_ref(k, k, before, np.array([[1], [-1]]), [0, 0], [0, 2, 3])
    assert np.array_equal(after[0][0], before[0][0]) and np.all(after[0][1, 0, 2:] == 0x7F)
    assert np.all(after[1][1, 0, :, 2:] == 0x7F) and np.all(after[1][1, 0, :, :2] != 0x7F)


def test_append_non_finite():
    k = np.zeros((2, 1, 64), np.float32)
    k[0, 0, :3] = [np.inf, -np.inf, np.nan]
    k[1, 0, 0] = 448.0
    c = kv8.append_ref(k, k, empty_cache(1, 1, 16, 64), np.array([[0]]), [0], [0, 2])
    assert c[2][0, 0] == 1.0 and list(c[0][0, 0, 0, :3]) == [0x7E, 0xFE, 0x7F] and c[0][0, 0, 1, 0] == 0x7E


def test_attention_of_equal_scores_is_the_mean():
    rng = np.random.default_rng(6)
    v = rng.standard_normal((20, 1, 64)).astype(np.float32)
    c = kv8.append_ref(np.zeros_like(v), v, empty_cache(2, 1, 16, 64), np.array([[0, 1]]), [0], [0, 20])
    q = rng.standard_normal((4, 2, 64))
    out, lse = kv8.attention_ref(q, c, np.array([[0, 1]]), [20], [0, 4], 0.125)
    _, vals, _ = kv8.gather(c, np.array([[0, 1]]), 0, 0, 20)
    for i in range(4):
        assert np.allclose(out[i], vals[:17 + i].mean(0)) and np.allclose(lse[i], np.log(17 + i))
    out, lse = kv8.attention_ref(q, c, np.array([[0, 1]]), [20], [0, 4], 0.125, window=3)
    assert np.allclose(out[3], vals[17:20].mean(0)) and np.allclose(lse, np.log(3))
    out, lse = kv8.attention_ref(q, c, np.array([[0, 1]]), [20], [0, 4], 0.125, causal=False)
    assert np.allclose(out, vals.mean(0)) and np.allclose(lse, np.log(20))


def test_attention_rows_without_keys():
    c = empty_cache(1, 1, 16, 64)
    q = np.ones((3, 1, 64))
    # no tokens at all, and more queries than tokens
    out, lse = kv8.attention_ref(q, c, np.array([[0]]), [0], [0, 3], 1.0)
    assert np.all(out == 0) and np.all(lse == -np.inf)
    c = kv8.append_ref(np.ones((1, 1, 64)), np.ones((1, 1, 64)), c, np.array([[0]]), [0], [0, 1])
    out, lse = kv8.attention_ref(q, c, np.array([[0]]), [1], [0, 3], 1.0)
    assert np.all(out[:2] == 0) and np.all(out[2] == 1) and np.all(np.isinf(lse[:2])) and np.isfinite(lse[2])


def test_decode_is_the_inverse_of_gather():
    c = empty_cache(2, 1, 16, 64)
    c[0][:], c[1][:] = 0x38, 0x40               # 1.0 and 2.0
    c[2][:], c[3][:] = 0.5, 4.0
    keys, vals, _ = kv8.gather(c, np.array([[1, 0]]), 0, 0, 17)
    assert np.all(keys == 0.5) and np.all(vals == 8.0) and keys.shape == (17, 64)
    assert e4m3.decode(np.uint8(0x38)) == 1.0
