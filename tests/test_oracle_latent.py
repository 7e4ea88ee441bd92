"""The oracle of latent attention, pinned by hand-made cases and by rules that
any right implementation keeps (CPU)."""

import numpy as np
import pytest

from oracle import e4m3, kv8
from oracle import latent as R


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_by_hand(interleaved):
    # pairs as complex numbers times e^(i angle); a quarter turn takes (a, b) to (-b, a)
    rng = np.random.default_rng(1)
    x, t = rng.standard_normal((5, 3, 32)), rng.uniform(-9, 9, (5, 16))
    angles = np.concatenate((np.cos(t), np.sin(t)), 1)
    y = R.rotate(x, angles[:, None], interleaved)
    pairs = (lambda v: v[..., 0::2] + 1j * v[..., 1::2]) if interleaved else (lambda v: v[..., :16] + 1j * v[..., 16:])
    assert np.allclose(pairs(y), pairs(x) * np.exp(1j * t)[:, None], rtol=0, atol=1e-14)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    one = R.rotate(np.arange(4.0), np.array([0, 0, 1.0, 1.0]), interleaved)
    assert list(one) == ([-1, 0, -3, 2] if interleaved else [-2, -3, 0, 1])


def test_scores_depend_on_the_distance_alone():
    # q at position i against r at j: the product after both rotations is that at i - j and 0
    rng = np.random.default_rng(2)
    q, r = rng.standard_normal((2, 64))
    f = 10000.0 ** (-np.arange(32) / 32)
    at = lambda p: np.concatenate((np.cos(p * f), np.sin(p * f)))  # noqa: E731
    for i, j in ((5, 3), (1000, 990), (70000, 69999)):
        assert np.isclose(R.rotate(q, at(i), True) @ R.rotate(r, at(j), True), R.rotate(q, at(i - j), True) @ r, atol=1e-9)


def test_norm():
    c = np.array([[3.0, 4.0] * 64, [0.0] * 128])
    y = R.normalise(c, np.full(128, 2.0), 0.5)
    assert np.allclose(y[0, :2], [6 / np.sqrt(13), 8 / np.sqrt(13)]) and np.all(y[1] == 0)


def test_quantise():
    y = np.zeros(256)
    y[0], y[1], y[128] = 448.0, -1.0, 1e-30
    codes, s = R.quantise(y)
    assert list(s) == [1.0, 2.0 ** -22] and e4m3.decode(codes)[:2].tolist() == [448.0, -1.0] and not e4m3.decode(codes)[128:].any()
    x = np.random.default_rng(3).standard_normal(512) * 2.0 ** np.arange(-2, 2).repeat(128)
    codes, s = R.quantise(x)
    back = e4m3.decode(codes) * s.repeat(128)
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s.repeat(128))).all()
    assert all(s[i] == kv8.pow2_scale(np.abs(x[128 * i:128 * i + 128]).max()) for i in range(4))


def caches(rng, n, block, L):
    blocks = -(-n // block) + 1
    table = rng.permutation(blocks)[None, :-1].astype(np.int32)
    return (np.full((blocks, block, L), np.nan), np.full((blocks, block, L // 8), np.nan), None), table


def test_append_token_by_token_equals_at_once():
    rng = np.random.default_rng(4)
    n, L, block = 37, 256, 16
    c, r, an = rng.standard_normal((n, L)), rng.standard_normal((n, 32)), rng.standard_normal((n, 32))
    empty, table = caches(rng, n, block, L)
    once, _ = R.append_ref(c, r, empty, table, [0], [0, n], an)
    step = empty
    for i in range(n):
        step, q = R.append_ref(c[i:i + 1], r[i:i + 1], step, table, [i], [0, 1], an, q=r[i:i + 1, None])
        assert np.array_equal(q[0, 0], R.rotate(r[i], an[i], True))
    for x, y in zip(once[:2], step[:2]):
        assert np.array_equal(x, y, equal_nan=True)
    got, ropes, there = R.tokens_of(once, table, 0, 5, n - 5)
    assert there.all() and np.array_equal(got, c[5:]) and np.array_equal(ropes, R.rotate(r, an, True)[5:])


@pytest.mark.parametrize("causal", [True, False])
def test_absorbed_equals_expanded(causal):
    # the same layer both ways: scores through the up-projection's key weights on the query's side or the token's
    rng = np.random.default_rng(5)
    m, n, heads, L, D = 40, 7, 3, 256, 64
    empty, table = caches(rng, m, 16, L)
    c, r = rng.standard_normal((m, L)), rng.standard_normal((m, L // 8))
    cache, _ = R.append_ref(c, r, empty, table, [0], [0, m], np.concatenate((np.ones((m, 16)), np.zeros((m, 16))), 1))
    wk, wv = rng.standard_normal((2, heads, D, L)) * L ** -0.5
    q, qr = rng.standard_normal((n, heads, D)), rng.standard_normal((n, heads, L // 8))
    out, _, lse = R.attention_ref(np.einsum("nhd,hdl->nhl", q, wk), qr, cache, table, [m], [0, n], 0.1, causal)
    kv = np.concatenate((np.einsum("ml,hdl->mhd", c, wk), np.einsum("ml,hdl->mhd", c, wv)), 2)
    out2, _, lse2 = R.expanded_ref(np.concatenate((q, qr), 2), kv, r, [0, n], [0, m], 0.1, causal)
    assert np.allclose(np.einsum("nhl,hdl->nhd", out, wv), out2) and np.allclose(lse, lse2)


def test_rows_that_see_nothing_and_equal_scores():
    rng = np.random.default_rng(6)
    empty, table = caches(rng, 20, 16, 256)
    c = rng.standard_normal((20, 256))
    cache, _ = R.append_ref(c, np.zeros((20, 32)), empty, table, [0], [0, 20], np.zeros((20, 32)))
    out, size, lse = R.attention_ref(np.zeros((23, 1, 256)), np.zeros((23, 1, 32)), cache, table, [20], [0, 23], 1.0)
    assert not out[:3].any() and np.isneginf(lse[:3]).all()
    for i in range(20):
        assert np.allclose(out[3 + i, 0], c[:i + 1].mean(0)) and np.isclose(lse[3 + i, 0], np.log(i + 1))
        assert np.allclose(size[3 + i, 0], np.abs(c[:i + 1]).mean(0))
    table[0, 1] = 99                                                         # tokens 16 .. 19 are nobody's
    out, _, lse = R.attention_ref(np.zeros((1, 1, 256)), np.zeros((1, 1, 32)), cache, table, [20], [0, 1], 1.0)
    assert np.allclose(out[0, 0], c[:16].mean(0)) and np.isclose(lse[0, 0], np.log(16))


def test_places_before_the_first_token():
    rng = np.random.default_rng(7)
    empty, table = caches(rng, 20, 16, 256)
    c, r, an = rng.standard_normal((6, 256)), rng.standard_normal((6, 32)), rng.standard_normal((9, 32))
    cache, q = R.append_ref(c, r, empty, table, [-4], [0, 6], an, q=r[:, None])
    want, _ = R.append_ref(c[4:], r[4:], empty, table, [0], [0, 2], an)
    assert np.array_equal(cache[0], want[0], equal_nan=True) and np.array_equal(cache[1], want[1], equal_nan=True)
    assert np.isnan(q[:4]).all() and np.isfinite(q[4:]).all()
    got, _, there = R.tokens_of(cache, table, 0, -3, 5)
    assert there.tolist() == [False] * 3 + [True] * 2 and np.array_equal(got[3:], c[4:])
