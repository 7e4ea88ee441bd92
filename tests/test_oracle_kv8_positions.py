"""Where queries stand in the oracle's attention: by the sequence's length, also
past the tokens that its block table has room for (CPU)."""

import numpy as np
import pytest

from oracle import kv8


@pytest.mark.parametrize("window,seen", [(0, [28, 29, 30, 31, 32, 32, 32]), (5, [5, 5, 5, 5, 5, 4, 3])])
def test_lengths_past_the_table(window, seen):
    # two blocks of 16, 34 tokens, 7 queries: they stand at 27 .. 33 and see what lies below 32
    k = np.zeros((32, 1, 64), np.float32)
    v = np.random.default_rng(1).standard_normal((32, 1, 64)).astype(np.float32)
    empty = (np.full((2, 1, 16, 64), 0x7F, np.uint8), np.full((2, 1, 64, 16), 0x7F, np.uint8),
             np.full((2, 1), np.nan, np.float32), np.full((2, 1), np.nan, np.float32))
    table = np.array([[1, 0]])
    cache = kv8.append_ref(k, v, empty, table, [0], [0, 32])
    _, vals, _ = kv8.gather(cache, table, 0, 0, 32)
    out, lse = kv8.attention_ref(np.ones((7, 1, 64)), cache, table, [34], [0, 7], 1.0, window=window)
    for i, n in enumerate(seen):
        hi = min(27 + i + 1, 32)
        assert np.allclose(out[i, 0], vals[hi - n:hi].mean(0)) and np.isclose(lse[i, 0], np.log(n))


def test_a_window_past_the_table():
    cache = (np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1, 64, 16), np.uint8), np.ones((1, 1)), np.ones((1, 1)))
    out, lse = kv8.attention_ref(np.ones((1, 1, 64)), cache, np.array([[0]]), [40], [0, 1], 1.0, window=3)
    assert np.all(out == 0) and np.all(np.isneginf(lse))
