"""Infinite latents under absorbed attention: a row that sees one takes from it
what the definition says, in a step with masks as in one that every row sees
wholly (bounds as derived in test_gpu_latent)."""

import numpy as np
import pytest

from oracle import latent as R
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import running
from tests.test_gpu_latent_forms import attend, queries, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [np.inf, -np.inf])
@pytest.mark.parametrize("L,block", [(512, 64), (256, 16)])
@pytest.mark.parametrize("at", [3, 70, 127, 128, 129, 131])
def test_a_score_of_minus_infinity_keeps_the_infinite_channel(rows, gpu, what, L, block, at):  # noqa: F811
    # where q is of the other sign the token's weight is 0, and 0 times infinity
    # makes that channel of the row NaN and leaves the others; else the whole row
    print(f"[case] infinite latent {rows} {what} {L} {at}", flush=True)
    rng = np.random.default_rng(at)
    cache, table = T.filled(rng, [132], block, L, False)
    cache[0][table[0, at // block], at % block, [5, L - 2]] = what, 1.0
    q, qr = queries(rng, 4, 20, L)
    q[..., 5] = np.where(np.abs(q[..., 5]) < 0.1, 1.0, q[..., 5])
    out, lse = attend(gpu, q, qr, cache, table, [132], [0, 4])
    with np.errstate(invalid="ignore"):
        want = R.attention_ref(q, qr, cache, table, [132], [0, 4], (L * 3 / 8) ** -0.5)
    seen = np.arange(4) + 128 >= at
    hidden = seen[:, None] & (np.sign(q[..., 5]) != np.sign(what))
    assert hidden.any() and np.isnan(want[0][hidden][:, 5]).all() and np.isfinite(want[2][hidden]).all()
    T.check_out(out, lse, want)


@pytest.mark.parametrize("L", [256, 512])
def test_infinities_of_several_tokens_and_sequences(rows, gpu, L):  # noqa: F811
    # in both halves of a step, in channels of every wave, and in a step that a longer sequence sees wholly
    rng = np.random.default_rng(L)
    lens, new = [60, 150, 64], [2, 3, 1]
    cache, table = T.filled(rng, lens, 32, L, False)
    for seq, at, channel, what in ((0, 2, 7, np.inf), (0, 40, L // 4 + 1, -np.inf), (1, 20, L // 2 + 3, np.inf), (1, 135, L - 1, np.inf),
                                   (1, 149, 0, -np.inf), (2, 63, 9, np.inf)):
        cache[0][table[seq, at // 32], at % 32, channel] = what
    q, qr = queries(rng, sum(new), 9, L)
    # the signs that give every token here a score of minus infinity, but for every third head
    for row, seq in enumerate(np.repeat(np.arange(3), new)):
        for s, channel, sign in ((0, 7, -1), (0, L // 4 + 1, 1), (1, L // 2 + 3, -1), (1, L - 1, -1), (1, 0, 1), (2, 9, -1)):
            if s == seq:
                q[row, :, channel] = sign * np.maximum(np.abs(q[row, :, channel]), 0.125) * np.where(np.arange(9) % 3 == 2, -1, 1)
    out, lse = attend(gpu, q, qr, cache, table, lens, running(new))
    with np.errstate(invalid="ignore"):
        want = R.attention_ref(q, qr, cache, table, lens, running(new), (L * 3 / 8) ** -0.5)
    assert np.isnan(want[0]).any() and np.isfinite(want[2]).any()
    T.check_out(out, lse, want)
