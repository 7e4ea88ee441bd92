"""Latent operators: tokens whose place lies before the first one are nobody's:
append ignores them, gather leaves their rows."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import latent as R
from tests import gpu_harness as H
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import bf16, i32, running

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f8", [False, True])
def test_append_before_the_first_token(gpu, f8):
    # sequence 0 begins 3 tokens before its cache, 1 wholly before it, 2 stands at 0
    L, P, block, ctx, new = 256, 32, 16, [-3, -40, 0], [8, 5, 4]
    rng = np.random.default_rng(1)
    table = np.array([[2, 0], [1, 3], [4, 5]], np.int32)
    before, an, total = T.blank(6, block, L, f8), T.angles(rng, 20, P), sum(new)
    wide, q = bf16(rng.standard_normal((total, L + P))), bf16(rng.standard_normal((total, 3, P)))
    x, qd = T.dev_bf16(wide, gpu), T.dev_bf16(q, gpu)
    cache = T.upload(before, gpu)
    dg.latent_append(x[:, :L], x[:, L:], cache, i32(table, gpu), i32(ctx, gpu), i32(running(new), gpu), max(new),
                     H.f32_to_device(an, gpu), q_rope=qd)
    want, turned = R.append_ref(wide[:, :L], wide[:, L:], before, table, ctx, running(new), an, q=q)
    ignored = np.isnan(turned).all((1, 2))
    assert ignored.nonzero()[0].tolist() == [0, 1, 2, 8, 9, 10, 11, 12]
    got = T.host(qd)
    assert np.array_equal(got[ignored], q[ignored])
    assert (np.abs(got - turned)[~ignored] <= 2.0 ** -8 * np.abs(turned)[~ignored] + 2.0 ** -17).all()
    assert np.array_equal(np.isnan(T.host(cache[1])), np.isnan(want[1]))
    if f8:
        assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), want[0])
        assert np.array_equal(cache[2].cpu().numpy(), want[2], equal_nan=True)
    else:
        assert np.array_equal(T.host(cache[0]), want[0], equal_nan=True)


@pytest.mark.parametrize("f8", [False, True])
def test_gather_before_the_first_token(gpu, f8):
    rng = np.random.default_rng(2)
    L, starts, lens = 512, [-5, -30, 3], [20, 10, 9]
    cache, table = T.filled(rng, [40, 40, 40], 16, L, f8)
    total = sum(lens)
    rows = torch.full((total, L), 7.0, dtype=torch.bfloat16, device=gpu)
    rope = torch.full((total, L // 8), 7.0, dtype=torch.bfloat16, device=gpu)
    dg.latent_gather(T.upload(cache, gpu), i32(table, gpu), i32(running(lens), gpu), rows, rope, starts=i32(starts, gpu))
    got, got_rope, at = T.host(rows), T.host(rope), 0
    for s, (a, n) in enumerate(zip(starts, lens)):
        c, r, there = R.tokens_of(cache, table, s, a, n)
        assert there.tolist() == [a + i >= 0 for i in range(n)]
        assert np.array_equal(got[at:at + n][there], c[there]) and np.array_equal(got_rope[at:at + n][there], r[there])
        assert (got[at:at + n][~there] == 7).all() and (got_rope[at:at + n][~there] == 7).all()
        at += n
