"""Latent operators: padded batches whose rows come out even, tokens that are
not finite under a norm, outputs that overlap, tensors of another device
(bounds as derived in test_gpu_latent)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import latent as R
from tests import gpu_harness as H
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import bf16, i32, running
from tests.test_gpu_latent_forms import attend, queries, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,f8,heads,new,lens,most", [
    (512, True, 40, [3, 1, 0, 2], [300, 130, 90, 2], 3),
    (512, False, 16, [1, 0, 0, 1], [700, 64, 0, 1], 1),
    (256, False, 64, [0, 2, 0], [40, 515, 77], 2),
    (256, True, 5, [2, 4, 1], [0, 260, 900], 4),
])
def test_padded_batch_of_as_many_rows_as_its_longest_times_its_sequences(rows, gpu, L, f8, heads, new, lens, most):  # noqa: F811
    # neighbouring workgroups count on one tile each of every sequence, and find sequences that have fewer
    print(f"[case] padded {rows} {L} {f8} {heads} {new}", flush=True)
    rng = np.random.default_rng(sum(lens))
    cache, table = T.filled(rng, lens, 32, L, f8)
    total, real = most * len(new), sum(new)
    q, qr = queries(rng, total, heads, L)
    q[real:], qr[real:] = np.nan, np.nan
    out, lse = attend(gpu, q, qr, cache, table, lens, running(new), most=most)
    want = R.attention_ref(q[:real], qr[:real], cache, table, lens, running(new), (L * 3 / 8) ** -0.5)
    T.check_out(out[:real], lse[:real], want)
    assert torch.isnan(out[real:]).all() and torch.isnan(lse[real:]).all()


@pytest.mark.parametrize("f8", [False, True])
def test_append_of_tokens_that_are_not_finite_with_a_norm(gpu, f8):
    L, P, block = 256, 32, 16
    c = np.ones((4, L), np.float32)
    c[0, 5], c[1, 7], c[2, 200] = np.nan, np.inf, -np.inf
    table = np.array([[1]], np.int32)
    cache = T.upload(T.blank(2, block, L, f8), gpu)
    an = T.angles(np.random.default_rng(0), 4, P)
    norm = torch.full((L,), 2.0, dtype=torch.bfloat16, device=gpu)
    dg.latent_append(T.dev_bf16(c, gpu), torch.ones((4, P), dtype=torch.bfloat16, device=gpu), cache, i32(table, gpu), i32([0], gpu),
                     i32([0, 4], gpu), 4, H.f32_to_device(an, gpu), norm=norm, eps=0.0)
    got = cache[0][1, :4].float()
    if f8:
        got = got * cache[2][1, :4].repeat_interleave(128, 1)
    got = got.cpu().numpy()
    assert np.isnan(got[0]).all()
    for row, at in ((1, 7), (2, 200)):
        assert np.isnan(got[row, at]) and (np.delete(got[row], at) == 0).all()
    assert (got[3] == 2).all()


def test_outputs_that_overlap_are_refused(gpu):
    rng = np.random.default_rng(3)
    cache, table = T.filled(rng, [9], 16, 256, False)
    on, t, lens, cu = T.upload(cache, gpu), i32(table, gpu), i32([9], gpu), i32([0, 2], gpu)
    q, qr = (T.dev_bf16(x, gpu) for x in queries(rng, 2, 4, 256))
    one = torch.zeros((1, 4, 256), dtype=torch.bfloat16, device=gpu)
    with pytest.raises(dg.DGError):
        dg.latent_attention(q, qr, on, t, lens, cu, 2, one.expand(2, 4, 256))
    with pytest.raises(dg.DGError):
        dg.latent_attention(q, qr, on, t, lens, cu, 2, q.flatten()[:1280].clone().as_strided((2, 4, 256), (256, 256, 1)))
    with pytest.raises(dg.DGError):
        dg.latent_append(q[:, 0], qr[:, 0], on, t, i32([0], gpu), cu, 2, torch.zeros((4, 32), device=gpu), q_rope=qr,
                         q_out=one[..., :32].expand(2, 4, 32))
    # one set of queries for all tokens is no output
    out, same = torch.empty_like(q), torch.empty_like(q)
    dg.latent_attention(q[:1].expand(2, 4, 256), qr[:1].expand(2, 4, 32), on, t, lens, cu, 2, out)
    dg.latent_attention(q[:1].repeat(2, 1, 1), qr[:1].repeat(2, 1, 1), on, t, lens, cu, 2, same)
    assert torch.equal(out, same)


def test_tensors_of_another_device_are_refused(gpu, monkeypatch):
    rng = np.random.default_rng(4)
    cache, table = T.filled(rng, [9], 16, 256, False)
    on, t, lens, cu = T.upload(cache, gpu), i32(table, gpu), i32([9], gpu), i32([0, 2], gpu)
    q, qr = (T.dev_bf16(x, gpu) for x in queries(rng, 2, 4, 256))
    kv, wide = (torch.zeros((2, 4, n), dtype=torch.bfloat16, device=gpu) for n in (128, 96))
    out, angles, rope = torch.zeros_like(q), torch.zeros((16, 32), device=gpu), qr[:, 0].contiguous()
    packed = q[:, 0].contiguous()
    here = torch.cuda.current_device()
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here + 1)      # seen from another one
    for call in (lambda: dg.latent_append(packed, rope, on, t, i32([0], gpu), cu, 2, angles),
                 lambda: dg.latent_gather(on, t, cu, packed, rope),
                 lambda: dg.latent_attention(q, qr, on, t, lens, cu, 2, out),
                 lambda: dg.latent_expanded_attention(wide, kv, rope, cu, cu, 2, out[..., :64].contiguous())):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert (out == 0).all()
