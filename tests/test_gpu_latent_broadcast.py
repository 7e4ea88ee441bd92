"""Latent operators: one query for all heads, by a stride of 0 from head to head."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests import gpu_harness as H
from tests import test_gpu_latent as T
from tests.test_gpu_kv8 import i32
from tests.test_gpu_latent_forms import queries, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 3])
def test_queries_shared_by_all_heads(rows, gpu, tokens):  # noqa: F811
    rng = np.random.default_rng(tokens)
    cache, table = T.filled(rng, [90], 16, 256, False)
    on, t, lens, cu = T.upload(cache, gpu), i32(table, gpu), i32([90], gpu), i32([0, tokens], gpu)
    q, qr = (T.dev_bf16(x, gpu) for x in queries(rng, tokens, 20, 256))
    wide, wider = q[:, :1].expand(-1, 20, -1), qr[:, :1].expand(-1, 20, -1)
    for a, b in ((wide, qr), (q, wider), (wide, wider)):
        outs = [torch.empty_like(q) for _ in range(2)]
        dg.latent_attention(a, b, on, t, lens, cu, tokens, outs[0])
        dg.latent_attention(a.contiguous(), b.contiguous(), on, t, lens, cu, tokens, outs[1])
        assert torch.equal(*outs)
    # outputs stay apart
    with pytest.raises(dg.DGError):
        dg.latent_attention(q, qr, on, t, lens, cu, tokens, torch.empty_like(q)[:, :1].expand(-1, 20, -1))


def test_rope_parts_shared_by_all_heads(gpu):
    rng = np.random.default_rng(5)
    cache, an = dg.empty_latent_cache(2, 256, 16, "bf16", gpu), H.f32_to_device(T.angles(rng, 9, 32), gpu)
    x, qr = (T.dev_bf16(rng.standard_normal(s), gpu) for s in ((4, 288), (4, 1, 32)))
    args = (x[:, :256], x[:, 256:], cache, i32([[1]], gpu), i32([2], gpu), i32([0, 4], gpu), 4, an)
    outs = [torch.zeros((4, 35, 32), dtype=torch.bfloat16, device=gpu) for _ in range(2)]
    dg.latent_append(*args, q_rope=qr.expand(-1, 35, -1), q_out=outs[0])
    dg.latent_append(*args, q_rope=qr.expand(-1, 35, -1).contiguous(), q_out=outs[1])
    assert torch.equal(*outs) and outs[0].abs().sum() > 0
    with pytest.raises(dg.DGError):
        dg.latent_append(*args, q_rope=qr.expand(-1, 35, -1))                # in place
