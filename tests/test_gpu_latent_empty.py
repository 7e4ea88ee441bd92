"""Latent operators and the 8-bit cache take arrays without tokens whatever
their strides: those that come from numpy have strides of 0."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests.test_gpu_kv8 import i32

pytestmark = pytest.mark.gpu


def none(gpu, *shape):
    x = torch.from_numpy(np.zeros(shape, np.float32)).to(gpu).bfloat16()
    assert x.numel() == 0
    return x.as_strided(shape, (0,) * len(shape))


def test_expanded_attention_without_keys(gpu):
    q = torch.ones((3, 4, 96), dtype=torch.bfloat16, device=gpu)
    out, lse = torch.full((3, 4, 64), float("nan"), dtype=torch.bfloat16, device=gpu), torch.full((3, 4), float("nan"), device=gpu)
    dg.latent_expanded_attention(q, none(gpu, 0, 4, 128), none(gpu, 0, 32), i32([0, 3], gpu), i32([0, 0], gpu), 3, out, lse)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_no_tokens_at_all(gpu):
    cache, angles = dg.empty_latent_cache(2, 256, 16, "bf16", gpu), torch.zeros((4, 32), device=gpu)
    t, one, cu = i32([[1]], gpu), i32([3], gpu), i32([0, 0], gpu)
    dg.latent_append(none(gpu, 0, 256), none(gpu, 0, 32), cache, t, one, cu, 1, angles, q_rope=none(gpu, 0, 4, 32),
                     q_out=none(gpu, 0, 4, 32))
    out = none(gpu, 0, 4, 256)
    assert dg.latent_attention(none(gpu, 0, 4, 256), none(gpu, 0, 4, 32), cache, t, one, cu, 1, out) is out
    kv8 = dg.empty_kv8_cache(2, 2, 128, block=16, device=gpu)
    dg.kv8_append(none(gpu, 0, 2, 128), none(gpu, 0, 2, 128), kv8, t, one, cu, 1)
    with pytest.raises(ValueError):
        dg.latent_append(none(gpu, 0, 128), none(gpu, 0, 32), cache, t, one, cu, 1, angles)
