"""Every compiled form of expanded latent attention (bounds as derived in test_gpu_latent)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from oracle import latent as R
from tests import test_gpu_latent as T
from tests import test_gpu_latent_forms as F
from tests.test_gpu_kv8 import bf16, i32, running

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["latent_prompt16", "latent_prompt32", "latent_prompt64", "latent_prompt128"])
def form(request, monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", request.param)
    return request.param


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,heads,new,lens", T.EXPANDED + [
    (128, 3, [1], [1000]), (128, 2, [17, 1, 3], [640, 129, 31]), (64, 4, [33, 16], [700, 128]), (128, 1, [40], [383])])
def test_expanded(form, gpu, D, heads, new, lens, causal):
    T.test_expanded(gpu, D, heads, new, lens, causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_finite(form, gpu, D, what):
    F.test_expanded_values_that_are_not_finite(gpu, D, what)


def test_many_prompts(form, gpu):
    F.test_expanded_many_prompts(gpu)


def test_rows_far_apart(form, gpu):
    F.test_expanded_rows_far_apart(gpu)


def test_same_bits(form, gpu):
    F.test_expanded_same_bits(gpu)


@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_fall_and_climb(form, gpu, D):
    # each 32 tokens have scores far from the last ones', down and up again: parts whose references lie 2^100 apart
    rng = np.random.default_rng(5)
    keys, heads, n = 600, 2, 20
    q, kv, r = (bf16(rng.standard_normal(s)) for s in ((n, heads, D * 3 // 2), (keys, heads, 2 * D), (keys, D // 2)))
    q[..., 0] = 1
    kv[..., 0] = (np.abs(np.arange(keys) // 32 - 9) * 64)[:, None]
    out, lse = torch.empty((n, heads, D), dtype=torch.bfloat16, device=gpu), torch.empty((n, heads), device=gpu)
    dg.latent_expanded_attention(T.dev_bf16(q, gpu), T.dev_bf16(kv, gpu), T.dev_bf16(r, gpu), i32(running([n]), gpu),
                                 i32(running([keys]), gpu), n, out, lse, scale=0.125)
    r_out, w, l = R.expanded_ref(q, kv, r, [0, n], [0, keys], 0.125)
    # scale sum |q||k| < 72 + 80: twice the bound's 80, so e < 2^-11, and 2 e of W
    assert (np.abs(T.host(out) - r_out) <= 2.0 ** -8 * np.abs(r_out) + (2.0 ** -8 + 2.0 ** -10) * w).all()
    assert (np.abs(lse.cpu().numpy() - l) <= 2.0 ** -11 + 2.0 ** -20 * np.abs(l)).all()
