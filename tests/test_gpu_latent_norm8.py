"""Normalised latents of 512 into the e4m3 cache, as such a layer keeps them
(bounds as derived in test_gpu_latent)."""

import pytest

from tests import test_gpu_latent as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block,heads,ctx,new,pairs", [
    (64, 8, [3, 60, 0], [40, 5, 1], True), (16, 40, [0], [1], False), (128, 0, [127, 300], [129, 2], True)])
def test_append(gpu, block, heads, ctx, new, pairs):
    T.test_append(gpu, 512, True, block, heads, ctx, new, pairs, True)
