"""The cache's calls through the binding where there is nothing: no sequences,
no blocks, a table of no width."""

import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests.test_gpu_kv8 import i32, way  # noqa: F401

pytestmark = pytest.mark.gpu


def test_no_sequences(way, gpu):  # noqa: F811
    cache = dg.empty_kv8_cache(4, 2, 64, 16, gpu)
    for x in cache:
        x.view(torch.uint8).fill_(3)
    table, none, cu = torch.zeros((0, 5), dtype=torch.int32, device=gpu), i32([], gpu), i32([0], gpu)
    x, q = (torch.zeros((0, n, 64), dtype=torch.bfloat16, device=gpu) for n in (2, 4))
    dg.kv8_append(x, x, cache, table, none, cu, 0)
    assert dg.kv8_attention(q, cache, table, none, cu, 0, torch.empty_like(q)).shape == (0, 4, 64)
    assert all((y.view(torch.uint8) == 3).all() for y in cache)


@pytest.mark.parametrize("blocks,width", [(0, 3), (0, 0), (4, 0)])
@pytest.mark.parametrize("new", [1, 40])
def test_no_blocks(way, gpu, blocks, width, new):  # noqa: F811
    cache = dg.empty_kv8_cache(blocks, 2, 64, 16, gpu)
    table, lens, cu = torch.zeros((2, width), dtype=torch.int32, device=gpu), i32([new, 5], gpu), i32([0, new, new + 1], gpu)
    x, q = (torch.ones((new + 1, n, 64), dtype=torch.bfloat16, device=gpu) for n in (2, 4))
    dg.kv8_append(x, x, cache, table, i32([0, 4], gpu), cu, new)
    out, lse = torch.full_like(q, 7.0), torch.zeros((new + 1, 4), device=gpu)
    dg.kv8_attention(q, cache, table, lens, cu, new, out, lse)
    assert (out == 0).all() and (lse == float("-inf")).all()
