"""Calls on an empty batch, pool or table: their arrays have no elements, and
their pointers may be null (CPU: no-ops, or as far as the missing device)."""

import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests.test_abi_serving import APPEND, ATTEND, call

POOL = dict(num_blocks=0, k_codes=None, v_codes=None, k_scales=None, v_scales=None)


@pytest.mark.parametrize("changed,status", [
    (dict(batch=0, table=None, ctx=None), 0), (dict(max_blocks=0, table=None), 0), (POOL, 0),
    (dict(batch=0, table=None, ctx=None, total=0, most=0, k=None, v=None, **POOL), 0),
    (dict(POOL, num_blocks=1), 1), (dict(table=None), 1), (dict(ctx=None), 1), (dict(batch=0, cu=None), 1),
])
def test_append(changed, status):
    assert call(dg.lib().dg_kv8_append, APPEND, **changed) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls' arguments are no real memory")
@pytest.mark.parametrize("changed,status", [
    (dict(batch=0, table=None, lens=None), 0), (dict(total=0, q=None, out=None, lse=None, **POOL), 0),
    (POOL, 4), (dict(max_blocks=0, table=None), 4),           # queries without keys are written on the device
    (dict(POOL, num_blocks=1), 1), (dict(table=None), 1), (dict(lens=None), 1),
])
def test_attention(changed, status):
    assert call(dg.lib().dg_kv8_attention, ATTEND, **changed) == status
