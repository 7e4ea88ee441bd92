"""Latent operators: a stride of 0 from head to head is taken for rows that are
read and refused for rows that are written (CPU: a call that passes ends at the
missing device)."""

import ctypes

import pytest

import fp8_block_scaled_nt_amd as dg
from tests.test_abi_latent import APPEND, ATTEND, NO_DEVICE, no_gpu
from tests.test_abi_serving import call


@no_gpu
@pytest.mark.parametrize("changed,status", [
    (dict(q_head=0), NO_DEVICE), (dict(r_head=0), NO_DEVICE), (dict(q_head=0, q_stride=0, r_head=0, r_stride=0), NO_DEVICE),
    (dict(q_head=8), 2), (dict(r_head=56), 2), (dict(q_head=-512), 2), (dict(o_head=0), 2), (dict(o_head=0, o_stride=1 << 40), 2),
    (dict(o_head=0, total=1), 2), (dict(o_head=0, h_q=1), NO_DEVICE), (dict(o_head=0, o_stride=504, h_q=1), 2)])
def test_attention(changed, status):
    assert call(dg.lib().dg_latent_attention, ATTEND, **changed) == status


@no_gpu
@pytest.mark.parametrize("changed,status", [
    (dict(q_head=0), NO_DEVICE), (dict(q_head=0, q_stride=0), NO_DEVICE), (dict(q_head=8), 2), (dict(o_head=0), 2),
    (dict(o_head=0, total=1), 2), (dict(o_head=0, h_q=1), NO_DEVICE)])
def test_append(changed, status):
    apart = dict(APPEND, q_out=ctypes.c_void_p(0x20000))
    assert call(dg.lib().dg_latent_append, apart, **changed) == status


def test_append_in_place():
    # the rows that are read are then the ones that are written
    assert call(dg.lib().dg_latent_append, dict(APPEND, q_out=APPEND["q"], o_stride=APPEND["q_stride"]), q_head=0, o_head=0) == 2
