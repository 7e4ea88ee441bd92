"""Host-side refusals of the latent attention entry points (CPU: every case
below fails validation, is a no-op, or ends at the missing device)."""

import ctypes

import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests.test_abi_serving import ATTEND as KV8
from tests.test_abi_serving import GOOD, ODD, OFF4, call

NO_DEVICE = 4
CACHE = dict(latent=GOOD, rope=GOOD, scales=None, table=GOOD)
POOL = dict(latent_dim=512, block=64, num_blocks=8, max_blocks=4)
APPEND = dict(c=GOOD, c_stride=2112, r=GOOD, r_stride=2112, **CACHE, ctx=GOOD, cu=GOOD, angles=GOOD, positions=100, norm=GOOD,
              eps=1e-6, q=GOOD, q_stride=1536, q_head=192, q_out=GOOD, o_stride=512, o_head=64, interleaved=1, batch=2, total=5,
              most=3, h_q=8, **POOL)
GATHER = dict(**CACHE, starts=GOOD, cu=GOOD, to_latent=GOOD, to_rope=GOOD, batch=2, total=5, **POOL)
ATTEND = dict(q=GOOD, q_stride=4096, q_head=512, qr=GOOD, r_stride=1536, r_head=192, **CACHE, lens=GOOD, cu=GOOD, out=GOOD,
              o_stride=4096, o_head=512, lse=GOOD, scale=0.1, causal=1, batch=2, total=5, most=3, h_q=8, **POOL)
EXPAND = dict(q=GOOD, q_stride=1536, kv=GOOD, kv_stride=2048, r=GOOD, r_stride=64, cu_q=GOOD, cu_kv=GOOD, out=GOOD, lse=GOOD,
              scale=0.1, causal=1, batch=2, total=5, total_kv=9, most=3, heads=8, head_dim=128)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the calls' arguments are no real memory")


@pytest.fixture(scope="module")
def lib():
    return dg.lib()


ALL = [
    (dict(latent=None), 1), (dict(rope=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(batch=-1), 1), (dict(total=-1), 1),
    (dict(num_blocks=-1), 1), (dict(max_blocks=-1), 1), (dict(latent_dim=384), 2), (dict(latent_dim=0), 2), (dict(block=48), 2),
    (dict(block=8), 2), (dict(block=256), 2), (dict(batch=70000), 2), (dict(max_blocks=1 << 25), 2), (dict(latent=ODD), 3),
    (dict(rope=ODD), 3), (dict(scales=ODD), 3), (dict(table=OFF4), 3), (dict(cu=OFF4), 3), (dict(total=0), 0), (dict(batch=0), 0),
    (dict(batch=0, table=None), 0),
]


@pytest.mark.parametrize("changed,status", ALL + [
    (dict(c=None), 1), (dict(r=None), 1), (dict(ctx=None), 1), (dict(angles=None), 1), (dict(q_out=None), 1), (dict(most=-1), 1),
    (dict(positions=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(h_q=0), 1), (dict(h_q=40000), 1),
    (dict(c_stride=504), 2), (dict(c_stride=516), 2), (dict(r_stride=60), 2), (dict(q_stride=-8), 2), (dict(q_head=60), 2),
    (dict(q_head=100), 2), (dict(o_head=56), 2), (dict(c=ODD), 3), (dict(q=ODD), 3), (dict(q_out=ODD), 3), (dict(angles=ODD), 3),
    (dict(norm=ODD), 3), (dict(ctx=OFF4), 3), (dict(most=0), 0), (dict(positions=0), 0), (dict(positions=0, angles=None), 0),
    (dict(total=0, c=None, r=None), 0), (dict(total=(1 << 25) + 1, most=1), 2),
    (dict(q=GOOD, q_out=GOOD, o_stride=1536), 1),                            # in place, with other strides from head to head
])
def test_append(lib, changed, status):
    # q and q_out of the other cases lie apart
    args = dict(APPEND, q_out=ctypes.c_void_p(0x20000)) if "q_out" not in changed else APPEND
    assert call(lib.dg_latent_append, args, **changed) == status
    assert (len(lib.dg_last_error_message()) > 0) == (status != 0)


@pytest.mark.parametrize("changed,status", ALL + [
    (dict(to_latent=None), 1), (dict(to_rope=None), 1), (dict(to_latent=ODD), 3), (dict(starts=OFF4), 3), (dict(num_blocks=0), 0),
    (dict(max_blocks=0, table=None), 0), (dict(total=(1 << 25) + 1), 2)])
def test_gather(lib, changed, status):
    assert call(lib.dg_latent_gather, GATHER, **changed) == status


@pytest.mark.parametrize("changed,status", ALL + [
    (dict(q=None), 1), (dict(qr=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(most=-1), 1), (dict(h_q=0), 1),
    (dict(h_q=40000), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(most=1 << 28), 2), (dict(q_head=504), 2), (dict(q_head=516), 2), (dict(r_head=32), 2), (dict(o_head=256), 2),
    (dict(o_stride=4), 2), (dict(q=ODD), 3), (dict(qr=ODD), 3), (dict(out=ODD), 3), (dict(lse=OFF4), 3), (dict(lens=OFF4), 3),
    (dict(most=0), 0), (dict(total=0, q=None, qr=None, out=None, lse=None), 0)])
def test_attention(lib, changed, status):
    assert call(lib.dg_latent_attention, ATTEND, **changed) == status


@pytest.mark.parametrize("changed,status", [
    (dict(q=None), 1), (dict(kv=None), 1), (dict(r=None), 1), (dict(out=None), 1), (dict(cu_q=None), 1), (dict(cu_kv=None), 1),
    (dict(batch=-1), 1), (dict(total=-1), 1), (dict(total_kv=-1), 1), (dict(most=-1), 1), (dict(heads=0), 1), (dict(scale=-0.5), 1),
    (dict(head_dim=96), 2), (dict(q_stride=1528), 2), (dict(kv_stride=2044), 2), (dict(kv_stride=1 << 26), 2), (dict(r_stride=56), 2),
    (dict(r_stride=1 << 26), 2), (dict(batch=70000), 2), (dict(total=1 << 24, most=1 << 24), 2), (dict(q=ODD), 3), (dict(kv=ODD), 3),
    (dict(r=ODD), 3), (dict(out=ODD), 3), (dict(cu_kv=OFF4), 3), (dict(total=0), 0), (dict(batch=0), 0), (dict(most=0), 0),
    (dict(total=0, q=None, out=None, lse=None), 0)])
@no_gpu
def test_expanded(lib, changed, status):
    got = call(lib.dg_latent_expanded_attention, EXPAND, **changed)
    assert got == status or (changed.get("total") == 1 << 24 and got == NO_DEVICE)


@no_gpu
def test_calls_that_would_run_need_a_device(lib):
    assert call(lib.dg_latent_append, dict(APPEND, q_out=ctypes.c_void_p(0x20000))) == NO_DEVICE
    assert call(lib.dg_latent_append, APPEND, q=None, q_out=None) == NO_DEVICE
    assert call(lib.dg_latent_append, APPEND, q=None, num_blocks=0, latent=None, rope=None) == NO_DEVICE
    assert call(lib.dg_latent_gather, GATHER, scales=GOOD, starts=None) == NO_DEVICE
    assert call(lib.dg_latent_attention, ATTEND) == NO_DEVICE
    # queries without tokens are written on the device
    assert call(lib.dg_latent_attention, ATTEND, num_blocks=0, latent=None, rope=None) == NO_DEVICE
    assert call(lib.dg_latent_expanded_attention, EXPAND, total_kv=0, kv=None, r=None) == NO_DEVICE


def test_workspace_size(lib):
    size = ctypes.c_size_t(7)
    f = lib.dg_latent_attention_workspace_size
    assert f(512, 1, 128, None) == 1
    for args, status in (((384, 1, 8), 2), ((512, -1, 8), 1), ((512, 1, 0), 1), ((512, 1 << 28, 8), 2)):
        assert f(*args, ctypes.byref(size)) == status and size.value == 0
        size.value = 7


@no_gpu
@pytest.mark.parametrize("name,status", [("latent_rows16", NO_DEVICE), ("latent_rows64", NO_DEVICE), ("latent_rows48", 1)])
def test_forced_forms(lib, monkeypatch, name, status):
    monkeypatch.setenv("DG_FORCE_CONFIG", name)
    size = ctypes.c_size_t(0)
    assert call(lib.dg_latent_attention, ATTEND) == call(lib.dg_kv8_attention, KV8) == status
    assert lib.dg_latent_attention_workspace_size(512, 1, 8, ctypes.byref(size)) == status
    assert call(lib.dg_latent_attention, ATTEND, total=0) == 0


@pytest.mark.parametrize("stride,head,total,heads,status", [
    (4096, 512, 5, 8, 4), (512, 512 * 5, 5, 8, 4), (512, 512, 5, 1, 4), (0, 512, 1, 8, 4), (8192, 520, 5, 8, 4), (1 << 62, 512, 5, 8, 4),
    (0, 512, 5, 8, 2), (504, 512, 5, 1, 2), (4088, 512, 5, 8, 2), (512, 512, 5, 8, 2), (512, 512 * 5 - 8, 5, 8, 2), (504, 1 << 62, 5, 8, 2),
])
@no_gpu
def test_rows_that_are_written_lie_apart(lib, stride, head, total, heads, status):
    # a call that passes ends at the missing device
    changed = dict(o_stride=stride, o_head=head, total=total, h_q=heads)
    assert call(lib.dg_latent_attention, ATTEND, **changed) == status
    changed.update(o_stride=stride // 8, o_head=head // 8)
    if all(x % 64 == 0 for x in (stride, head)):
        assert call(lib.dg_latent_append, dict(APPEND, q_out=ctypes.c_void_p(0x20000)), **changed) == status


@pytest.mark.parametrize("name,status", [("latent_prompt16", NO_DEVICE), ("latent_prompt128", NO_DEVICE), ("latent_prompt48", 1)])
@no_gpu
def test_forced_forms_of_prompts(lib, monkeypatch, name, status):
    monkeypatch.setenv("DG_FORCE_CONFIG", name)
    assert call(lib.dg_latent_expanded_attention, EXPAND) == call(lib.dg_latent_attention, ATTEND) == status
    assert call(lib.dg_latent_expanded_attention, EXPAND, total=0) == 0
