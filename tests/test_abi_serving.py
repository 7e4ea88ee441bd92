"""Host-side refusals of the 4-bit weight and 8-bit cache entry points (CPU:
every case below fails validation, or is a no-op, before a device is touched)."""

import ctypes

import pytest

import fp8_block_scaled_nt_amd as dg

P = ctypes.c_void_p
GOOD, ODD, OFF4 = P(0x10000), P(0x10004), P(0x10002)


@pytest.fixture(scope="module")
def lib():
    return dg.lib()


def call(f, args, **changed):
    args = dict(args, **changed)
    return f(*args.values(), None)


W4 = dict(a=GOOD, codes=GOOD, scales=GOOD, zeros=None, d=GOOD, m=4, n=64, k=256, group=128, format=0)


@pytest.mark.parametrize("changed,status", [
    (dict(a=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(d=None), 1), (dict(m=-1), 1), (dict(n=0), 1),
    (dict(format=2), 1), (dict(format=1), 1), (dict(zeros=GOOD), 1),              # zeros and the format disagree
    (dict(group=16), 2), (dict(group=256), 2), (dict(group=0), 2), (dict(k=0), 2), (dict(k=192), 2), (dict(k=-128), 2),
    (dict(a=ODD), 3), (dict(scales=ODD), 3), (dict(zeros=ODD, format=1), 3), (dict(m=0), 0), (dict(m=0, a=None, d=None), 0),
])
def test_w4_gemm(lib, changed, status):
    assert call(lib.dg_bf16_w4_gemm_nt, W4, **changed) == status
    assert (len(lib.dg_last_error_message()) > 0) == (status != 0)


@pytest.mark.parametrize("changed,status", [
    (dict(x=None), 1), (dict(codes=None), 1), (dict(zeros=GOOD), 1), (dict(n=-1), 1), (dict(format=-1), 1), (dict(k=100), 2),
    (dict(x=ODD), 3), (dict(codes=ODD), 3),
])
def test_w4_quantise(lib, changed, status):
    args = dict(x=GOOD, x_bf16=1, codes=GOOD, scales=GOOD, zeros=None, n=64, k=256, group=64, format=0)
    assert call(lib.dg_quantize_b_w4, args, **changed) == status
    if "x" not in changed:
        args = dict(codes=GOOD, scales=GOOD, zeros=None, w=GOOD, n=64, k=256, group=64, format=0)
        assert call(lib.dg_dequantize_b_w4, args, **changed) == status


CACHE = dict(k_codes=GOOD, v_codes=GOOD, k_scales=GOOD, v_scales=GOOD, table=GOOD)
SIZES = dict(batch=2, total=5, most=3, h_kv=2, d=128, block=64, num_blocks=8, max_blocks=4)
APPEND = dict(k=GOOD, k_stride=256, v=GOOD, v_stride=256, **CACHE, ctx=GOOD, cu=GOOD, **SIZES)
ATTEND = dict(q=GOOD, q_stride=1024, **CACHE, lens=GOOD, cu=GOOD, out=GOOD, lse=GOOD, scale=0.1, causal=1, window=0,
              **{n: v for n, v in list(SIZES.items())[:3]}, h_q=8, **{n: v for n, v in list(SIZES.items())[3:]})

BOTH = [
    (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(batch=-1), 1),
    (dict(total=-1), 1), (dict(most=-1), 1), (dict(h_kv=0), 1), (dict(num_blocks=-1), 1), (dict(max_blocks=-1), 1),
    (dict(d=96), 2), (dict(d=0), 2), (dict(block=48), 2), (dict(block=8), 2), (dict(block=256), 2), (dict(batch=70000), 2),
    (dict(max_blocks=1 << 25), 2),
    (dict(k_codes=ODD), 3), (dict(v_codes=ODD), 3), (dict(k_scales=OFF4), 3), (dict(table=OFF4), 3), (dict(cu=OFF4), 3),
    (dict(batch=0), 0), (dict(total=0), 0), (dict(most=0), 0),
]


@pytest.mark.parametrize("changed,status", BOTH + [
    (dict(k=None), 1), (dict(ctx=None), 1), (dict(k_stride=255), 2), (dict(v_stride=248), 2), (dict(v=ODD), 3),
    (dict(total=0, k=None, v=None), 0), (dict(max_blocks=0), 0), (dict(num_blocks=0), 0),
])
def test_append(lib, changed, status):
    assert call(lib.dg_kv8_append, APPEND, **changed) == status
    assert (len(lib.dg_last_error_message()) > 0) == (status != 0)


@pytest.mark.parametrize("changed,status", BOTH + [
    (dict(q=None), 1), (dict(out=None), 1), (dict(lens=None), 1), (dict(window=-1), 1), (dict(scale=-0.5), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(window=5, causal=0), 1),
    (dict(h_q=7), 2), (dict(h_q=0), 2), (dict(q_stride=1020), 2), (dict(q_stride=0), 2), (dict(total=1 << 30, most=1 << 30, h_q=64, q_stride=8192), 2),
    (dict(q=ODD), 3), (dict(out=ODD), 3), (dict(lse=OFF4), 3), (dict(total=0, q=None, out=None), 0),
])
def test_attention(lib, changed, status):
    assert call(lib.dg_kv8_attention, ATTEND, **changed) == status
    assert (len(lib.dg_last_error_message()) > 0) == (status != 0)


def test_workspace_size(lib):
    assert lib.dg_kv8_attention_workspace_size(128, None) == 1
    out = ctypes.c_size_t(7)
    assert lib.dg_kv8_attention_workspace_size(96, ctypes.byref(out)) == 2 and out.value == 0


def test_no_device_is_reported(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert call(lib.dg_bf16_w4_gemm_nt, W4) == 4
    assert call(lib.dg_kv8_append, APPEND) == 4
    assert call(lib.dg_kv8_attention, ATTEND) == 4
