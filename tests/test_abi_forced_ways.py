"""DG_FORCE_CONFIG at the entry points that choose between two ways: an unknown
name is refused, names of other entry points' configurations are not (CPU: the
check comes before a device is touched)."""

import ctypes

import pytest
import torch

import fp8_block_scaled_nt_amd as dg
from tests.test_abi_serving import ATTEND, W4, call

INVALID, NO_DEVICE = 1, 4


def calls(lib):
    size = ctypes.c_size_t(0)
    return (call(lib.dg_bf16_w4_gemm_nt, W4), call(lib.dg_kv8_attention, ATTEND),
            lib.dg_bf16_w4_workspace_size(4, 64, 256, 128, 0, ctypes.byref(size)))


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls' arguments are no real memory")
@pytest.mark.parametrize("name,status", [("w4_tiles", INVALID), ("kv8", INVALID), ("w4_rows", NO_DEVICE), ("w4_tile", NO_DEVICE),
                                         ("kv8_split", NO_DEVICE), ("kv8_prompt", NO_DEVICE), ("dense_64x64_w4_s3", NO_DEVICE),
                                         ("", NO_DEVICE)])
def test_names(monkeypatch, name, status):
    monkeypatch.setenv("DG_FORCE_CONFIG", name)
    lib = dg.lib()
    assert calls(lib) == (status,) * 3
    if status == INVALID:
        assert name in lib.dg_last_error_message().decode()


def test_calls_with_nothing_to_do_stay_no_ops(monkeypatch):
    monkeypatch.setenv("DG_FORCE_CONFIG", "w4_tiles")
    assert call(dg.lib().dg_bf16_w4_gemm_nt, W4, m=0) == 0 and call(dg.lib().dg_kv8_attention, ATTEND, total=0) == 0
