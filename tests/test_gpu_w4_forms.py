"""Every compiled form of the 4-bit product against the oracle: both formats,
groups of 32, 64 and 128, K that fills whole units of 128 and K that does not,
each number of rows that the row and tile kernels are built for, K in splits.
Tolerances as in test_gpu_w4."""

import pytest
import torch

import fp8_block_scaled_nt_amd as dg
import oracle
from tests import gpu_harness as H
from tests.test_gpu_w4 import activations, to_device, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e2m1", "u4"])
@pytest.mark.parametrize("group,k", [(32, 1152), (32, 1120), (64, 1152), (64, 1088), (128, 1152)])
@pytest.mark.parametrize("way,m", [("w4_rows", 3), ("w4_rows", 8), ("w4_rows", 16), ("w4_rows", 37), ("w4_tile", 2), ("w4_tile", 29),
                                   ("w4_tile", 64), ("w4_tile", 70)])
def test_forms(gpu, monkeypatch, way, m, group, k, fmt):
    print(f"[case] {way} {fmt} {m}x145x{k} g{group}", flush=True)
    monkeypatch.setenv("DG_FORCE_CONFIG", way)
    n = 145
    w = oracle.quantize_w4(weights(n, k, n + k), fmt, group)
    a, ref_a = activations(m, k, m + k, gpu)
    assert (dg.bf16_w4_workspace_size(m, n, k, group, fmt) > 0) == (way == "w4_tile")
    d, flat = H.sentinel_bf16((m, n), gpu, 256)
    dg.bf16_w4_gemm_nt(a, to_device(*w, gpu), d)
    torch.cuda.synchronize()
    res = oracle.tolerance_check(H.d_float(d), oracle.w4_gemm_ref(ref_a, *w))
    assert res["ok"], res
    assert H.guard_untouched(flat, m * n)
