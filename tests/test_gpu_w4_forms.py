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


@pytest.mark.parametrize("way", ["w4_rows", "w4_tile"])
def test_infinities_and_the_range_of_u4(gpu, monkeypatch, way):
    monkeypatch.setenv("DG_FORCE_CONFIG", way)
    n, k = 24, 128
    x = weights(n, k, 3)
    a = torch.zeros((3, k), device=gpu)
    a[0, 9] = float("inf")
    a[1, 9], a[1, 10] = 2.0 ** 119, 1.0      # 143 |a| is within fp32's range
    a[2, 9] = 2.0 ** 122                     # and here past it
    for fmt in ("e2m1", "u4"):
        w = oracle.quantize_w4(x, fmt, 32)
        d = torch.empty((3, n), dtype=torch.bfloat16, device=gpu)
        dg.bf16_w4_gemm_nt(a.bfloat16(), to_device(*w, gpu), d)
        value = torch.from_numpy(oracle.dequantize_w4(*w)[:, 9]).to(gpu)
        got = d.double()
        if fmt == "u4":
            assert torch.isnan(got[0]).all() and not torch.isfinite(got[2]).any()
        else:
            assert torch.equal(got[0][value != 0], (value * float("inf"))[value != 0]) and torch.isnan(got[0][value == 0]).all()
            assert ((got[2] - value * 2.0 ** 122).abs() <= 2.0 ** 114 * value.abs()).all()
        # one large term: rounded to bf16, and for u4 two fp32 roundings of terms 143 s |a|
        scale = torch.from_numpy(w[1][:, 0]).to(gpu).double()
        assert ((got[1] - value * 2.0 ** 119).abs() <= 2.0 ** 111 * value.abs() + 2.0 ** (119 - 24 + 8) * scale + 1.0).all()
