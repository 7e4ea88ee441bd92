"""The profiling hook times the product with 4-bit weights, like any other
GEMM, and clears itself there."""

import pytest
import torch

import fp8_block_scaled_nt_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["w4_rows", "w4_tile"])
def test_hook_times_the_4_bit_product(gpu, monkeypatch, way):
    monkeypatch.setenv("DG_FORCE_CONFIG", way)
    w = dg.quantize_b_w4(torch.randn(4096, 4096, device=gpu), "u4", 64)
    a, d = torch.randn(32, 4096, device=gpu).bfloat16(), torch.empty((32, 4096), dtype=torch.bfloat16, device=gpu)
    x, y = torch.randn(512, 4096, device=gpu).bfloat16(), torch.empty((512, 512), dtype=torch.bfloat16, device=gpu)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def run():
        dg.bf16_w4_gemm_nt(a, w, d)
        dg.dequantize_b_w4(w)            # no GEMM: leaves the hook alone

    run()
    start.record()
    stop.record()
    torch.cuda.synchronize()
    dg.profile_next_launch(start, stop)
    run()
    torch.cuda.synchronize()
    spent = start.elapsed_time(stop)
    whole = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    whole[0].record()
    for _ in range(10):
        dg.bf16_w4_gemm_nt(a, w, d)
    whole[1].record()
    dg.bf16_gemm_nt(x, x[:512].contiguous(), y)
    torch.cuda.synchronize()
    assert start.elapsed_time(stop) == spent                     # no later launch took the hook
    each = whole[0].elapsed_time(whole[1]) / 10
    assert each / 4 < spent < 4 * each                           # the kernel alone, against calls in a row
