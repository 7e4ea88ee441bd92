"""4-bit weights with group scales on the GPU against the oracle.

Codes, scales and zeros are compared bit for bit (both sides decide them by
the same fp32 arithmetic).  Products are held to the oracle's acceptance rule
(8e-3 |r| + 1e-3 rms): half an ulp of the bf16 output is 1.95e-3 |r|; the
fp32 sums add at most k 2^-24 sum |a w| (for u4 17 times that, since codes
enter as 128 + c), under 1e-3 rms at these sizes.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_nt_amd as dg
import oracle
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


def weights(n, k, seed):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[0] = 0                                  # all-zero groups take the amax floor
    w[-1] = np.abs(w[-1])                     # one-sided groups
    return oracle.bf16_round(w)


def to_device(codes, scales, zeros, dev):
    return (torch.from_numpy(codes).to(dev), H.f32_to_device(scales, dev).bfloat16(),
            None if zeros is None else torch.from_numpy(zeros).to(dev))


def activations(m, k, seed, dev):
    a = torch.from_numpy(np.random.default_rng(seed).standard_normal((m, k)).astype(np.float32)).bfloat16()
    return a.to(dev), a.double().numpy()


SIZES = [
    (1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 96, 32), (3, 33, 1056, 32), (2, 2112, 7168, 128), (5, 1001, 1088, 64),
    (15, 100, 192, 64), (16, 64, 4096, 128), (17, 130, 640, 128), (31, 48, 224, 32), (33, 257, 512, 64),
    (64, 512, 1024, 128), (64, 31, 2016, 32), (65, 80, 384, 64), (130, 65, 256, 128), (1, 40, 16384, 128),
]


@pytest.fixture(params=["", "w4_rows", "w4_tile"])
def way(request, monkeypatch):
    """The library's own choice between its two ways of a product, and each of them."""
    if request.param:
        monkeypatch.setenv("DG_FORCE_CONFIG", request.param)
    return request.param


@pytest.mark.parametrize("fmt", ["e2m1", "u4"])
@pytest.mark.parametrize("m,n,k,group", SIZES)
def test_gemm(way, gpu, m, n, k, group, fmt):
    print(f"[case] w4 {fmt} {m}x{n}x{k} g{group}", flush=True)
    w = oracle.quantize_w4(weights(n, k, n + k), fmt, group)
    a, ref_a = activations(m, k, m + k, gpu)
    d, flat = H.sentinel_bf16((m, n), gpu, 256)
    dg.bf16_w4_gemm_nt(a, to_device(*w, gpu), d)
    torch.cuda.synchronize()
    res = oracle.tolerance_check(H.d_float(d), oracle.w4_gemm_ref(ref_a, *w))
    assert res["ok"], res
    assert H.guard_untouched(flat, m * n)


# large enough for tiles to be chosen, K in splits, odd sizes, more than one tile of rows
@pytest.mark.parametrize("fmt,m,n,k,group", [("u4", 65, 2113, 7264, 32), ("e2m1", 64, 4096, 7168, 64), ("u4", 33, 4001, 7168, 128)])
def test_gemm_large(gpu, fmt, m, n, k, group):
    print(f"[case] w4 {fmt} {m}x{n}x{k} g{group}", flush=True)
    w = oracle.quantize_w4(weights(n, k, n + k), fmt, group)
    a, ref_a = activations(m, k, m + k, gpu)
    assert dg.bf16_w4_workspace_size(m, n, k, group, fmt) > 0
    d, flat = H.sentinel_bf16((m, n), gpu, 256)
    dev = to_device(*w, gpu)
    dg.bf16_w4_gemm_nt(a, dev, d)
    again = torch.empty_like(d)
    dg.bf16_w4_gemm_nt(a, dev, again)
    torch.cuda.synchronize()
    res = oracle.tolerance_check(H.d_float(d), oracle.w4_gemm_ref(ref_a, *w))
    assert res["ok"], res
    assert H.guard_untouched(flat, m * n) and torch.equal(d, again)


def test_gemm_split_in_a_graph(gpu):
    m, n, k = 48, 4096, 8192
    w = to_device(*oracle.quantize_w4(weights(n, k, 5), "u4", 128), gpu)
    a, _ = activations(m, k, 6, gpu)
    d = torch.empty((m, n), dtype=torch.bfloat16, device=gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    # a stream that has no workspace yet cannot get one while it captures
    with pytest.raises(dg.DGError) as refused:
        with torch.cuda.graph(graph, stream=side):
            dg.bf16_w4_gemm_nt(a, w, d)
    assert refused.value.status == 7
    torch.cuda.synchronize()
    dg.reserve_workspace(dg.bf16_w4_workspace_size(m, n, k, 128, "u4"), side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dg.bf16_w4_gemm_nt(a, w, d)
    for i in range(4):
        x, _ = activations(m, k, 7 + i, gpu)
        want = torch.empty_like(d)
        dg.bf16_w4_gemm_nt(x, w, want)
        a.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)


@pytest.mark.parametrize("fmt", ["e2m1", "u4"])
def test_gemm_extremes(way, gpu, fmt):
    # every code, scales over 2^+-40, zeros at both ends, large and tiny activations
    n, k, group = 48, 256, 32
    rng = np.random.default_rng(9)
    codes = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    scales = np.exp2(rng.integers(-40, 40, (n, 1)).astype(np.float32)) * np.ones((1, k // group), np.float32)
    zeros = rng.choice(np.array([0, 15, 8], np.uint8), (n, k // group)) if fmt == "u4" else None
    a = (rng.standard_normal((4, k)) * np.exp2(np.array([[-60.0], [0], [30], [60]]))).astype(np.float32)
    a = oracle.bf16_round(a)
    d = torch.empty((4, n), dtype=torch.bfloat16, device=gpu)
    dg.bf16_w4_gemm_nt(H.f32_to_device(a, gpu).bfloat16(), to_device(codes, scales, zeros, gpu), d)
    r = oracle.w4_gemm_ref(a, codes, scales, zeros)
    got = H.d_float(d)
    for i in range(4):
        for j in range(n):
            size = np.abs(a[i].astype(np.float64)) @ np.abs(oracle.dequantize_w4(codes[j:j + 1], scales[j:j + 1],
                                                            None if zeros is None else zeros[j:j + 1])[0])
            # bf16 rounding, and k + 8 fp32 roundings of terms up to 143/1 of the largest |c - z| they stand for
            assert abs(got[i, j] - r[i, j]) <= 2 ** -8 * abs(r[i, j]) + (k + 8) * 2 ** -24 * 19 * size, (i, j)


def test_gemm_nan_and_inf_stay_in_their_row(way, gpu):
    w = oracle.quantize_w4(weights(40, 256, 1), "u4", 64)
    a, _ = activations(3, 256, 2, gpu)
    clean = torch.empty((3, 40), dtype=torch.bfloat16, device=gpu)
    dg.bf16_w4_gemm_nt(a, to_device(*w, gpu), clean)
    a[1, 7] = float("nan")
    a[2, 9] = float("inf")
    d = torch.empty_like(clean)
    dg.bf16_w4_gemm_nt(a, to_device(*w, gpu), d)
    assert torch.equal(d[0], clean[0]) and torch.isnan(d[1]).all() and not torch.isfinite(d[2]).any()


def test_gemm_repeats_and_streams(way, gpu):
    w = to_device(*oracle.quantize_w4(weights(96, 2048, 3), "e2m1", 128), gpu)
    a, _ = activations(7, 2048, 4, gpu)
    d = [torch.empty((7, 96), dtype=torch.bfloat16, device=gpu) for _ in range(3)]
    dg.bf16_w4_gemm_nt(a, w, d[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dg.bf16_w4_gemm_nt(a, w, d[1])
    torch.cuda.current_stream().wait_stream(side)
    dg.bf16_w4_gemm_nt(a, w, d[2])
    assert torch.equal(d[0], d[1]) and torch.equal(d[0], d[2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt,n,k,group", [("e2m1", 1, 32, 32), ("e2m1", 37, 384, 128), ("u4", 5, 224, 32),
                                           ("u4", 64, 1024, 64), ("e2m1", 130, 192, 64), ("u4", 3, 128, 128)])
def test_quantize(gpu, fmt, n, k, group, dtype):
    print(f"[case] w4 quantise {fmt} {n}x{k} g{group} {dtype}", flush=True)
    x = weights(n, k, k)
    if dtype == torch.float32:
        x = (x * np.float32(1.2345)).astype(np.float32)
    x[-1, :6] = [0.0, -0.0, 3.0, -448.0, 1e-30, -2.5]
    if dtype == torch.bfloat16:
        x = oracle.bf16_round(x)
    codes, scales, zeros = dg.quantize_b_w4(H.f32_to_device(x, gpu).to(dtype), fmt, group)
    ref = oracle.quantize_w4(x, fmt, group)
    assert np.array_equal(scales.float().cpu().numpy(), ref[1])
    assert np.array_equal(codes.cpu().numpy(), ref[0])
    assert zeros is None if ref[2] is None else np.array_equal(zeros.cpu().numpy(), ref[2])
    w = dg.dequantize_b_w4((codes, scales, zeros))
    assert np.array_equal(w.float().cpu().numpy(), oracle.bf16_round(oracle.dequantize_w4(*ref)))


def test_quantize_ties_and_many_scales(gpu):
    # every midpoint between e2m1 values and its neighbours, at scales over many binades; random values for
    # the correctly rounded quotient
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    near = np.concatenate([np.nextafter(mids, np.float32(0)), mids, np.nextafter(mids, np.float32(9)), [6.0, 0.0, -0.0]])
    row = np.concatenate([near, -near, np.zeros(128 - 2 * near.size)]).astype(np.float32)
    x = np.stack([row * np.float32(s) for s in (1.0, 0.5, 2.0 ** -10, 2.0 ** 20, 1.0078125, 1.9921875 * 2.0 ** -7)])
    rng = np.random.default_rng(31)
    more = (rng.standard_normal((200, 128)) * np.exp2(rng.integers(-12, 12, (200, 1)))).astype(np.float32)
    x = np.concatenate([x, more])
    for fmt in ("e2m1", "u4"):
        codes, scales, zeros = dg.quantize_b_w4(H.f32_to_device(x, gpu), fmt, 128)
        ref = oracle.quantize_w4(x, fmt, 128)
        assert np.array_equal(scales.float().cpu().numpy(), ref[1])
        assert np.array_equal(codes.cpu().numpy(), ref[0])
        assert zeros is None if ref[2] is None else np.array_equal(zeros.cpu().numpy(), ref[2])


def test_binding_refuses(gpu):
    a = torch.zeros((2, 128), dtype=torch.bfloat16, device=gpu)
    d = torch.zeros((2, 8), dtype=torch.bfloat16, device=gpu)
    w = dg.quantize_b_w4(torch.zeros((8, 128), device=gpu), "u4", 64)
    dg.bf16_w4_gemm_nt(a, w, d)
    with pytest.raises(ValueError):
        dg.bf16_w4_gemm_nt(a[:, :64].contiguous(), w, d)
    with pytest.raises(ValueError):
        dg.bf16_w4_gemm_nt(a, (w[0], w[1], w[2][:, :1].contiguous()), d)
    with pytest.raises(TypeError):
        dg.bf16_w4_gemm_nt(a, (w[0], w[1].float(), w[2]), d)
    with pytest.raises(ValueError):
        dg.bf16_w4_gemm_nt(a.cpu(), w, d)
    with pytest.raises(ValueError):
        dg.quantize_b_w4(torch.zeros((8, 128), device=gpu), "int4", 64)
    with pytest.raises(ValueError):
        dg.quantize_b_w4(torch.zeros((8, 96), device=gpu), "u4", 64)
    with pytest.raises(dg.DGError):  # a group of 16 reaches the library's own check
        dg.bf16_w4_gemm_nt(a, (w[0], torch.zeros((8, 8), dtype=torch.bfloat16, device=gpu), None), d)
    empty = torch.zeros((0, 128), dtype=torch.bfloat16, device=gpu)
    assert dg.bf16_w4_gemm_nt(empty, w, d[:0]).shape == (0, 8)
