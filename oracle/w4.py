"""4-bit weights with group scales: quantiser and product.  Test infrastructure only.

A weight matrix [n, k] holds 4-bit codes with one bf16 scale per row and group
of K, and in the integer format one zero point beside it:

    w[n, k] = s[n, g] * (c[n, k] - z[n, g]),   g = k // group

"e2m1": c is the e2m1 value of the code, z = 0.  "u4": c is the code 0..15.
Codes are packed two per byte as in ``e2m1.pack``.  Scales are kept here as
float32 arrays whose values are bf16.

The quantiser decides codes by fp32 arithmetic with IEEE divisions (numpy
float32), against the scale after its rounding to bf16.
"""

import numpy as np

from . import e2m1
from .check import bf16_round

AMAX_FLOOR = np.float32(1e-4)


def quantize_w4(x, fmt, group):
    """float32 [n, k] -> (packed codes, scales float32 of bf16 values, zeros uint8 or None)."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    n, k = x.shape
    g = x.reshape(n, k // group, group)
    if fmt == "e2m1":
        amax = np.maximum(np.abs(g).max(2), AMAX_FLOOR)
        s = bf16_round(amax / np.float32(6))
        codes = e2m1.encode((g / s[..., None]).astype(np.float32))
        return e2m1.pack(codes.reshape(n, k)), s, None
    lo, hi = np.minimum(g.min(2), np.float32(0)), np.maximum(g.max(2), np.float32(0))
    s = bf16_round(np.maximum(hi - lo, AMAX_FLOOR) / np.float32(15))
    z = np.minimum(np.rint(-lo / s), np.float32(15))
    codes = np.clip(np.rint(g / s[..., None]) + z[..., None], 0, 15).astype(np.uint8)
    return e2m1.pack(codes.reshape(n, k)), s, z.astype(np.uint8)


def dequantize_w4(codes, scales, zeros):
    """The float64 weights [n, k] that packed codes stand for (exact)."""
    n, groups = scales.shape
    c = e2m1.decode_packed(codes) if zeros is None else e2m1.unpack(codes).astype(np.float64)
    c = c.reshape(n, groups, -1)
    if zeros is not None:
        c = c - zeros.astype(np.float64)[..., None]
    return (c * scales.astype(np.float64)[..., None]).reshape(n, -1)


def w4_gemm_ref(a, codes, scales, zeros):
    """a [m, k] (values exact in float64) times the weights, float64 [m, n]."""
    return np.asarray(a, np.float64) @ dequantize_w4(codes, scales, zeros).T
