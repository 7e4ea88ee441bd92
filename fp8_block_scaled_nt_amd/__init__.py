"""Python binding of the gfx950 FP8 block-scaled NT GEMM library (libdg.so).

The binding only marshals arguments: it checks dtypes, shapes and devices of
torch tensors, passes their device pointers and the current HIP stream to the
C ABI (include/dg.h), and raises on a non-zero status.  Every step of the
computation runs in the library's HIP kernels; there is no fallback.  PyTorch
supplies device memory and streams.

Layouts (all row-major, packed):
  a    [m, k] e4m3 codes (torch.float8_e4m3fn or uint8); masked: [g, max_m, k]
  sfa  slab-major fp32 [k/128, get_sfa_ld(m)]; masked: [g, k/128, get_sfa_ld(max_m)]
  b    [n, k] e4m3; grouped: [g, n, k]
  sfb  fp32 [ceil(n/128), k/128]; grouped: [g, ceil(n/128), k/128]
  d    bf16 [m, n]; masked: [g, max_m, n]
  hq   (SwiGLU) e4m3 [g, max_m, inter]; hs fp32 [g, inter/128, get_sfa_ld(max_m)]
  FP4  a [m, k/2], b [n, k/2] uint8, two e2m1 codes per byte (low nibble first),
       with the FP8 scale layouts
  W4   (codes, scales, zeros): uint8 [n, k/2], two codes per byte (low nibble
       first), bf16 [n, k/group], and uint8 [n, k/group] or None; without zeros
       the codes are e2m1, with them integers 0..15
  KV8  (k_codes, v_codes, k_scales, v_scales): e4m3 [blocks, h_kv, block, d],
       e4m3 [blocks, h_kv, d, block], fp32 [blocks, h_kv] each; block tables
       int32 [batch, max_blocks]
"""

import ctypes
import os

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# DG_LIBRARY names another build of the same library (e.g. one whose host
# code is compiled with sanitizers); by default the in-tree libdg.so
LIB_PATH = os.environ.get("DG_LIBRARY") or os.path.join(_PKG_DIR, "libdg.so")

__all__ = [
    "DGError", "lib", "fp8_gemm_nt", "fp8_gemm_nt_noalloc", "m_grouped_fp8_gemm_nt_contiguous",
    "m_grouped_fp8_gemm_nt_masked", "m_grouped_fp8_gemm_nt_masked_swiglu", "m_grouped_fp8_gemm_nt_contiguous_swiglu",
    "quantize_a_1x128", "quantize_b_128x128",
    "k_grouped_fp8_gemm_nt", "bf16_gemm_nt", "fp4_gemm_nt", "quantize_a_1x128_fp4", "quantize_b_128x128_fp4", "get_m_alignment_for_contiguous_layout", "get_sfa_ld", "empty_sfa",
    "profile_next_launch",
    "reserve_workspace", "dense_workspace_size",
    "bf16_w4_gemm_nt", "bf16_w4_workspace_size", "quantize_b_w4", "dequantize_b_w4",
    "empty_kv8_cache", "kv8_append", "kv8_attention", "kv8_attention_workspace_size",
]


class DGError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, status, message):
        super().__init__(f"dg status {status}: {message}")
        self.status = status


_lib = None
_vp, _ci, _cl = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_SIGNATURES = {
    "dg_fp8_gemm_nt": [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _vp],
    "dg_fp8_gemm_nt_noalloc": [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _vp],
    "dg_m_grouped_fp8_gemm_nt_contiguous": [_vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp],
    "dg_m_grouped_fp8_gemm_nt_masked": [_vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _vp],
    "dg_m_grouped_fp8_gemm_nt_masked_swiglu": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _vp],
    "dg_m_grouped_fp8_gemm_nt_contiguous_swiglu": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp],
    "dg_k_grouped_fp8_gemm_nt": [_vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp],
    "dg_bf16_gemm_nt": [_vp, _vp, _vp, _ci, _ci, _ci, _vp],
    "dg_fp4_gemm_nt": [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _vp],
    "dg_quantize_a_1x128_fp4": [_vp, _vp, _vp, _ci, _ci, _vp],
    "dg_quantize_b_128x128_fp4": [_vp, _vp, _vp, _ci, _ci, _vp],
    "dg_get_m_alignment_for_contiguous_layout": [],
    "dg_get_sfa_ld": [_ci],
    "dg_quantize_a_1x128": [_vp, _vp, _vp, _ci, _ci, _vp],
    "dg_quantize_b_128x128": [_vp, _vp, _vp, _ci, _ci, _vp],
    "dg_status_string": [_ci],
    "dg_last_error_message": [],
    "dg_version": [],
    "dg_profile_next_launch": [_vp, _vp],
    "dg_reserve_workspace": [ctypes.c_size_t, _vp],
    "dg_dense_workspace_size": [_ci, _ci, _ci, _ci, ctypes.POINTER(ctypes.c_size_t)],
    "dg_bf16_w4_gemm_nt": [_vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _vp],
    "dg_bf16_w4_workspace_size": [_ci, _ci, _ci, _ci, _ci, ctypes.POINTER(ctypes.c_size_t)],
    "dg_quantize_b_w4": [_vp, _ci, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp],
    "dg_dequantize_b_w4": [_vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp],
    "dg_kv8_append": [_vp, _cl, _vp, _cl] + [_vp] * 7 + [_ci] * 8 + [_vp],
    "dg_kv8_attention": [_vp, _cl] + [_vp] * 9 + [ctypes.c_float] + [_ci] * 11 + [_vp],
    "dg_kv8_attention_workspace_size": [_ci, ctypes.POINTER(ctypes.c_size_t)],
}
_RESTYPES = {"dg_status_string": ctypes.c_char_p, "dg_last_error_message": ctypes.c_char_p,
             "dg_version": ctypes.c_char_p}


def lib():
    """Load libdg.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run fp8_block_scaled_nt_amd/build.py")
        h = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGNATURES.items():
            f = getattr(h, name)
            f.argtypes = args
            f.restype = _RESTYPES.get(name, ctypes.c_int)
        _lib = h
    return _lib


def _check(status):
    if status != 0:
        msg = lib().dg_last_error_message().decode()
        raise DGError(status, msg or lib().dg_status_string(status).decode())


def _stream():
    """Handle of the current stream (as torch.cuda.current_stream().cuda_stream, 3.0 us, in 0.3 us)."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _need(t, name, dtypes, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def profile_next_launch(start_event, stop_event):
    """Make the next GEMM launch on this thread record the two torch.cuda.Event
    objects (timing enabled, already recorded once so they exist) at the start
    and end of the kernel itself."""
    _check(lib().dg_profile_next_launch(start_event._as_parameter_, stop_event._as_parameter_))


def reserve_workspace(nbytes, stream=None):
    """Size the split-K workspace of a stream (default: the current one) on
    the current device for `nbytes` of partial tiles, so that later calls on
    that stream allocate nothing (and can be captured in a graph)."""
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    _check(lib().dg_reserve_workspace(int(nbytes), st))


_DTYPES = {"fp8": 0, "bf16": 1, "fp4": 2}


def dense_workspace_size(m, n, k, dtype="fp8"):
    """Split-K workspace bytes a dense call (fp8_gemm_nt, bf16_gemm_nt or
    fp4_gemm_nt) of this shape makes on the current device; 0 if it does not
    split K.  Give it to reserve_workspace before capturing such calls."""
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be one of {sorted(_DTYPES)}")
    out = ctypes.c_size_t(0)
    _check(lib().dg_dense_workspace_size(_DTYPES[dtype], int(m), int(n), int(k), ctypes.byref(out)))
    return out.value


def get_m_alignment_for_contiguous_layout():
    return lib().dg_get_m_alignment_for_contiguous_layout()


def get_sfa_ld(m):
    return lib().dg_get_sfa_ld(int(m))


def empty_sfa(m, k, groups=None, device="cuda"):
    """Allocate a slab-major sfa buffer for m rows (optionally per group)."""
    shape = (k // 128, get_sfa_ld(m))
    if groups is not None:
        shape = (groups,) + shape
    return torch.empty(shape, dtype=torch.float32, device=device)


def fp8_gemm_nt(a_pair, b_pair, d):
    """D = A . B^T with block scales.  a_pair = (a [m,k], sfa), b_pair = (b [n,k], sfb),
    d: bf16 [m, n], written in place."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", _FP8, 2)
    _need(b, "b", _FP8, 2)
    _need(d, "d", (torch.bfloat16,), 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or tuple(d.shape) != (m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} b{tuple(b.shape)} d{tuple(d.shape)}")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)):
        raise ValueError(f"sfa must be [k/128, sfa_ld(m)] = {(k // 128, get_sfa_ld(m))}")
    if tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("sfb must be [ceil(n/128), k/128]")
    _check(lib().dg_fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), m, n, k, _stream()))
    return d


def fp8_gemm_nt_noalloc(a_pair, b_pair, d):
    """fp8_gemm_nt for callers that cannot allocate device memory: split-K
    scratch comes from the library's static per-GPU array (calls that
    overlap in time on one GPU race)."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", _FP8, 2)
    _need(b, "b", _FP8, 2)
    _need(d, "d", (torch.bfloat16,), 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or tuple(d.shape) != (m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} b{tuple(b.shape)} d{tuple(d.shape)}")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)) or tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_fp8_gemm_nt_noalloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), m, n, k, _stream()))
    return d


def m_grouped_fp8_gemm_nt_contiguous(a_pair, b_pair, d, m_indices):
    """Contiguous-layout grouped GEMM: row r of a uses expert m_indices[r]'s B."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", _FP8, 2)
    _need(b, "b", _FP8, 3)
    _need(d, "d", (torch.bfloat16,), 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 3)
    _need(m_indices, "m_indices", (torch.int32,), 1)
    m, k = a.shape
    g, n, _ = b.shape
    if b.shape[2] != k or tuple(d.shape) != (m, n) or m_indices.numel() != m:
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)) or tuple(sfb.shape) != (g, (n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_m_grouped_fp8_gemm_nt_contiguous(
        _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(m_indices), m, n, k, g, _stream()))
    return d


def m_grouped_fp8_gemm_nt_masked(a_pair, b_pair, d, masked_m, expected_m=0):
    """Masked-layout grouped GEMM: expert g computes its first masked_m[g] rows."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", _FP8, 3)
    _need(b, "b", _FP8, 3)
    _need(d, "d", (torch.bfloat16,), 3)
    _need(sfa, "sfa", (torch.float32,), 3)
    _need(sfb, "sfb", (torch.float32,), 3)
    _need(masked_m, "masked_m", (torch.int32,), 1)
    g, max_m, k = a.shape
    n = b.shape[1]
    if b.shape[0] != g or b.shape[2] != k or tuple(d.shape) != (g, max_m, n) or masked_m.numel() != g:
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (g, k // 128, get_sfa_ld(max_m)) or tuple(sfb.shape) != (g, (n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_m_grouped_fp8_gemm_nt_masked(
        _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m), g, max_m, n, k,
        int(expected_m), _stream()))
    return d


def m_grouped_fp8_gemm_nt_masked_swiglu(a_pair, b_pair, h_pair, masked_m, expected_m=0):
    """MoE FC1 + SwiGLU on the masked layout: B is [g, 2*inter, k] holding
    each expert's gate rows, then its up rows; h = silu(gate) * up of the
    valid rows is written as e4m3 codes hq [g, max_m, inter] with 1x128 fp32
    scales hs [g, inter/128, get_sfa_ld(max_m)], the A operand layout of the
    masked GEMM."""
    a, sfa = a_pair
    b, sfb = b_pair
    hq, hs = h_pair
    _need(a, "a", _FP8, 3)
    _need(b, "b", _FP8, 3)
    _need(hq, "hq", _FP8, 3)
    _need(sfa, "sfa", (torch.float32,), 3)
    _need(sfb, "sfb", (torch.float32,), 3)
    _need(hs, "hs", (torch.float32,), 3)
    _need(masked_m, "masked_m", (torch.int32,), 1)
    g, max_m, k = a.shape
    inter = b.shape[1] // 2
    if b.shape[0] != g or b.shape[2] != k or b.shape[1] != 2 * inter or masked_m.numel() != g:
        raise ValueError("shape mismatch")
    if tuple(hq.shape) != (g, max_m, inter) or tuple(hs.shape) != (g, inter // 128, get_sfa_ld(max_m)):
        raise ValueError("output shape mismatch")
    if tuple(sfa.shape) != (g, k // 128, get_sfa_ld(max_m)) or tuple(sfb.shape) != (g, (2 * inter + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_m_grouped_fp8_gemm_nt_masked_swiglu(
        _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(hq), _ptr(hs), _ptr(masked_m), g, max_m, inter, k,
        int(expected_m), _stream()))
    return hq, hs


def m_grouped_fp8_gemm_nt_contiguous_swiglu(a_pair, b_pair, h_pair, m_indices):
    """MoE FC1 + SwiGLU on the contiguous layout: B is [g, 2*inter, k] holding
    each expert's gate rows, then its up rows; h = silu(gate) * up of every
    row with a valid tag is written as e4m3 codes hq [m, inter] with 1x128
    fp32 scales hs [inter/128, get_sfa_ld(m)], the A operand layout of the
    contiguous GEMM."""
    a, sfa = a_pair
    b, sfb = b_pair
    hq, hs = h_pair
    _need(a, "a", _FP8, 2)
    _need(b, "b", _FP8, 3)
    _need(hq, "hq", _FP8, 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 3)
    _need(hs, "hs", (torch.float32,), 2)
    _need(m_indices, "m_indices", (torch.int32,), 1)
    m, k = a.shape
    g = b.shape[0]
    inter = b.shape[1] // 2
    if b.shape[2] != k or b.shape[1] != 2 * inter or m_indices.numel() != m:
        raise ValueError("shape mismatch")
    if tuple(hq.shape) != (m, inter) or tuple(hs.shape) != (inter // 128, get_sfa_ld(m)):
        raise ValueError("output shape mismatch")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)) or tuple(sfb.shape) != (g, (2 * inter + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_m_grouped_fp8_gemm_nt_contiguous_swiglu(
        _ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(hq), _ptr(hs), _ptr(m_indices), m, inter, k, g, _stream()))
    return hq, hs


def k_grouped_fp8_gemm_nt(a_pair, b_pair, d, k_sizes):
    """K-grouped GEMM: group g uses the k_sizes[g] K columns after the groups
    before it; d: bf16 [g, m, n], written in place (zero for empty groups)."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", _FP8, 2)
    _need(b, "b", _FP8, 2)
    _need(d, "d", (torch.bfloat16,), 3)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    _need(k_sizes, "k_sizes", (torch.int32,), 1)
    m, k = a.shape
    n = b.shape[0]
    g = k_sizes.numel()
    if b.shape[1] != k or tuple(d.shape) != (g, m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} b{tuple(b.shape)} d{tuple(d.shape)} groups={g}")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)) or tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_k_grouped_fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(k_sizes), g, m, n, k,
                                           _stream()))
    return d


def bf16_gemm_nt(a, b, d):
    """BF16 NT GEMM: d (bf16 [m, n]) = a (bf16 [m, k]) . b (bf16 [n, k])^T, in place."""
    _need(a, "a", (torch.bfloat16,), 2)
    _need(b, "b", (torch.bfloat16,), 2)
    _need(d, "d", (torch.bfloat16,), 2)
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k or tuple(d.shape) != (m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} b{tuple(b.shape)} d{tuple(d.shape)}")
    _check(lib().dg_bf16_gemm_nt(_ptr(a), _ptr(b), _ptr(d), m, n, k, _stream()))
    return d


def quantize_a_1x128(x, q=None, sfa=None):
    """fp32 [m, k] (or [g, m, k]) -> (e4m3 codes, slab-major sfa)."""
    _need(x, "x", (torch.float32,), x.dim())
    if x.dim() == 3:
        g, m, k = x.shape
        q = torch.empty((g, m, k), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
        sfa = empty_sfa(m, k, g, x.device) if sfa is None else sfa
        for i in range(g):
            quantize_a_1x128(x[i], q[i], sfa[i])
        return q, sfa
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
    sfa = empty_sfa(m, k, None, x.device) if sfa is None else sfa
    _need(q, "q", _FP8, 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    if tuple(q.shape) != (m, k) or tuple(sfa.shape) != (k // 128, get_sfa_ld(m)):
        raise ValueError("output shape mismatch")
    _check(lib().dg_quantize_a_1x128(_ptr(x), _ptr(q), _ptr(sfa), m, k, _stream()))
    return q, sfa


def quantize_b_128x128(x, q=None, sfb=None):
    """fp32 [n, k] (or [g, n, k]) -> (e4m3 codes, sfb [.., ceil(n/128), k/128])."""
    _need(x, "x", (torch.float32,), x.dim())
    if x.dim() == 3:
        g, n, k = x.shape
        q = torch.empty((g, n, k), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
        sfb = torch.empty((g, (n + 127) // 128, k // 128), dtype=torch.float32, device=x.device) if sfb is None else sfb
        for i in range(g):
            quantize_b_128x128(x[i], q[i], sfb[i])
        return q, sfb
    n, k = x.shape
    q = torch.empty((n, k), dtype=torch.float8_e4m3fn, device=x.device) if q is None else q
    sfb = torch.empty(((n + 127) // 128, k // 128), dtype=torch.float32, device=x.device) if sfb is None else sfb
    _need(q, "q", _FP8, 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    if tuple(q.shape) != (n, k) or tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("output shape mismatch")
    _check(lib().dg_quantize_b_128x128(_ptr(x), _ptr(q), _ptr(sfb), n, k, _stream()))
    return q, sfb


def fp4_gemm_nt(a_pair, b_pair, d):
    """FP4 NT GEMM: a (uint8 [m, k/2], two e2m1 codes per byte) with sfa
    (slab-major [k/128, get_sfa_ld(m)]), b (uint8 [n, k/2]) with sfb
    ([ceil(n/128), k/128]); d is bf16 [m, n], written in place."""
    a, sfa = a_pair
    b, sfb = b_pair
    _need(a, "a", (torch.uint8,), 2)
    _need(b, "b", (torch.uint8,), 2)
    _need(d, "d", (torch.bfloat16,), 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    m, kh = a.shape
    n = b.shape[0]
    k = 2 * kh
    if b.shape[1] != kh or tuple(d.shape) != (m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} b{tuple(b.shape)} d{tuple(d.shape)}")
    if tuple(sfa.shape) != (k // 128, get_sfa_ld(m)) or tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("scale shape mismatch")
    _check(lib().dg_fp4_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), m, n, k, _stream()))
    return d


def quantize_a_1x128_fp4(x, q=None, sfa=None):
    """fp32 [m, k] -> (packed e2m1 codes uint8 [m, k/2], slab-major sfa)."""
    _need(x, "x", (torch.float32,), 2)
    m, k = x.shape
    q = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device) if q is None else q
    sfa = empty_sfa(m, k, None, x.device) if sfa is None else sfa
    _need(q, "q", (torch.uint8,), 2)
    _need(sfa, "sfa", (torch.float32,), 2)
    if tuple(q.shape) != (m, k // 2) or tuple(sfa.shape) != (k // 128, get_sfa_ld(m)):
        raise ValueError("output shape mismatch")
    _check(lib().dg_quantize_a_1x128_fp4(_ptr(x), _ptr(q), _ptr(sfa), m, k, _stream()))
    return q, sfa


def quantize_b_128x128_fp4(x, q=None, sfb=None):
    """fp32 [n, k] -> (packed e2m1 codes uint8 [n, k/2], sfb [ceil(n/128), k/128])."""
    _need(x, "x", (torch.float32,), 2)
    n, k = x.shape
    q = torch.empty((n, k // 2), dtype=torch.uint8, device=x.device) if q is None else q
    sfb = torch.empty(((n + 127) // 128, k // 128), dtype=torch.float32, device=x.device) if sfb is None else sfb
    _need(q, "q", (torch.uint8,), 2)
    _need(sfb, "sfb", (torch.float32,), 2)
    if tuple(q.shape) != (n, k // 2) or tuple(sfb.shape) != ((n + 127) // 128, k // 128):
        raise ValueError("output shape mismatch")
    _check(lib().dg_quantize_b_128x128_fp4(_ptr(x), _ptr(q), _ptr(sfb), n, k, _stream()))
    return q, sfb


_W4_FORMATS = {"e2m1": 0, "u4": 1}


def _w4_shape(b_triple):
    """(codes, scales, zeros, n, k, group, format) of a W4 triple, checked."""
    codes, scales, zeros = b_triple
    _need(codes, "codes", (torch.uint8,), 2)
    _need(scales, "scales", (torch.bfloat16,), 2)
    n, kh = codes.shape
    rows, groups = scales.shape
    if groups < 1 or rows != n or 2 * kh % groups:
        raise ValueError(f"scales {tuple(scales.shape)} do not fit codes {tuple(codes.shape)}")
    if zeros is not None:
        _need(zeros, "zeros", (torch.uint8,), 2)
        if zeros.shape != scales.shape:
            raise ValueError(f"zeros {tuple(zeros.shape)} do not fit scales {tuple(scales.shape)}")
    return codes, scales, zeros, n, 2 * kh, 2 * kh // groups, 0 if zeros is None else 1


def bf16_w4_gemm_nt(a, b_triple, d):
    """d (bf16 [m, n], in place) = a (bf16 [m, k]) . w^T for 4-bit weights
    w = scales * (codes - zeros), b_triple = (codes, scales, zeros or None)."""
    _need(a, "a", (torch.bfloat16,), 2)
    _need(d, "d", (torch.bfloat16,), 2)
    codes, scales, zeros, n, k, group, fmt = _w4_shape(b_triple)
    m, ka = a.shape
    if ka != k or d.shape != (m, n):
        raise ValueError(f"shape mismatch a{tuple(a.shape)} w({n}, {k}) d{tuple(d.shape)}")
    _check(lib().dg_bf16_w4_gemm_nt(a.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                    None if zeros is None else zeros.data_ptr(), d.data_ptr(), m, n, k, group, fmt,
                                    _stream()))
    return d


def bf16_w4_workspace_size(m, n, k, group=128, fmt="e2m1"):
    """Bytes of a stream's workspace that bf16_w4_gemm_nt takes for a shape;
    give it to reserve_workspace before capturing such calls."""
    if fmt not in _W4_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_W4_FORMATS)}")
    size = ctypes.c_size_t(0)
    _check(lib().dg_bf16_w4_workspace_size(int(m), int(n), int(k), int(group), _W4_FORMATS[fmt], ctypes.byref(size)))
    return size.value


def quantize_b_w4(x, fmt="e2m1", group=128):
    """bf16 or fp32 weights [n, k] -> (codes, scales, zeros or None), fmt "e2m1" or "u4"."""
    _need(x, "x", (torch.bfloat16, torch.float32), 2)
    if fmt not in _W4_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_W4_FORMATS)}")
    n, k = x.shape
    if group not in (32, 64, 128) or k < group or k % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide k = {k}, got {group}")
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((n, k // group), dtype=torch.bfloat16, device=x.device)
    zeros = torch.empty((n, k // group), dtype=torch.uint8, device=x.device) if fmt == "u4" else None
    _check(lib().dg_quantize_b_w4(x.data_ptr(), int(x.dtype == torch.bfloat16), codes.data_ptr(), scales.data_ptr(),
                                  None if zeros is None else zeros.data_ptr(), n, k, group, _W4_FORMATS[fmt], _stream()))
    return codes, scales, zeros


def dequantize_b_w4(b_triple, w=None):
    """(codes, scales, zeros or None) -> the bf16 weights [n, k] they stand for."""
    codes, scales, zeros, n, k, group, fmt = _w4_shape(b_triple)
    w = torch.empty((n, k), dtype=torch.bfloat16, device=codes.device) if w is None else w
    _need(w, "w", (torch.bfloat16,), 2)
    if tuple(w.shape) != (n, k):
        raise ValueError(f"w must be {(n, k)}, got {tuple(w.shape)}")
    _check(lib().dg_dequantize_b_w4(codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
                                    w.data_ptr(), n, k, group, fmt, _stream()))
    return w


def empty_kv8_cache(num_blocks, h_kv, d, block=64, device="cuda"):
    """An 8-bit key/value cache of num_blocks blocks of `block` tokens."""
    return (torch.empty((num_blocks, h_kv, block, d), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((num_blocks, h_kv, d, block), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((num_blocks, h_kv), dtype=torch.float32, device=device),
            torch.empty((num_blocks, h_kv), dtype=torch.float32, device=device))


def _kv8_shape(cache, block_table, lens, cu):
    """(num_blocks, h_kv, block, d, batch, max_blocks) of a cache and its tables, checked."""
    k_codes, v_codes, k_scales, v_scales = cache
    _need(k_codes, "k_codes", _FP8, 4)
    _need(v_codes, "v_codes", _FP8, 4)
    _need(k_scales, "k_scales", (torch.float32,), 2)
    _need(v_scales, "v_scales", (torch.float32,), 2)
    _need(block_table, "block_table", (torch.int32,), 2)
    _need(lens, "lens", (torch.int32,), 1)
    _need(cu, "cu", (torch.int32,), 1)
    num_blocks, h_kv, block, d = k_codes.shape
    per_head = (num_blocks, h_kv)
    if v_codes.shape != (num_blocks, h_kv, d, block) or k_scales.shape != per_head or v_scales.shape != per_head:
        raise ValueError("cache shape mismatch")
    batch, max_blocks = block_table.shape
    if lens.shape[0] != batch or cu.shape[0] != batch + 1:
        raise ValueError("the block table, the lengths and cu (batch + 1) disagree on the batch")
    return num_blocks, h_kv, block, d, batch, max_blocks


def _packed(x, name, heads, d):
    """Checks bf16 [total, heads, d] with packed heads; returns (total, elements from token to token)."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 3 or not x.is_cuda:
        raise TypeError(f"{name} must be a bf16 device tensor [tokens, heads, d]")
    total, h, dim = x.shape
    if h != heads or dim != d:
        raise ValueError(f"{name} must be [tokens, {heads}, {d}], got {tuple(x.shape)}")
    stride, s1, s2 = x.stride()
    if (s2 != 1 and d > 1) or (s1 != d and heads > 1):
        raise ValueError(f"the heads of a token of {name} must lie packed")
    return total, stride if total > 1 else heads * d


def kv8_append(k, v, cache, block_table, ctx_lens, cu_new, max_new):
    """Append packed new keys and values (bf16 [total, h_kv, d]; slices of a
    wider projection serve) behind the ctx_lens[i] cached tokens of each
    sequence, in place.  cu_new: int32 [batch + 1] running sums of the new
    tokens; max_new: the most of one sequence."""
    num_blocks, h_kv, block, d, batch, max_blocks = _kv8_shape(cache, block_table, ctx_lens, cu_new)
    total, ks = _packed(k, "k", h_kv, d)
    total_v, vs = _packed(v, "v", h_kv, d)
    if total != total_v:
        raise ValueError(f"k holds {total} tokens, v {total_v}")
    k_codes, v_codes, k_scales, v_scales = cache
    _check(lib().dg_kv8_append(k.data_ptr(), ks, v.data_ptr(), vs, k_codes.data_ptr(), v_codes.data_ptr(),
                               k_scales.data_ptr(), v_scales.data_ptr(), block_table.data_ptr(), ctx_lens.data_ptr(),
                               cu_new.data_ptr(), batch, total, max_new, h_kv, d, block, num_blocks, max_blocks,
                               _stream()))
    return cache


def kv8_attention(q, cache, block_table, kv_lens, cu_q, max_q, out, lse=None, scale=None, causal=True, window=0):
    """Attention of packed queries (bf16 [total, h_q, d]) over the cache; out
    bf16 [total, h_q, d] and lse fp32 [total, h_q] (or None) are written in
    place.  kv_lens counts the queries' own tokens; cu_q: int32 [batch + 1]
    running sums of the queries; max_q: the most of one sequence; scale:
    d ** -0.5 if None; window: the last so many tokens only (0: all)."""
    num_blocks, h_kv, block, d, batch, max_blocks = _kv8_shape(cache, block_table, kv_lens, cu_q)
    _need(out, "out", (torch.bfloat16,), 3)
    h_q = out.shape[1]
    total, stride = _packed(q, "q", h_q, d)
    if out.shape != (total, h_q, d):
        raise ValueError(f"out must be {tuple(q.shape)}, got {tuple(out.shape)}")
    if lse is not None:
        _need(lse, "lse", (torch.float32,), 2)
        if lse.shape != (total, h_q):
            raise ValueError(f"lse must be {(total, h_q)}, got {tuple(lse.shape)}")
    k_codes, v_codes, k_scales, v_scales = cache
    _check(lib().dg_kv8_attention(q.data_ptr(), stride, k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                  v_scales.data_ptr(), block_table.data_ptr(), kv_lens.data_ptr(), cu_q.data_ptr(),
                                  out.data_ptr(), None if lse is None else lse.data_ptr(),
                                  d ** -0.5 if scale is None else scale, causal, window, batch, total, max_q, h_q,
                                  h_kv, d, block, num_blocks, max_blocks, _stream()))
    return out


def kv8_attention_workspace_size(d):
    """Bytes of a stream's workspace that kv8_attention takes; give it to
    reserve_workspace before capturing such calls."""
    size = ctypes.c_size_t(0)
    _check(lib().dg_kv8_attention_workspace_size(int(d), ctypes.byref(size)))
    return size.value
