"""Python binding of ``libchipmunk.so`` (the C ABI in include/chipmunk.h).

Argument marshalling only: each function checks dtypes, shapes and devices of
the torch tensors it is given, passes their device pointers and the current
CUDA stream to the C entry point of the same name, and raises
``ChipmunkError`` on a non-zero status. Every step runs in the library's CUDA
kernels; there is no fallback. If the library is missing or cannot be loaded
the first call raises.

Layouts (all tensors on the same CUDA device, contiguous):

* MLP: x [T][D] bf16, w1t [H][D] bf16 (W1 transposed), b1 [H] bf16,
  w2 [H][D] bf16, b2 [D] bf16, idx [nb][k] int32, a_cache [nb][H][Bt] bf16,
  y_cache [T][D] fp32, out [T][D] bf16.
* Attention: q, k, v [T][h][128] bf16, idx [h][nb][k] int32, m_c, l_c [h][T]
  fp32, acc_c [h][T][128] fp32, o [T][h][128] bf16.
* Around them: 4-bit microscaled rows (``Fp4Rows``), ``linear_fp4`` x [T][K] or
  quantised, w [N][K] quantised, ``norm_residual`` res, y [T][D] with gate, scale,
  shift [B][D] (row-strided views of one projection are fine), ``qk_norm_rope``
  qkv [T][>= 3 h 128] (row-strided) to q, k, v [T][h][128].
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libchipmunk.so")

OK = 0
ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGNMENT, ERR_CUDA, ERR_DEVICE, ERR_UNSUPPORTED, ERR_WORKSPACE = 1, 2, 3, 4, 5, 6, 7
OP_TOPK, OP_MLP_DELTA, OP_ATTN_DELTA, OP_REFRESH, OP_MLP_DELTA_FP8, OP_LINEAR_FP4 = 0, 1, 2, 3, 4, 5
REFRESH_MLP, REFRESH_ATTN = 0, 1

EXPORTS = (
    "chipmunk_topk_cols", "chipmunk_mlp_delta", "chipmunk_mlp_delta_up", "chipmunk_mlp_delta_down",
    "chipmunk_attn_delta", "chipmunk_dense_refresh",
    "chipmunk_gather_cols", "chipmunk_scatter_cols", "chipmunk_workspace_bytes", "chipmunk_status_string",
    "chipmunk_last_error", "chipmunk_read_device_status", "chipmunk_version", "chipmunk_mlp_delta_noalloc",
    "chipmunk_selftest_bounded_wait", "chipmunk_mlp_delta_fp8", "chipmunk_quantize_e4m3_rows",
    "chipmunk_fp4_scale_bytes", "chipmunk_quantize_fp4_rows", "chipmunk_dequantize_fp4_rows", "chipmunk_linear_fp4",
    "chipmunk_norm_residual", "chipmunk_qk_norm_rope", "chipmunk_selftest_linear_fp4_form",
)
NOALLOC_SCRATCH_BYTES = 64 << 20


class ChipmunkError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"chipmunk status {status}: {message}")
        self.status = status


class MlpArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("H", ctypes.c_int64),
        ("Bt", ctypes.c_int32), ("k", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("w1t", ctypes.c_void_p), ("b1", ctypes.c_void_p),
        ("w2", ctypes.c_void_p), ("b2", ctypes.c_void_p), ("idx", ctypes.c_void_p),
        ("a_cache", ctypes.c_void_p), ("y_cache", ctypes.c_void_p), ("out", ctypes.c_void_p),
    ]


class MlpFp8Args(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("H", ctypes.c_int64),
        ("Bt", ctypes.c_int32), ("k", ctypes.c_int32),
        ("x8", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("w1t8", ctypes.c_void_p), ("s1", ctypes.c_void_p),
        ("b1", ctypes.c_void_p), ("w2_8", ctypes.c_void_p), ("g2", ctypes.c_void_p), ("s_delta", ctypes.c_float),
        ("idx", ctypes.c_void_p), ("a_cache", ctypes.c_void_p), ("y_cache", ctypes.c_void_p), ("out", ctypes.c_void_p),
    ]


class AttnArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("h", ctypes.c_int32), ("d", ctypes.c_int32),
        ("Bt", ctypes.c_int32), ("k", ctypes.c_int32), ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("kk", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("idx", ctypes.c_void_p), ("m_c", ctypes.c_void_p), ("l_c", ctypes.c_void_p),
        ("acc_c", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("cache_format", ctypes.c_int32), ("lse_c", ctypes.c_void_p), ("o_c", ctypes.c_void_p),
    ]


class RefreshArgs(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("first_step", ctypes.c_int32),
        ("mlp", MlpArgs), ("attn", AttnArgs), ("scores", ctypes.c_void_p),
    ]


class Fp4Args(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("format", ctypes.c_int32),
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("row_scales", ctypes.c_void_p),
    ]


class LinearFp4Args(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("N", ctypes.c_int64), ("act", ctypes.c_int32), ("out_type", ctypes.c_int32),
        ("x", ctypes.c_void_p), ("xq", Fp4Args), ("w", Fp4Args), ("bias", ctypes.c_void_p), ("out", ctypes.c_void_p),
    ]


class NormArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("D", ctypes.c_int64), ("B", ctypes.c_int64),
        ("res_type", ctypes.c_int32), ("y_type", ctypes.c_int32), ("mod_type", ctypes.c_int32),
        ("post_norm", ctypes.c_int32), ("norm", ctypes.c_int32), ("out_format", ctypes.c_int32),
        ("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
        ("res", ctypes.c_void_p), ("y", ctypes.c_void_p), ("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
        ("res_out", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p), ("ld_mod", ctypes.c_int64),
        ("offsets", ctypes.c_void_p), ("out", ctypes.c_void_p), ("out_scales", ctypes.c_void_p),
        ("out_row_scales", ctypes.c_void_p),
    ]


class HeadsArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("ld", ctypes.c_int64), ("h", ctypes.c_int32), ("pairs", ctypes.c_int32),
        ("eps", ctypes.c_float), ("qkv", ctypes.c_void_p), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
    ]


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads the shared library once (raises if it is missing)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise ChipmunkError(6, f"{path} not found: build it with `python -m dynamic_column_sparse_b200.build`")
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        sig = {
            "chipmunk_topk_cols": [vp, i64, i64, i64, i32, vp, i64, vp, sz, vp],
            "chipmunk_mlp_delta": [ctypes.POINTER(MlpArgs), vp, sz, vp],
            "chipmunk_mlp_delta_up": [ctypes.POINTER(MlpArgs), vp, sz, vp],
            "chipmunk_mlp_delta_down": [ctypes.POINTER(MlpArgs), vp, sz, vp],
            "chipmunk_attn_delta": [ctypes.POINTER(AttnArgs), vp, sz, vp],
            "chipmunk_dense_refresh": [ctypes.POINTER(RefreshArgs), vp, sz, vp],
            "chipmunk_gather_cols": [vp, i64, i64, i32, vp, i32, vp, vp],
            "chipmunk_scatter_cols": [vp, i64, i64, i32, vp, i32, vp, vp],
            "chipmunk_read_device_status": [ctypes.POINTER(i32), vp],
            "chipmunk_mlp_delta_noalloc": [ctypes.POINTER(MlpArgs), vp],
            "chipmunk_selftest_bounded_wait": [vp],
            "chipmunk_mlp_delta_fp8": [ctypes.POINTER(MlpFp8Args), vp, sz, vp],
            "chipmunk_quantize_e4m3_rows": [vp, i64, i64, vp, vp, vp],
            "chipmunk_quantize_fp4_rows": [vp, ctypes.POINTER(Fp4Args), vp],
            "chipmunk_dequantize_fp4_rows": [ctypes.POINTER(Fp4Args), i32, vp, vp],
            "chipmunk_linear_fp4": [ctypes.POINTER(LinearFp4Args), vp, sz, vp],
            "chipmunk_norm_residual": [ctypes.POINTER(NormArgs), vp],
            "chipmunk_qk_norm_rope": [ctypes.POINTER(HeadsArgs), vp],
            "chipmunk_selftest_linear_fp4_form": [i64, i64, i64, i32],
        }
        for name, argtypes in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = argtypes
            fn.restype = i32
        lib.chipmunk_workspace_bytes.argtypes = [i32, vp]
        lib.chipmunk_workspace_bytes.restype = sz
        lib.chipmunk_fp4_scale_bytes.argtypes = [i64, i64, i32]
        lib.chipmunk_fp4_scale_bytes.restype = sz
        lib.chipmunk_status_string.argtypes = [i32]
        lib.chipmunk_status_string.restype = ctypes.c_char_p
        lib.chipmunk_last_error.argtypes = []
        lib.chipmunk_last_error.restype = ctypes.c_char_p
        lib.chipmunk_version.argtypes = []
        lib.chipmunk_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(st: int):
    if st != OK:
        lib = load_library()
        raise ChipmunkError(st, f"{lib.chipmunk_status_string(st).decode()}: {lib.chipmunk_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def version() -> str:
    return load_library().chipmunk_version().decode()


def workspace_bytes(op: int, args=None) -> int:
    lib = load_library()
    return int(lib.chipmunk_workspace_bytes(op, None if args is None else ctypes.byref(args)))


def read_device_status(stream=None) -> int:
    lib = load_library()
    v = ctypes.c_int32(0)
    st = lib.chipmunk_read_device_status(ctypes.byref(v), _stream(stream))
    if st not in (OK, ERR_DEVICE):
        _check(st)
    return int(v.value)


# ------------------------------------------------------------------ top-k

def topk_cols(scores: torch.Tensor, k: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """k largest fp32 scores of each row (ties to the lower index) as ascending int32 indices."""
    lib = load_library()
    _need(scores, "scores", torch.float32)
    if scores.dim() != 2:
        raise ValueError("scores must be 2-D [rows][n]")
    rows, n = scores.shape
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=scores.device)
    _need(out, "out", torch.int32, (rows, k))
    _check(lib.chipmunk_topk_cols(_ptr(scores), rows, n, n, k, _ptr(out), k, None, 0, _stream(stream)))
    return out


# ------------------------------------------------------------------ MLP

def _mlp_args(x, w1t, b1, w2, b2, idx, a_cache, y_cache, out, Bt, k):
    T, D = x.shape
    H = w1t.shape[0]
    nb = (T + Bt - 1) // Bt
    _need(x, "x", torch.bfloat16, (T, D))
    _need(w1t, "w1t", torch.bfloat16, (H, D))
    _need(b1, "b1", torch.bfloat16, (H,))
    _need(w2, "w2", torch.bfloat16, (H, D))
    if b2 is not None:
        _need(b2, "b2", torch.bfloat16, (D,))
    if idx is not None:
        _need(idx, "idx", torch.int32, (nb, k))
    _need(a_cache, "a_cache", torch.bfloat16, (nb, H, Bt))
    _need(y_cache, "y_cache", torch.float32, (T, D))
    if out is not None:
        _need(out, "out", torch.bfloat16, (T, D))
    return MlpArgs(T, D, H, Bt, k, x.data_ptr(), w1t.data_ptr(), b1.data_ptr(), w2.data_ptr(),
                   0 if b2 is None else b2.data_ptr(), 0 if idx is None else idx.data_ptr(),
                   a_cache.data_ptr(), y_cache.data_ptr(), 0 if out is None else out.data_ptr())


def mlp_workspace_bytes(T: int, H: int, k: int, Bt: int = 128) -> int:
    a = MlpArgs(T, 64, H, Bt, k)
    return workspace_bytes(OP_MLP_DELTA, a)


def mlp_delta(x, w1t, b1, w2, idx, a_cache, y_cache, out=None, Bt=128, workspace=None, stream=None, part=None):
    """Sparse MLP step: recompute the selected columns, update a_cache / y_cache in place, write out.

    ``part`` = "up" or "down" runs only that kernel (chipmunk_mlp_delta_up /
    _down); both need the same workspace.
    """
    lib = load_library()
    k = idx.shape[1]
    a = _mlp_args(x, w1t, b1, w2, None, idx, a_cache, y_cache, out, Bt, k)
    need = workspace_bytes(OP_MLP_DELTA, a)
    if need and workspace is None:
        if part is not None:
            raise ValueError("a split MLP step needs an explicit workspace shared by both parts")
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = {None: lib.chipmunk_mlp_delta, "up": lib.chipmunk_mlp_delta_up, "down": lib.chipmunk_mlp_delta_down}[part]
    _check(fn(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def mlp_delta_noalloc(x, w1t, b1, w2, idx, a_cache, y_cache, out=None, Bt=128, stream=None):
    """mlp_delta without caller scratch: for callers that cannot allocate device
    memory. The library's fixed 64 MiB scratch array (reserved on a device at
    this call's first use there) is shared by every call, so calls must not
    overlap on the GPU; larger problems raise with status ERR_WORKSPACE."""
    lib = load_library()
    a = _mlp_args(x, w1t, b1, w2, None, idx, a_cache, y_cache, out, Bt, idx.shape[1])
    _check(lib.chipmunk_mlp_delta_noalloc(ctypes.byref(a), _stream(stream)))
    return out


def mlp_refresh(x, w1t, b1, w2, b2, a_cache, y_cache, idx, scores, out=None, Bt=128, first_step=False, stream=None):
    """Dense MLP step: rebuild a_cache / y_cache, write the column scores and the new selection idx."""
    lib = load_library()
    k = idx.shape[1]
    a = _mlp_args(x, w1t, b1, w2, b2, idx, a_cache, y_cache, out, Bt, k)
    _need(scores, "scores", torch.float32, (a_cache.shape[0], w1t.shape[0]))
    r = RefreshArgs(REFRESH_MLP, 1 if first_step else 0, a, AttnArgs(), scores.data_ptr())
    _check(lib.chipmunk_dense_refresh(ctypes.byref(r), None, 0, _stream(stream)))
    return out


# ------------------------------------------------------------------ FP8 MLP step

def _need_codes(t, name, shape):
    """e4m3 codes: torch.uint8 or torch.float8_e4m3fn storage."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def quantize_e4m3_rows(x, codes=None, scales=None, stream=None):
    """Rows of bf16 x [R][C] to e4m3 codes [R][C] (uint8) and per-row fp32 scales [R]: x ~ scale * code."""
    lib = load_library()
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    R, C = x.shape
    if codes is None:
        codes = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((R,), dtype=torch.float32, device=x.device)
    _need_codes(codes, "codes", (R, C))
    _need(scales, "scales", torch.float32, (R,))
    _check(lib.chipmunk_quantize_e4m3_rows(_ptr(x), R, C, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def mlp_fp8_workspace_bytes(T: int, H: int, k: int) -> int:
    return workspace_bytes(OP_MLP_DELTA_FP8, MlpFp8Args(T, 256, H, 128, k))


def mlp_delta_fp8(x8, sx, w1t8, s1, b1, w2_8, g2, s_delta, idx, a_cache, y_cache, out=None, workspace=None,
                  stream=None):
    """FP8 form of the sparse MLP step (chipmunk_mlp_delta_fp8): e4m3 operands with per-token (sx),
    per-hidden-unit (s1) scales, deltas rounded to e4m3 after multiplying by g2 = s2 / s_delta."""
    lib = load_library()
    T, D = x8.shape
    H = w1t8.shape[0]
    nb = (T + 127) // 128
    k = idx.shape[1]
    _need_codes(x8, "x8", (T, D))
    _need(sx, "sx", torch.float32, (T,))
    _need_codes(w1t8, "w1t8", (H, D))
    _need(s1, "s1", torch.float32, (H,))
    _need(b1, "b1", torch.bfloat16, (H,))
    _need_codes(w2_8, "w2_8", (H, D))
    _need(g2, "g2", torch.float32, (H,))
    _need(idx, "idx", torch.int32, (nb, k))
    _need(a_cache, "a_cache", torch.bfloat16, (nb, H, 128))
    _need(y_cache, "y_cache", torch.float32, (T, D))
    if out is not None:
        _need(out, "out", torch.bfloat16, (T, D))
    a = MlpFp8Args(T, D, H, 128, k, x8.data_ptr(), sx.data_ptr(), w1t8.data_ptr(), s1.data_ptr(), b1.data_ptr(),
                   w2_8.data_ptr(), g2.data_ptr(), float(s_delta), idx.data_ptr(), a_cache.data_ptr(),
                   y_cache.data_ptr(), 0 if out is None else out.data_ptr())
    need = workspace_bytes(OP_MLP_DELTA_FP8, a)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x8.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.chipmunk_mlp_delta_fp8(ctypes.byref(a), _ptr(workspace), ws_bytes, _stream(stream)))
    return out


# ------------------------------------------------------------------ attention

ATTN_CACHE_PARTIAL = 0
ATTN_CACHE_COMPACT = 1


def _attn_args(q, k, v, idx, m_c, l_c, acc_c, o, scale, kk, lse_c=None, o_c=None):
    """Partial-form cache (m_c, l_c, acc_c) or, with lse_c / o_c given, the compact form."""
    T, h, d = q.shape
    nb = (T + 127) // 128
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _need(t, name, torch.bfloat16, (T, h, d))
    _need(idx, "idx", torch.int32, (h, nb, kk))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lse_c is not None:
        _need(lse_c, "lse_c", torch.float32, (h, T))
        _need(o_c, "o_c", torch.bfloat16, (h, T, d))
        return AttnArgs(T, h, d, 128, kk, float(scale), q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(),
                        None, None, None, o.data_ptr(), ATTN_CACHE_COMPACT, lse_c.data_ptr(), o_c.data_ptr())
    _need(m_c, "m_c", torch.float32, (h, T))
    _need(l_c, "l_c", torch.float32, (h, T))
    _need(acc_c, "acc_c", torch.float32, (h, T, d))
    return AttnArgs(T, h, d, 128, kk, float(scale), q.data_ptr(), k.data_ptr(), v.data_ptr(), idx.data_ptr(),
                    m_c.data_ptr(), l_c.data_ptr(), acc_c.data_ptr(), o.data_ptr(), ATTN_CACHE_PARTIAL, None, None)


def attn_delta(q, k, v, idx, m_c, l_c, acc_c, o, scale=None, stream=None):
    """Sparse attention step: selected keys recomputed, merged with the cached complement partial into o."""
    lib = load_library()
    a = _attn_args(q, k, v, idx, m_c, l_c, acc_c, o, scale, idx.shape[2])
    _check(lib.chipmunk_attn_delta(ctypes.byref(a), None, 0, _stream(stream)))
    return o


def attn_delta_compact(q, k, v, idx, lse_c, o_c, o, scale=None, stream=None):
    """Sparse attention step against the compact complement cache (lse_c fp32 [h][T], o_c bf16 [h][T][d])."""
    lib = load_library()
    a = _attn_args(q, k, v, idx, None, None, None, o, scale, idx.shape[2], lse_c=lse_c, o_c=o_c)
    _check(lib.chipmunk_attn_delta(ctypes.byref(a), None, 0, _stream(stream)))
    return o


def attn_refresh_workspace_bytes(T: int, h: int, k: int, keep_mass: bool) -> int:
    """Workspace of an attention refresh: the row log-sum-exp, plus the fused mass/top-k kernel's row
    buffers when the mass is not kept (``scores=None``)."""
    a = AttnArgs(T, h, 128, 128, k, 1.0)
    return workspace_bytes(OP_REFRESH, RefreshArgs(REFRESH_ATTN, 0, MlpArgs(), a, 16 if keep_mass else None))


def attn_refresh(q, k, v, idx, m_c, l_c, acc_c, o, scores=None, scale=None, workspace=None, stream=None, lse_c=None,
                 o_c=None):
    """Dense attention step: o, new selection idx and the complement cache (partial form m_c, l_c, acc_c;
    or, with lse_c and o_c given and m_c, l_c, acc_c None, the compact form). With ``scores`` [h][nb][T]
    fp32 the attention mass is also written there; without it the mass stays in the workspace's row
    buffers (the top-k is taken on it inside the mass kernel)."""
    lib = load_library()
    a = _attn_args(q, k, v, idx, m_c, l_c, acc_c, o, scale, idx.shape[2], lse_c=lse_c, o_c=o_c)
    T, h = q.shape[0], q.shape[1]
    if scores is not None:
        _need(scores, "scores", torch.float32, (h, (T + 127) // 128, T))
    r = RefreshArgs(REFRESH_ATTN, 0, MlpArgs(), a, None if scores is None else scores.data_ptr())
    need = workspace_bytes(OP_REFRESH, r)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.chipmunk_dense_refresh(ctypes.byref(r), _ptr(workspace), ws_bytes, _stream(stream)))
    return o


# ------------------------------------------------------------------ cache columns

def gather_cols(a_cache, idx, packed=None, stream=None):
    """packed[b][j] = a_cache[b][idx[b][j]] (each a run of Bt bf16)."""
    lib = load_library()
    nb, H, Bt = a_cache.shape
    k = idx.shape[1]
    _need(a_cache, "a_cache", torch.bfloat16)
    _need(idx, "idx", torch.int32, (nb, k))
    if packed is None:
        packed = torch.empty((nb, k, Bt), dtype=torch.bfloat16, device=a_cache.device)
    _need(packed, "packed", torch.bfloat16, (nb, k, Bt))
    _check(lib.chipmunk_gather_cols(_ptr(a_cache), nb, H, Bt, _ptr(idx), k, _ptr(packed), _stream(stream)))
    return packed


def scatter_cols(packed, idx, a_cache, stream=None):
    """a_cache[b][idx[b][j]] = packed[b][j]."""
    lib = load_library()
    nb, H, Bt = a_cache.shape
    k = idx.shape[1]
    _need(a_cache, "a_cache", torch.bfloat16)
    _need(idx, "idx", torch.int32, (nb, k))
    _need(packed, "packed", torch.bfloat16, (nb, k, Bt))
    _check(lib.chipmunk_scatter_cols(_ptr(packed), nb, H, Bt, _ptr(idx), k, _ptr(a_cache), _stream(stream)))
    return a_cache


# ------------------------------------------------------------------ around the sparse layers

NVFP4, MXFP4 = 0, 1
_FP4_FORMATS = {"nvfp4": NVFP4, "mxfp4": MXFP4}
_ACTS = {"none": 0, "gelu": 1}
_NORMS = {"none": 0, "layer": 1, "rms": 2}
_NORM_OUT = {"bf16": 0, "e4m3": 1, "nvfp4": 2, "mxfp4": 3}
_PAIRS = {"interleaved": 0, "halves": 1}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _pick(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(str, table))}, got {key!r}") from None


_BF16, _F32, _U8, _I32 = ((t,) for t in (torch.bfloat16, torch.float32, torch.uint8, torch.int32))
_BF16_F32 = (torch.bfloat16, torch.float32)


def _device_of(t, name, dtypes) -> int:
    """Ordinal of the CUDA device of a 2-D tensor of one of ``dtypes``."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return dev


def _here(t, name, dtypes, shape, dev) -> int:
    """Address of a contiguous tensor of one of ``dtypes`` and of ``shape`` on device ordinal ``dev``."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on CUDA device {dev}, is on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


_DEVICES = [torch.device("cuda", i) for i in range(64)]


def _empty(shape, dtype, dev, stream):
    """Uninitialised memory on device ordinal ``dev`` that belongs to the stream that will use it. (Sizes one by
    one: a tuple of them costs torch.empty almost a microsecond more.)"""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=_DEVICES[dev])
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=_DEVICES[dev])


# the current stream's handle without building a Stream object (microseconds, on every call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev, stream, fn, *args):
    """Runs a C entry point (stream last) with device ordinal ``dev`` current, on ``stream`` or dev's current stream."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on CUDA device {dev}")
    else:
        handle = stream.cuda_stream
    if dev == _current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != OK:
        _check(st)


def _fp4_sizes(rows, cols, fmt):
    """(format, bytes of codes, of block scales, of row scales) of rows x cols 4-bit values, each from a
    256-byte boundary when laid one after the other."""
    f = _FP4_FORMATS.get(fmt)
    if f is None:
        f = _pick(_FP4_FORMATS, fmt, "fmt")
    if not 0 <= rows <= 1 << 30 or not 32 <= cols <= 65536 or cols % 32:
        raise ValueError(f"{rows} rows x {cols} columns: columns must be a multiple of 32 in [32, 65536]")
    tiles = (rows + 127 >> 7) * (cols + 255 >> 8)
    if f == NVFP4:
        return f, (rows * (cols >> 1) + 255) & -256, tiles << 11, (rows * 4 + 255) & -256
    return f, (rows * (cols >> 1) + 255) & -256, tiles << 10, 0


class Fp4Rows:
    """Rows of 4-bit microscaled values: ``codes`` uint8 [rows][cols / 2] (lower column in the low
    nibble), ``scales`` uint8 (block scales in the tensor core's order, ``fp4_scale_bytes`` of
    them), ``row_scales`` fp32 [rows] (nvfp4; None for mxfp4): powers of two out of ``quantize_fp4_rows``, any
    scale from 2^-110 to 2^117 in rows made elsewhere (a tensor's one scale, repeated). The header of
    the C ABI defines both formats and the order of the block scales."""

    __slots__ = ("_codes", "_scales", "_row_scales", "_buf", "fmt", "rows", "cols", "device_index", "args")

    def __init__(self, codes, scales, row_scales, fmt, rows, cols):
        f, _, n, _ = _fp4_sizes(rows, cols, fmt)
        if not isinstance(codes, torch.Tensor):
            raise TypeError("codes must be a torch.Tensor")
        dev = codes.get_device()
        if dev < 0:
            raise ValueError("codes must be on a CUDA device")
        if not isinstance(scales, torch.Tensor) or scales.numel() != n:
            raise ValueError(f"scales must hold {n} bytes")
        if f == MXFP4 and row_scales is not None:
            raise ValueError("mxfp4 rows have no row scales")
        self.args = Fp4Args(rows, cols, f, _here(codes, "codes", _U8, (rows, cols // 2), dev),
                            _here(scales, "scales", _U8, scales.shape, dev),
                            _here(row_scales, "row_scales", _F32, (rows,), dev) if f == NVFP4 else None)
        self._codes, self._scales, self._row_scales, self._buf = codes, scales, row_scales, None
        self.fmt, self.rows, self.cols, self.device_index = fmt, rows, cols, dev

    @classmethod
    def _empty(cls, rows, cols, fmt, dev, stream):
        """Uninitialised rows in one allocation; the tensors over its parts are made when asked for."""
        f, codes, scales, rs = _fp4_sizes(rows, cols, fmt)
        q = cls.__new__(cls)
        q._buf = _empty((codes + scales + rs,), torch.uint8, dev, stream)
        q._codes = q._scales = q._row_scales = None
        q.fmt, q.rows, q.cols, q.device_index = fmt, rows, cols, dev
        at = q._buf.data_ptr()
        q.args = Fp4Args(rows, cols, f, at, at + codes, at + codes + scales if f == NVFP4 else None)
        return q

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buf[:self.rows * (self.cols // 2)].view(self.rows, self.cols // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            _, c, n, _ = _fp4_sizes(self.rows, self.cols, self.fmt)
            self._scales = self._buf[c:c + n]
        return self._scales

    @property
    def row_scales(self):
        if self._row_scales is None and self.fmt == "nvfp4":
            _, c, n, _ = _fp4_sizes(self.rows, self.cols, self.fmt)
            self._row_scales = self._buf[c + n:c + n + 4 * self.rows].view(torch.float32)
        return self._row_scales

    @property
    def device(self):
        return _DEVICES[self.device_index]


def fp4_scale_bytes(rows: int, cols: int, fmt: str) -> int:
    """Bytes of the block scales of rows x cols 4-bit values."""
    return _fp4_sizes(rows, cols, fmt)[2]


def empty_fp4_rows(rows: int, cols: int, fmt: str, device, stream=None) -> Fp4Rows:
    """Uninitialised 4-bit rows for a quantising call to fill."""
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"device must be a CUDA device, got {dev}")
    return Fp4Rows._empty(rows, cols, fmt, torch.cuda.current_device() if dev.index is None else dev.index, stream)


def quantize_fp4_rows(x, fmt="nvfp4", out: Fp4Rows | None = None, stream=None) -> Fp4Rows:
    """Rows of bf16 x [R][C] to 4-bit microscaled rows (C a multiple of 32)."""
    lib = _lib or load_library()
    dev = _device_of(x, "x", _BF16)
    R, C = x.shape
    px = _here(x, "x", _BF16, (R, C), dev)
    if out is None:
        out = Fp4Rows._empty(R, C, fmt, dev, stream)
    elif (out.rows, out.cols, out.fmt, out.device_index) != (R, C, fmt, dev):
        raise ValueError(f"out holds {out.rows} x {out.cols} {out.fmt} on {out.device}, x needs {R} x {C} {fmt} on {x.device}")
    _call(dev, stream, lib.chipmunk_quantize_fp4_rows, px, out.args)
    return out


def dequantize_fp4_rows(q: Fp4Rows, out=None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The values that 4-bit rows stand for, [R][C] in bf16 (exact for what ``quantize_fp4_rows`` made) or fp32."""
    lib = _lib or load_library()
    dev = q.device_index
    if out is None:
        out = _empty((q.rows, q.cols), dtype, dev, stream)
    po = _here(out, "out", _BF16_F32, (q.rows, q.cols), dev)
    _call(dev, stream, lib.chipmunk_dequantize_fp4_rows, q.args, _TYPES[out.dtype], po)
    return out


def linear_fp4_workspace_bytes(T: int, K: int, fmt: str) -> int:
    """Workspace of a linear_fp4 call that quantises its x (none for quantised x, nor for a few rows)."""
    _, codes, scales, rows = _fp4_sizes(T, K, fmt)
    return 0 if T <= 8 and T * (K + 255 & -256) <= 8192 else codes + scales + rows


def linear_fp4(x, w: Fp4Rows, bias=None, out=None, act="none", out_dtype=torch.bfloat16, workspace=None, stream=None):
    """act(x w^T + bias) on 4-bit operands: x bf16 [T][K] (quantised inside, into ``workspace``) or
    Fp4Rows [T][K], w Fp4Rows [N][K], bias bf16 [N], out [T][N] bf16 or fp32. Calls that run at
    the same time, captured ones included, must not share a workspace."""
    lib = _lib or load_library()
    dev, N, K = w.device_index, w.rows, w.cols
    px = pw = None
    ws_bytes = 0
    if isinstance(x, Fp4Rows):
        T = x.rows
        if x.cols != K or x.fmt != w.fmt or x.device_index != dev:
            raise ValueError(f"x holds {x.cols} columns of {x.fmt} on {x.device}, w {K} of {w.fmt} on {w.device}")
        xq = x.args
    else:
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a 2-D tensor or Fp4Rows")
        T = x.shape[0]
        px = _here(x, "x", _BF16, (T, K), dev)
        xq = Fp4Args()
        if workspace is None:
            ws_bytes = linear_fp4_workspace_bytes(T, K, w.fmt)
            if ws_bytes:
                workspace = _empty((ws_bytes,), torch.uint8, dev, stream)
        else:
            if workspace.get_device() != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on {w.device}")
            ws_bytes = workspace.numel() * workspace.element_size()
        pw = None if workspace is None else workspace.data_ptr()
    pb = None if bias is None else _here(bias, "bias", _BF16, (N,), dev)
    if out is None:
        out = _empty((T, N), out_dtype, dev, stream)
    po = _here(out, "out", _BF16_F32, (T, N), dev)
    a = LinearFp4Args(T, N, _pick(_ACTS, act, "act"), _TYPES[out.dtype], px, xq, w.args, pb, po)
    _call(dev, stream, lib.chipmunk_linear_fp4, a, pw, ws_bytes)
    return out


def _mod_row(t, name, dtype, shape, ld, dev) -> int:
    """Address of a gate, scale or shift [B][D] of the others' type and row stride."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError("gate, scale and shift must be tensors of one type, bfloat16 or float32")
    if t.get_device() != dev or t.shape != shape or t.stride(1) != 1:
        raise ValueError(f"{name} must be {list(shape)} on CUDA device {dev} with consecutive columns, "
                         f"is {list(t.shape)} on {t.device}")
    if shape[0] > 1 and t.stride(0) != ld:
        raise ValueError("gate, scale and shift must have the same row stride")
    return t.data_ptr()


def norm_residual(res, y=None, *, gate=None, post_norm="none", post_weight=None, res_scale=1.0, res_out=None,
                  norm="layer", weight=None, bias=None, scale=None, shift=None, offsets=None, eps=1e-6, out=None,
                  out_format="bf16", stream=None):
    """r = res_scale * res + gate * post(y); h = (pre(r) * weight + bias) * (1 + scale) + shift.

    res [T][D] and y [T][D] bf16 or fp32; gate, scale, shift [B][D] of one type (bf16 or fp32), row
    strides allowed; offsets int32 [B + 1] on the device (rows outside it are left as they were) or
    None for one sample. Returns (res_out, h): res_out is written when it is given (``res`` itself
    updates in place) or when y is; h is bf16, (e4m3 codes, row scales) or Fp4Rows as out_format
    says, into ``out`` when given, or None for out_format=None."""
    lib = _lib or load_library()
    dev = _device_of(res, "res", _BF16_F32)
    shape = res.shape
    T, D = shape
    p_res = _here(res, "res", _BF16_F32, shape, dev)
    p_y = p_out = p_sc = p_rs = None
    y_type = 0
    if y is not None:
        p_y, y_type = _here(y, "y", _BF16_F32, shape, dev), _TYPES[y.dtype]
        if res_out is None:
            res_out = _empty(shape, res.dtype, dev, stream)
    p_ro = None if res_out is None else _here(res_out, "res_out", (res.dtype,), shape, dev)
    p_pw = None if post_weight is None else _here(post_weight, "post_weight", _BF16, (D,), dev)
    p_w = None if weight is None else _here(weight, "weight", _BF16, (D,), dev)
    p_b = None if bias is None else _here(bias, "bias", _BF16, (D,), dev)
    B, p_off = 1, None
    if offsets is not None:
        B = offsets.numel() - 1
        if B < 1:
            raise ValueError("offsets must hold at least two values")
        p_off = _here(offsets, "offsets", _I32, (B + 1,), dev)
    first = gate if gate is not None else scale if scale is not None else shift
    p_gate = p_scale = p_shift = None
    mod_type = ld = 0
    if first is not None:
        if not isinstance(first, torch.Tensor) or first.dtype not in _BF16_F32 or first.dim() != 2:
            raise TypeError("gate, scale and shift must be 2-D tensors of one type, bfloat16 or float32")
        mod_type, ld = _TYPES[first.dtype], first.stride(0) if B > 1 else D
        like = (first.dtype, (B, D), ld, dev)
        p_gate = None if gate is None else _mod_row(gate, "gate", *like)
        p_scale = None if scale is None else _mod_row(scale, "scale", *like)
        p_shift = None if shift is None else _mod_row(shift, "shift", *like)
    h, f = None, 0
    if out_format is not None:
        f = _pick(_NORM_OUT, out_format, "out_format")
        if f == 0:
            h = _empty(shape, torch.bfloat16, dev, stream) if out is None else out
            p_out = _here(h, "out", _BF16, shape, dev)
        elif f == 1:
            h = (_empty(shape, torch.uint8, dev, stream), _empty((T,), torch.float32, dev, stream)) if out is None else out
            _need_codes(h[0], "out codes", shape)
            if h[0].get_device() != dev:
                raise ValueError(f"out codes must be on {res.device}")
            p_out, p_rs = h[0].data_ptr(), _here(h[1], "out scales", _F32, (T,), dev)
        else:
            h = Fp4Rows._empty(T, D, out_format, dev, stream) if out is None else out
            if not isinstance(h, Fp4Rows) or (h.rows, h.cols, h.fmt, h.device_index) != (T, D, out_format, dev):
                raise ValueError(f"out must be Fp4Rows of {T} x {D} {out_format} on {res.device}")
            p_out, p_sc, p_rs = h.args.codes, h.args.scales, h.args.row_scales
    a = NormArgs(T, D, B, _TYPES[res.dtype], y_type, mod_type, _pick(_NORMS, post_norm, "post_norm"),
                 _pick(_NORMS, norm, "norm"), f, eps, res_scale, p_res, p_y, p_pw, p_gate, p_ro, p_w, p_b, p_scale, p_shift,
                 ld, p_off, p_out, p_sc, p_rs)
    _call(dev, stream, lib.chipmunk_norm_residual, a)
    return res_out, h


def qk_norm_rope(qkv, h, q_weight, k_weight, cos, sin, pairs="interleaved", eps=1e-6, q=None, k=None, v=None,
                 stream=None):
    """Heads out of a fused projection: qkv bf16 [T][>= 3 h 128] (rows may be strided), RMS norm of each
    q and k head with q_weight, k_weight bf16 [128], rotation by cos, sin fp32 [T][64]; returns q, k,
    v bf16 [T][h][128]."""
    lib = _lib or load_library()
    dev = _device_of(qkv, "qkv", _BF16)
    T, C = qkv.shape
    if qkv.stride(1) != 1 or C < 3 * h * 128:
        raise ValueError(f"qkv must have consecutive columns, at least {3 * h * 128}, has shape {tuple(qkv.shape)}")
    shape = (T, h, 128)
    if q is None:
        q = _empty(shape, torch.bfloat16, dev, stream)
    if k is None:
        k = _empty(shape, torch.bfloat16, dev, stream)
    if v is None:
        v = _empty(shape, torch.bfloat16, dev, stream)
    a = HeadsArgs(T, qkv.stride(0) if T > 1 else 3 * h * 128, h, _pick(_PAIRS, pairs, "pairs"), eps, qkv.data_ptr(),
                  _here(q_weight, "q_weight", _BF16, (128,), dev), _here(k_weight, "k_weight", _BF16, (128,), dev),
                  _here(cos, "cos", _F32, (T, 64), dev), _here(sin, "sin", _F32, (T, 64), dev),
                  _here(q, "q", _BF16, shape, dev), _here(k, "k", _BF16, shape, dev), _here(v, "v", _BF16, shape, dev))
    _call(dev, stream, lib.chipmunk_qk_norm_rope, a)
    return q, k, v
