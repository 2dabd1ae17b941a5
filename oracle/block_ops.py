"""64-bit definitions of the operators around a block's sparse layers (numpy; test infrastructure only).

Written from the definitions in the C header's comments: 4-bit microscaled rows, the product on
them, norms with gate and residual, and the head split with norm and rotation. Inputs are float64
arrays holding the device values exactly. Shares no code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _floor_log2(a):
    """floor(log2 a) of a > 0, exactly."""
    return np.frexp(a)[1] - 1


def round_to(a, table):
    """Index of the nearest entry of an ascending table, ties to the even index, saturating."""
    a = np.asarray(a, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, a, side="left"), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def e4m3_table():
    """The non-negative finite e4m3 values in code order (codes 0 .. 126)."""
    sub = np.arange(8) * 2.0 ** -9
    normal = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.concatenate([sub, normal])[:127]


_E4M3 = e4m3_table()


def quantize_fp4(x, fmt):
    """x [R][C] -> codes [R][C] (0..15), block scale bytes [R][C / block], row scales [R] (nvfp4; else None)."""
    R, C = x.shape
    n = BLOCK[fmt]
    v = x.reshape(R, C // n, n)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        amax = np.abs(v).max(axis=2) if C else np.zeros((R, 0))      # NaN propagates
        if fmt == "mxfp4":
            bad = ~np.isfinite(amax)
            e = np.where(amax > 0, _floor_log2(np.where(bad | (amax == 0), 1.0, amax)) - 2, -127)
            e = np.maximum(e, -127)
            sb = np.where(bad, 255, e + 127).astype(np.uint8)
            rs = None
            step = np.where(bad, np.nan, np.ldexp(1.0, e))
        else:
            row = amax.max(axis=1)
            bad = ~np.isfinite(row)
            e = np.clip(_floor_log2(np.where(bad | (row == 0), 1.0, row)) - 10, -110, 117)
            rs = np.where(bad, np.nan, np.where(row == 0, 1.0, np.ldexp(1.0, e)))
            sb = np.where(bad[:, None], 0, round_to(np.nan_to_num(amax / (6 * rs[:, None])), _E4M3)).astype(np.uint8)
            step = _E4M3[sb] * rs[:, None]
        t = np.nan_to_num(np.abs(v) / step[:, :, None], nan=0.0, posinf=0.0)
    t = np.where(step[:, :, None] > 0, t, 0.0)
    codes = round_to(t, E2M1)
    codes = codes + 8 * (np.signbit(v) & (codes > 0))
    return codes.reshape(R, C).astype(np.uint8), sb, rs


def fp4_values(codes, sb, rs, fmt):
    """The values codes and scales stand for."""
    R, C = codes.shape
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    if fmt == "mxfp4":
        step = np.where(sb == 255, np.nan, np.ldexp(1.0, sb.astype(np.int64) - 127))
    else:
        step = _E4M3[sb] * rs[:, None]
    return (mag.reshape(R, -1, BLOCK[fmt]) * step[:, :, None]).reshape(R, C)


def scale_offset(r, b, C, fmt):
    """Byte of the scale of row r, block b."""
    tiles = -(-C // 256) * (256 // BLOCK[fmt] // 4)
    return (r // 128 * tiles + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def gelu(u):
    return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))


def linear(xv, wv, bias=None, act="none"):
    o = xv @ wv.T
    if bias is not None:
        o = o + bias
    return gelu(o) if act == "gelu" else o


def norm(x, kind, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(axis=1, keepdims=True)
    return x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)


def norm_residual(res, y=None, gate=None, post="none", post_w=None, res_scale=1.0, kind="layer", w=None, b=None,
                  scale=None, shift=None, eps=1e-6):
    """One sample: gate, scale, shift [D]. Returns (r, h)."""
    r = res_scale * res
    if y is not None:
        p = norm(y, post, eps)
        if post_w is not None:
            p = p * post_w
        r = r + (p if gate is None else p * gate)
    h = norm(r, kind, eps)
    if w is not None:
        h = h * w
    if b is not None:
        h = h + b
    if scale is not None:
        h = h * (1 + scale)
    if shift is not None:
        h = h + shift
    return r, h


def qk_norm_rope(qkv, h, qw, kw, cos, sin, pairs, eps):
    T = qkv.shape[0]
    q, k, v = (qkv[:, i * h * 128:(i + 1) * h * 128].reshape(T, h, 128) for i in range(3))

    def one(x, w):
        x = x / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps) * w
        c, s = cos[:, None, :], sin[:, None, :]
        o = np.empty_like(x)
        ia, ib = (slice(0, None, 2), slice(1, None, 2)) if pairs == "interleaved" else (slice(0, 64), slice(64, None))
        a, b = x[..., ia], x[..., ib]
        o[..., ia], o[..., ib] = a * c - b * s, a * s + b * c
        return o

    return one(q, qw), one(k, kw), v
