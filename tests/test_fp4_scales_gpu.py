"""4-bit rows whose row scales are not the quantiser's powers of two (weights of another tool's making).

Tolerances: a product scales its fp32 sums by both row scales in at most five roundings (u = 2^-24 each),
within the 16u that (K / 64 + 8) * 2u * S grants the epilogue. A value is code * block scale (exact, six bits)
times the row scale, one rounding in fp32 (u of it) and, stored as bf16, half a step more."""
import numpy as np
import pytest

from linear_forms import NAMES, SIZES
from oracle import block_ops as R
from test_linear_forms_gpu import U, Product, cm, f64, status_clear  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def unpacked(q):
    packed = q.codes.cpu().numpy()
    return np.stack([packed & 15, packed >> 4], axis=2).reshape(packed.shape[0], -1)


def block_scales(q):
    b = np.arange(q.cols // R.BLOCK[q.fmt])
    return q.scales.cpu().numpy()[R.scale_offset(np.arange(q.rows)[:, None], b[None, :], q.cols, q.fmt)]


def free_scales(q, seed=0):
    """Multiplies q's row scales by factors with full significands; returns the factors as they took effect (64 bits)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    old = q.row_scales.clone()
    q.row_scales.mul_(1 + torch.rand(q.rows, generator=g, device="cuda"))
    assert float(q.row_scales.bfloat16().float().eq(q.row_scales).float().mean()) < 0.1
    return (q.row_scales.double() / old.double())[:, None]


@pytest.mark.parametrize("rows,cols", [(1, 32), (70, 288), (300, 1056)])
def test_values_with_free_row_scales(cm, rows, cols):
    import torch
    q = cm.quantize_fp4_rows(torch.randn(rows, cols, device="cuda").bfloat16())
    free_scales(q)
    values = R.fp4_values(unpacked(q), block_scales(q), f64(q.row_scales), "nvfp4")
    for dtype, allowed in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8 * (1 + U) + U)):
        d = np.abs(f64(cm.dequantize_fp4_rows(q, dtype=dtype)) - values)
        assert np.all(d <= allowed * np.abs(values)), f"{dtype}: worst {np.max(d / np.maximum(np.abs(values), 1e-300)):.3g}"


CASES = [(form, *sizes[0]) for form, sizes in SIZES.items()]


@pytest.mark.parametrize("form,T,N,K", CASES, ids=[NAMES[c[0]] for c in CASES])
def test_products_with_free_row_scales(cm, form, T, N, K):
    """All of w's scales free, then only one row's: its tile alone takes them in full."""
    import torch
    p = Product(cm, T, N, K, "nvfp4")
    sums, mag, ones = p.sums, p.mag, p.w.row_scales.clone()
    f = free_scales(p.w)
    p.sums, p.mag = sums * f.t(), mag * f.t()
    p.check(out_dtype=torch.float32)
    p.check()
    p.check(act="gelu", out_dtype=torch.float32, bias=False)
    one = N // 2 + 3
    free = p.w.row_scales[one].clone()
    p.w.row_scales.copy_(ones)
    p.w.row_scales[one] = free
    f[:one] = 1
    f[one + 1:] = 1
    p.sums, p.mag = sums * f.t(), mag * f.t()
    p.check(out_dtype=torch.float32)
    # x's too
    fx = free_scales(p.xq, 1)
    p.sums, p.mag = p.sums * fx, p.mag * fx
    p.check(out_dtype=torch.float32, quantised=True)
