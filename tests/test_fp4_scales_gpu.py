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


def check_range(got, ref, slack):
    """Finite where the definition is clear of the type's largest number, an infinity of its sign where it is beyond."""
    import torch
    stored, step = (2.0 ** -8, 2.0 ** -133) if got.dtype == torch.bfloat16 else (U, 2.0 ** -149)
    got, top = got.double(), float(torch.finfo(torch.bfloat16).max)
    inside, beyond = ref.abs() + slack < top * (1 - 2.0 ** -7), ref.abs() - slack > 2.0 ** 128
    d = (got - ref).abs()[inside] - (stored * ref.abs() + slack + step)[inside]
    assert bool(got[inside].isfinite().all()) and float(d.max()) <= 0
    assert torch.equal(got[beyond], torch.sign(ref[beyond]) * float("inf"))
    assert not bool(got.isnan().any())
    return inside, beyond


@pytest.mark.parametrize("form,T,N,K", CASES, ids=[NAMES[c[0]] for c in CASES])
def test_row_scales_far_from_one(cm, form, T, N, K):
    """Rows of x and w from 2^-100 to 2^100: the product of two row scales leaves fp32's range both ways."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(form)
    e = lambda n: torch.randint(-5, 6, (n, 1), generator=g, device="cuda") * 20
    ex, ew = e(T), e(N)
    x = (torch.randn(T, K, generator=g, device="cuda") * torch.exp2(ex.float())).bfloat16()
    w = (torch.randn(N, K, generator=g, device="cuda") * torch.exp2(ew.float())).bfloat16()
    x[:, K // 2:] = 0
    w[::5, :K // 2] = 0                      # sums of nothing but zeros
    wq, xq = cm.quantize_fp4_rows(w), cm.quantize_fp4_rows(x)
    xv, wv = (cm.dequantize_fp4_rows(q, dtype=torch.float32).double() for q in (xq, wq))
    ref, S = xv @ wv.t(), xv.abs() @ wv.abs().t()
    for dtype in (torch.float32, torch.bfloat16):
        out = cm.linear_fp4(x, wq, out_dtype=dtype)
        inside, beyond = check_range(out, ref, (K / 64 + 8) * 2 * U * S)
        assert bool(beyond.any()) and not bool(out[:, ::5].any())
    bias = torch.randn(N, generator=g, device="cuda").bfloat16()
    out = cm.linear_fp4(xq, wq, bias, out_dtype=torch.float32)
    check_range(out, ref + bias.double(), (K / 64 + 8) * 2 * U * (S + bias.double().abs()))


def test_small_products_are_not_lost(cm):
    """Both operands small: sums of 4096 equal terms land where fp32 still holds them, their scales' product not."""
    import torch
    for T in (2, 40):
        x = torch.full((T, 4096), 2.0 ** -95, device="cuda").bfloat16()
        w = cm.quantize_fp4_rows(torch.full((136, 4096), 2.0 ** -40, device="cuda").bfloat16())
        for a in (x, cm.quantize_fp4_rows(x)):
            out = cm.linear_fp4(a, w, out_dtype=torch.float32).double()
            v = cm.dequantize_fp4_rows(cm.quantize_fp4_rows(x), dtype=torch.float32).double()
            ref = v @ cm.dequantize_fp4_rows(w, dtype=torch.float32).double().t()
            check_range(out.float(), ref, (4096 / 64 + 8) * 2 * U * ref)
