"""The norms over many rows: every CTA walks several, with the next row's loads in flight, the
statistics' shared buffers in turn and the sample of one row carried to the next. Held to the
64-bit definition with the tolerances of the few-row tests, all rows compared."""
import numpy as np
import pytest

from test_block_ops_gpu import bf16, check_norm, cm, rows_of, status_clear  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

# rows held by 1, 2, 4, 6, 8, 12 and 16 warps with y; 1, 2, 4, 8 and 16 without
WIDTHS = [264, 1024, 1536, 3072, 4096, 6144, 8192]


@pytest.mark.parametrize("D", WIDTHS)
def test_norm_of_many_rows(cm, D):
    rng = np.random.default_rng(D)
    T = 7000 if D < 1024 else 3500
    check_norm(cm, rng, T, D, "layer", "rms")
    check_norm(cm, rng, T, D, "rms", "layer", res="fp32", inplace=True)
    check_norm(cm, rng, T, D, "layer", y=False)
    check_norm(cm, rng, T, D, "rms", y=False, res="fp32")


def spread(T, kind):
    """Sample ends over T rows: long samples with empty and one-row ones between, or hundreds of short ones."""
    if kind == "long":   # a CTA's first rows belong to no sample, its last ones neither
        a = T // 3
        return [a, a, a + 1, a + 2, a + T // 4, a + T // 4, T - T // 4]
    ends = np.cumsum(np.random.default_rng(1).integers(0, 60, 400))
    return [3] + [int(3 + e) for e in ends if 3 + e < T - 5] + [T - 5]


@pytest.mark.parametrize("D,kind", [(256, "short"), (256, "long"), (1536, "long"), (3072, "short"), (8192, "long")])
def test_packed_samples_over_many_rows(cm, D, kind):
    rng = np.random.default_rng(D + 1)
    T = 6000 if D == 256 else 3000
    off = spread(T, kind)
    check_norm(cm, rng, T, D, "layer", "rms", B=len(off) - 1, offsets=off)
    check_norm(cm, rng, T, D, "rms", y=False, B=len(off) - 1, offsets=off, mod="fp32")


@pytest.mark.parametrize("y", [True, False])
@pytest.mark.parametrize("D", [1536, 3072, 8192])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "e4m3"])
def test_quantised_output_of_many_rows_equals_the_quantiser(cm, fmt, D, y):
    """Byte for byte the quantiser's rows of the bf16 output, over packed samples; rows of none keep their bytes."""
    import torch
    rng = np.random.default_rng(D)
    T = 4000
    x = bf16(rows_of(rng, T, D))
    off = spread(T, "long")
    B = len(off) - 1
    m = bf16(rng.standard_normal((B, 3 * D)) * 0.4)
    kw = dict(scale=m[:, D:2 * D], shift=m[:, 2 * D:], offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    if y:
        kw.update(y=bf16(rng.standard_normal((T, D))), gate=m[:, :D], post_norm="rms")
    _, h = cm.norm_residual(x, **kw)
    lo, hi = off[0], off[-1]
    if fmt == "e4m3":
        got = (torch.full((T, D), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((T,), 5.0, device="cuda"))
        cm.norm_residual(x, out_format=fmt, out=got, **kw)
        codes, scales = cm.quantize_e4m3_rows(h[lo:hi].contiguous())
        assert torch.equal(got[0][lo:hi], codes) and torch.equal(got[1][lo:hi], scales)
        outside = torch.cat([got[0][:lo], got[0][hi:]])
        assert bool((outside == 0x5A).all()) and bool((got[1][:lo] == 5).all()) and bool((got[1][hi:] == 5).all())
        return
    got, ref = (cm.empty_fp4_rows(T, D, fmt, "cuda") for _ in range(2))
    h[:lo] = 0
    h[hi:] = 0
    cm.quantize_fp4_rows(h, fmt, out=ref)
    got.codes.copy_(ref.codes)
    got.scales.copy_(ref.scales)
    got.codes[lo:hi] = 0x5A
    got.codes[:lo] = 0x3C
    if fmt == "nvfp4":
        got.row_scales.fill_(5.0)
    cm.norm_residual(x, out_format=fmt, out=got, **kw)
    assert torch.equal(got.codes[lo:hi], ref.codes[lo:hi]) and torch.equal(got.scales, ref.scales)
    assert bool((got.codes[:lo] == 0x3C).all()) and not bool(got.codes[hi:].any())
    if fmt == "nvfp4":
        assert torch.equal(got.row_scales[lo:hi], ref.row_scales[lo:hi])
        assert bool((got.row_scales[:lo] == 5).all()) and bool((got.row_scales[hi:] == 5).all())
