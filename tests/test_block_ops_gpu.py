"""The operators around a block's sparse layers on the GPU against their 64-bit definitions.

Tolerances. A result stored as bf16 is off by at most half a step, 2^-8 of its value; the fp32
arithmetic before it is bounded per operator (u = 2^-24):
* quantised rows and their values are exact (the definition makes every rounding unambiguous);
* products: fp32 sums of exact terms. Each instruction adds 64 columns to the running sum, whose
  rounding is at most one step, 2u, of at most S = sum |x w|; 8 more cover the epilogue, so
  (K / 64 + 8) * 2u * S;
* norms: a thread sums at most 32 columns, then 5 shuffles and at most 16 warps join (under 64
  roundings) for each of mean and variance, so each statistic is good to 64u of the magnitudes it
  sums; with a post norm before it the pre norm sees two such errors. 256u of the magnitudes that
  enter an output covers both;
* heads: 8 columns and 4 shuffles for the mean square, the rotation's two products: 32u of the
  pair's magnitudes.
"""
import math

import numpy as np
import pytest

from oracle import block_ops as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def cm():
    from dynamic_column_sparse_b200 import chipmunk
    chipmunk.load_library()
    return chipmunk


@pytest.fixture(autouse=True)
def status_clear(cm):
    yield
    import torch
    torch.cuda.synchronize()
    assert cm.read_device_status() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def f32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def rows_of(rng, T, D):
    """Rows of different sizes, a few loud columns."""
    x = rng.standard_normal((T, D)) * np.exp2(rng.integers(-3, 4, (T, 1)))
    x[:, rng.integers(0, D, max(1, D // 100))] *= 30
    return x


def close(got, ref, slack, what, stored=2.0 ** -8):
    assert got.shape == ref.shape, what
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    fine = np.isfinite(ref)
    d = np.abs(got - ref)[fine]
    allowed = (stored * np.abs(ref) + slack)[fine]
    assert np.all(d <= allowed), f"{what}: {np.count_nonzero(d > allowed)} of {d.size} outside, worst {np.max(d / np.maximum(allowed, 1e-300)):.3g} of the bound"


# ------------------------------------------------------------------ 4-bit rows

def border_rows(fmt):
    """Rows whose quotients sit on, or one bf16 step beside, every rounding border of the codes, for many
    block scales; with the block's largest value fixing the scale."""
    n = R.BLOCK[fmt]
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    blocks = []
    for m in range(128, 256):           # every bf16 significand as the block's largest magnitude
        top = m / 128.0 * 4
        if fmt == "mxfp4":
            s = 2.0 ** (math.floor(math.log2(top)) - 2)
        else:                           # the row's largest value is 8 * 255 / 128: row scale 2^-7
            s = R._E4M3[R.round_to(np.array([top / (6 * 2.0 ** -7)]), R._E4M3)][0] * 2.0 ** -7
        b = np.zeros(n)
        b[0] = top
        v = borders * s
        up, down = v * (1 + 2.0 ** -7), v * (1 - 2.0 ** -7)
        picks = np.concatenate([v, up, down])[: n - 1] if n > 21 else np.concatenate([v, (up if m % 2 else down)])
        b[1:1 + len(picks)] = picks
        b *= np.where(np.arange(n) % 3 == 2, -1, 1)
        blocks.append(b)
    x = np.stack(blocks).reshape(8, -1)
    x[:, -1] = 8 * 255 / 128.0
    return x


def special_rows():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, 96))
    x[0] = 0
    x[1, :32] = 0                       # an all-zero block among others
    x[2] *= 2.0 ** -130                 # subnormal bf16 magnitudes
    x[3] *= 2.0 ** 120
    x[4, 40] = 2.0 ** 100               # the other blocks' scales vanish beside it
    x[5] *= 2.0 ** -105                 # the row scale's lower clamp
    x[6, 7] = np.inf
    x[7, 70] = -np.inf
    x[8, 95] = np.nan
    x[9] = -1.5
    x[10, ::2] = 0
    x[11] = np.where(np.arange(96) % 2, 6.0, -5.0)
    return x


def quant_inputs(fmt):
    rng = np.random.default_rng(3)
    yield "border", border_rows(fmt)
    yield "special", special_rows()
    for shape in [(1, 32), (3, 64), (129, 96), (260, 1056), (5, 16384), (2, 65536), (1, 4128)]:
        yield f"{shape}", rows_of(rng, *shape)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_and_dequantize_are_exact(cm, fmt):
    import torch
    for name, x in quant_inputs(fmt):
        xd = bf16(x)
        rows, C = xd.shape
        ref_codes, ref_sb, ref_rs = R.quantize_fp4(f64(xd), fmt)
        q = cm.empty_fp4_rows(rows, C, fmt, "cuda")
        q.scales.fill_(0xAB)
        cm.quantize_fp4_rows(xd, fmt, out=q)
        packed = q.codes.cpu().numpy()
        codes = np.empty((rows, C), np.uint8)
        codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
        if fmt == "nvfp4":
            rs = f64(q.row_scales)
            np.testing.assert_array_equal(rs, ref_rs, err_msg=name)
            live = np.isfinite(ref_rs)[:, None] & np.ones((1, C), bool)
        else:
            live = np.repeat(ref_sb != 255, 32, axis=1)
        codes[codes == 8] = 0                                         # the sign of a zero is free
        np.testing.assert_array_equal(codes[live], ref_codes[live], err_msg=name)
        # every scale byte: the rows' own, zeros in their padding to 256 columns, nothing past the last row
        ref = np.full(q.scales.numel(), 0xAB, np.uint8)
        nb = C // R.BLOCK[fmt]
        for b in range(-(-C // 256) * 256 // R.BLOCK[fmt]):
            ref[R.scale_offset(np.arange(rows), b, C, fmt)] = ref_sb[:, b] if b < nb else 0
        np.testing.assert_array_equal(q.scales.cpu().numpy(), ref, err_msg=name)
        values = R.fp4_values(ref_codes, ref_sb, ref_rs, fmt)
        np.testing.assert_array_equal(f64(cm.dequantize_fp4_rows(q, dtype=torch.float32)), values, err_msg=name)
        np.testing.assert_array_equal(f64(cm.dequantize_fp4_rows(q)), values, err_msg=name)


# ------------------------------------------------------------------ products

def fp4_operand(cm, rng, rows, cols, fmt):
    q = cm.quantize_fp4_rows(bf16(rows_of(rng, rows, cols)), fmt)
    return q


def check_linear(cm, rng, T, N, K, fmt, act="none", bias=True, out_dtype=None, quantised=False, xd=None):
    import torch
    out_dtype = out_dtype or torch.bfloat16
    xd = bf16(rows_of(rng, T, K)) if xd is None else xd
    w = cm.quantize_fp4_rows(bf16(rng.standard_normal((N, K)) / math.sqrt(K)), fmt)
    b = bf16(rng.standard_normal(N)) if bias else None
    xq = cm.quantize_fp4_rows(xd, fmt)
    out = cm.linear_fp4(xq if quantised else xd, w, b, act=act, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    xv = R.fp4_values(*R.quantize_fp4(f64(xd), fmt), fmt)
    wv = f64(cm.dequantize_fp4_rows(w, dtype=torch.float32))
    u = R.linear(xv, wv, None if b is None else f64(b))
    ref = R.gelu(u) if act == "gelu" else u
    S = np.abs(xv) @ np.abs(wv).T + (0 if b is None else np.abs(f64(b)))
    # GELU's slope is below 1.13, its own evaluation a few 2^-21 of its argument
    slack = (K / 64 + 8) * 2 * U * S * (1.13 if act == "gelu" else 1) + (2.0 ** -19 * np.abs(u) if act == "gelu" else 0)
    close(f64(out), ref, slack, f"linear T={T} N={N} K={K} {fmt}", stored=2.0 ** -8 if out_dtype == torch.bfloat16 else U)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [
    (128, 128, 256), (1, 8, 32), (1, 1024, 512), (130, 136, 288), (2, 4104, 64), (7, 264, 2080), (33, 200, 1056),
    (300, 640, 4128), (129, 128, 16384), (65, 384, 96), (513, 1160, 544),
    # around the form for a few rows: 8 and 9 rows, its longest rows and the next
    (8, 136, 96), (9, 136, 96), (8, 264, 1024), (8, 264, 1056), (2, 136, 4096), (1, 128, 8192), (1, 128, 8224), (3, 20000, 256),
    # few rows against few and many weight rows, short and long sums
    (1, 3072, 3072), (8, 3072, 3072), (5, 512, 1824), (8, 1000, 4096), (1, 256, 65536), (2, 200, 32768), (1, 9216, 1056),
    (8, 128, 16384), (1, 64, 1536), (7, 1160, 12288), (4, 6000, 2048),
])
def test_linear_matches_definition(cm, fmt, T, N, K):
    check_linear(cm, np.random.default_rng(T * 7 + N + K), T, N, K, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(1, 72, 32), (5, 1000, 544), (8, 4104, 4096), (40, 264, 320), (300, 520, 1056)])
def test_linear_of_rows_and_of_their_codes_agree(cm, fmt, T, N, K):
    """Every term is exact and the order of the sums is the tensor core's, so the forms may differ by
    the rounding of the running sum only; the codes themselves are the same."""
    import torch
    rng = np.random.default_rng(T)
    x = bf16(rows_of(rng, T, K))
    w = fp4_operand(cm, rng, N, K, fmt)
    q = cm.quantize_fp4_rows(x, fmt)
    a, b = (cm.linear_fp4(v, w, out_dtype=torch.float32) for v in (x, q))
    S = np.abs(f64(cm.dequantize_fp4_rows(q, dtype=torch.float32))) @ np.abs(f64(cm.dequantize_fp4_rows(w, dtype=torch.float32))).T
    close(f64(a), f64(b), (K / 64 + 8) * 4 * U * S, "rows against codes", stored=2 * U)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,N,K", [(1, 72, 96), (40, 264, 320), (257, 1032, 800)])
def test_linear_epilogues(cm, fmt, T, N, K):
    import torch
    rng = np.random.default_rng(11)
    check_linear(cm, rng, T, N, K, fmt, act="gelu")
    check_linear(cm, rng, T, N, K, fmt, bias=False)
    check_linear(cm, rng, T, N, K, fmt, out_dtype=torch.float32)
    check_linear(cm, rng, T, N, K, fmt, act="gelu", out_dtype=torch.float32, quantised=True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T", [12, 140])
def test_linear_special_rows_stay_in_their_rows(cm, fmt, T):
    """Zero rows give the bias, rows with an infinity or NaN give NaN, the others are not touched by them."""
    rng = np.random.default_rng(2)
    x = np.concatenate([special_rows(), rows_of(rng, T - 12, 96)])
    x[3] *= 2.0 ** -100
    x[4] *= 2.0 ** -90
    check_linear(cm, rng, T, 136, 96, fmt, xd=bf16(x))


def test_linear_does_not_write_past_its_output(cm):
    import torch
    rng = np.random.default_rng(8)
    for T, N in [(1, 72), (130, 200), (40, 136)]:
        w = fp4_operand(cm, rng, N, 128, "nvfp4")
        big = torch.full((T + 64, N), 7.0, dtype=torch.bfloat16, device="cuda")
        cm.linear_fp4(bf16(rows_of(rng, T, 128)), w, out=big[:T])
        assert bool((big[T:] == 7).all()) and not bool((big[:T] == 7).all())


# ------------------------------------------------------------------ norms

def check_norm(cm, rng, T, D, kind="layer", post="none", y=True, res="bf16", ydt="bf16", mod="bf16", B=1, offsets=None,
               gate=True, affine=False, res_scale=1.0, eps=1e-6, mean=0.0, inplace=False):
    import torch
    to = {"bf16": bf16, "fp32": f32}
    xd = to[res](rng.standard_normal((T, D)) * 2 + mean)
    yd = to[ydt](rng.standard_normal((T, D)) * 0.7 + mean / 3) if y else None
    m = to[mod](rng.standard_normal((B, 3 * D + 8)) * 0.4)
    g, sc, sh = m[:, :D], m[:, D:2 * D], m[:, 2 * D:3 * D]
    pw = bf16(1 + 0.2 * rng.standard_normal(D)) if post != "none" else None
    w, b = (bf16(1 + 0.2 * rng.standard_normal(D)), bf16(0.3 * rng.standard_normal(D))) if affine else (None, None)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x64, y64 = f64(xd), None if yd is None else f64(yd)
    keep = torch.full_like(xd, 5.0)
    r_out = xd if inplace else keep if y else None
    if inplace:
        x64 = x64.copy()
    h_out = torch.full((T, D), 9.0, dtype=torch.bfloat16, device="cuda")
    r, h = cm.norm_residual(xd, yd, gate=g if gate and y else None, post_norm=post, post_weight=pw, res_scale=res_scale,
                            res_out=r_out, norm=kind, weight=w, bias=b, scale=sc, shift=sh, offsets=off, eps=eps,
                            out=h_out)
    spans = [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    in_sample = np.zeros(T, bool)
    o = lambda t: None if t is None else f64(t)
    for s, (lo, hi) in enumerate(spans):
        if lo >= hi:
            continue
        in_sample[lo:hi] = True
        ys = None if y64 is None else y64[lo:hi]
        gs = f64(g)[s] if gate and y else None
        rr, hh = R.norm_residual(x64[lo:hi], ys, gs, post, o(pw), res_scale, kind, o(w), o(b), f64(sc)[s], f64(sh)[s], eps)
        M = np.abs(res_scale * x64[lo:hi])
        if ys is not None:
            py = np.abs(ys)
            if post != "none":
                py = py + py.mean(axis=1, keepdims=True)
                cy = ys - ys.mean(axis=1, keepdims=True) if post == "layer" else ys
                sy = 1 / np.sqrt((cy * cy).mean(axis=1, keepdims=True) + eps)
                py = py * sy + np.abs(cy) * sy * (1 + py.mean(axis=1, keepdims=True) * sy)
            if pw is not None:
                py = py * np.abs(o(pw))
            M = M + (py if gs is None else py * np.abs(gs))
        if y:
            close(f64(r)[lo:hi], rr, 256 * U * M, "res_out", stored=2.0 ** -8 if res == "bf16" else U)
        c = rr - rr.mean(axis=1, keepdims=True) if kind == "layer" else rr
        rstd = 1 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
        # the mean's and the variance's errors reach every column; the variance's relative error is
        # that of its squares plus what the columns' own errors, weighted by c, add
        mean_M = M.mean(axis=1, keepdims=True)
        M = (M + mean_M) * rstd + np.abs(c) * rstd * (1 + mean_M * rstd)
        f = np.abs(1 + f64(sc)[s])
        M = M * f * (1 if w is None else np.abs(o(w))) + (0 if b is None else np.abs(o(b)) * f) + np.abs(f64(sh)[s])
        close(f64(h)[lo:hi], hh, 256 * U * M, f"h T={T} D={D}")
    if not in_sample.all():
        assert bool((h[torch.from_numpy(~in_sample).cuda()] == 9).all())
        if y and not inplace:
            assert bool((r[torch.from_numpy(~in_sample).cuda()] == 5).all())


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,D", [(1, 8), (3, 64), (5, 264), (2, 1024), (33, 1032), (1, 3000), (9, 4096), (4, 4104),
                                 (3, 8192), (2, 10000), (2, 16384)])
def test_norm_matches_definition(cm, kind, T, D):
    rng = np.random.default_rng(T + D)
    check_norm(cm, rng, T, D, kind, y=False)
    check_norm(cm, rng, T, D, kind, post="rms")
    check_norm(cm, rng, T, D, kind, post="layer", res="fp32", res_scale=0.5)
    check_norm(cm, rng, T, D, kind, post="none", affine=True, ydt="fp32", mod="fp32")


def test_norm_types_and_options(cm):
    rng = np.random.default_rng(1)
    for res in ("bf16", "fp32"):
        for ydt in ("bf16", "fp32"):
            for mod in ("bf16", "fp32"):
                check_norm(cm, rng, 17, 520, "layer", "rms", res=res, ydt=ydt, mod=mod, gate=(mod == "bf16"))
    check_norm(cm, rng, 40, 3000, "layer", "layer", mean=300.0)      # a mean far above the spread
    check_norm(cm, rng, 40, 512, "rms", "rms", eps=0.1)
    check_norm(cm, rng, 5000, 256, "layer", "none")                  # more rows than the grid holds at once
    check_norm(cm, rng, 33, 1032, "layer", "rms", inplace=True)


@pytest.mark.parametrize("offsets", [[0, 40], [0, 0, 40], [0, 13, 13, 14, 35], [5, 6, 30, 30, 39], [0, 0, 0], [40, 40],
                                     [0, 1, 2, 3, 4, 5, 6, 7, 8, 9]])
@pytest.mark.parametrize("D", [264, 1536])
def test_norm_packed_samples(cm, offsets, D):
    rng = np.random.default_rng(6)
    check_norm(cm, rng, 40, D, "layer", "rms", B=len(offsets) - 1, offsets=offsets)


@pytest.mark.parametrize("D", [32, 64, 288, 1056, 1504, 3072, 5152, 8192, 10016, 16384])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4", "e4m3"])
def test_norm_quantised_output_equals_the_quantiser(cm, D, fmt):
    """The quantised rows are those of the bf16 output, byte for byte."""
    import torch
    rng = np.random.default_rng(D)
    T = 140
    x, y = bf16(rows_of(rng, T, D)), bf16(rng.standard_normal((T, D)))
    x[3] = 0
    y[3] = 0
    m = bf16(rng.standard_normal((1, 3 * D)) * 0.4)
    kw = dict(gate=m[:, :D], post_norm="rms", scale=m[:, D:2 * D], shift=m[:, 2 * D:] if D != 64 else None)
    r, h = cm.norm_residual(x, y, **kw)
    r2, q = cm.norm_residual(x, y, out_format=fmt, **kw)
    assert torch.equal(r, r2)
    if fmt == "e4m3":
        codes, scales = cm.quantize_e4m3_rows(h)
        assert torch.equal(codes, q[0]) and torch.equal(scales, q[1])
        return
    ref = cm.empty_fp4_rows(T, D, fmt, "cuda")
    got = cm.empty_fp4_rows(T, D, fmt, "cuda")
    ref.scales.fill_(0x5A)
    got.scales.fill_(0x5A)
    cm.quantize_fp4_rows(h, fmt, out=ref)
    cm.norm_residual(x, y, out_format=fmt, out=got, **kw)
    for g in (got,):
        assert torch.equal(g.codes, ref.codes) and torch.equal(g.scales, ref.scales)
        if fmt == "nvfp4":
            assert torch.equal(g.row_scales, ref.row_scales)
    assert torch.equal(q.codes, ref.codes)


def test_norm_residual_only(cm):
    import torch
    rng = np.random.default_rng(4)
    x, y = bf16(rng.standard_normal((37, 264))), bf16(rng.standard_normal((37, 264)))
    g = bf16(rng.standard_normal((1, 264)))
    r, h = cm.norm_residual(x, y, gate=g, res_scale=2.0, out_format=None)
    assert h is None
    M = np.abs(2 * f64(x)) + np.abs(f64(y) * f64(g))
    close(f64(r), 2 * f64(x) + f64(y) * f64(g), 8 * U * M, "residual only")


def test_norm_rows_that_are_not_finite_stay_in_their_rows(cm):
    import torch
    rng = np.random.default_rng(4)
    for D in (264, 2048):
        x = rng.standard_normal((9, D))
        clean = bf16(x)
        x[2, 5], x[6, 200] = np.nan, np.inf
        _, h = cm.norm_residual(bf16(x))
        _, ref = cm.norm_residual(clean)
        bad = torch.zeros(9, dtype=torch.bool, device="cuda")
        bad[2] = bad[6] = True
        assert bool(h[2].isnan().all()) and bool(h[6].isnan().any())
        assert torch.equal(h[~bad], ref[~bad])


# ------------------------------------------------------------------ heads

@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("T,h,extra", [(1, 1, 0), (3, 1, 8), (7, 3, 40), (130, 24, 0), (33, 5, 1000), (2, 129, 0)])
def test_heads_match_definition(cm, pairs, T, h, extra):
    rng = np.random.default_rng(T + h)
    x = rng.standard_normal((T, 3 * h * 128 + extra))
    x[0, :128] = 0                                                    # a head of zeros: eps alone
    qkv = bf16(x)
    qw, kw = bf16(1 + 0.2 * rng.standard_normal(128)), bf16(1 + 0.2 * rng.standard_normal(128))
    ang = rng.uniform(-20, 20, (T, 64))
    cos, sin = f32(np.cos(ang)), f32(np.sin(ang))
    got = cm.qk_norm_rope(qkv, h, qw, kw, cos, sin, pairs=pairs)
    ref = R.qk_norm_rope(f64(qkv), h, f64(qw), f64(kw), f64(cos), f64(sin), pairs, 1e-6)
    # the pair's magnitudes: rotate |a|, |b| with |cos|, |sin| and only plus signs
    for name, g, r, w in (("q", got[0], ref[0], qw), ("k", got[1], ref[1], kw)):
        pair = np.sqrt((r * r).reshape(T, h, 64, 2).sum(3).repeat(2, axis=2)) if pairs == "interleaved" else \
            np.tile(np.sqrt(r[..., :64] ** 2 + r[..., 64:] ** 2), 2)
        close(f64(g), r, 32 * U * 1.5 * pair, name)
    np.testing.assert_array_equal(f64(got[2]), ref[2])


def test_heads_from_rows_of_a_wider_tensor(cm):
    import torch
    rng = np.random.default_rng(9)
    wide = bf16(rng.standard_normal((20, 2 * 3 * 2 * 128)))
    qw = bf16(np.ones(128))
    c, s = f32(np.ones((20, 64))), f32(np.zeros((20, 64)))
    view = wide[:, :3 * 2 * 128]
    a = cm.qk_norm_rope(view, 2, qw, qw, c, s)
    b = cm.qk_norm_rope(view.contiguous(), 2, qw, qw, c, s)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


# ------------------------------------------------------------------ addresses

def test_tensors_at_16_byte_offsets(cm):
    """Rows that start 16 bytes into an allocation (the loads and stores of 32 bytes do not apply)."""
    import torch
    rng = np.random.default_rng(31)
    T, C, N = 37, 288, 72

    def shifted(t):
        flat = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        flat[8:].copy_(t.reshape(-1))
        return flat[8:].view(t.shape)

    x = bf16(rows_of(rng, T, C))
    xs = shifted(x)
    assert xs.data_ptr() % 32 == 16
    w = fp4_operand(cm, rng, N, C, "nvfp4")
    for fmt in ("nvfp4", "mxfp4"):
        a, b = cm.quantize_fp4_rows(x, fmt), cm.quantize_fp4_rows(xs, fmt)
        assert torch.equal(a.codes, b.codes)
        va, vb = cm.dequantize_fp4_rows(a), shifted(torch.zeros_like(x))
        cm.dequantize_fp4_rows(a, out=vb)
        assert torch.equal(va, vb)
    for t in (1, T):
        oa, ob = cm.linear_fp4(x[:t], w), shifted(torch.zeros((t, N), dtype=torch.bfloat16, device="cuda"))
        cm.linear_fp4(xs[:t], w, out=ob)
        assert torch.equal(oa, ob)
    _, ha = cm.norm_residual(x)
    _, hb = cm.norm_residual(xs, out=shifted(torch.zeros_like(x)))
    assert torch.equal(ha, hb)


def test_tensors_past_31_bit_offsets(cm):
    """More than 2^31 values: the last rows are what the same rows alone give."""
    import torch
    bf = torch.bfloat16
    T, C = 66000, 32768
    x = torch.zeros((T, C), dtype=bf, device="cuda")
    tail = torch.randn(3, C, device="cuda").bfloat16()
    x[-3:] = tail
    q = cm.quantize_fp4_rows(x, "nvfp4")
    del x
    v = cm.dequantize_fp4_rows(q)
    assert torch.equal(v[-3:], cm.dequantize_fp4_rows(cm.quantize_fp4_rows(tail, "nvfp4")))
    del q, v
    T, D = 132000, 16384
    x = torch.zeros((T, D), dtype=bf, device="cuda")
    x[-3:] = tail[:, :D]
    _, h = cm.norm_residual(x, out=torch.empty_like(x))
    assert torch.equal(h[-3:], cm.norm_residual(tail[:, :D].contiguous())[1])
    del x, h
    T, N = 264000, 8192
    x = torch.zeros((T, 64), dtype=bf, device="cuda")
    x[-3:] = tail[:, :64]
    w = cm.quantize_fp4_rows(torch.randn(N, 64, device="cuda").bfloat16(), "mxfp4")
    out = cm.linear_fp4(x, w)
    assert torch.equal(out[-3:], cm.linear_fp4(cm.quantize_fp4_rows(tail[:, :64].contiguous(), "mxfp4"), w))
    del x, out
    T, h = 120000, 48
    qkv = torch.zeros((T, 3 * h * 128), dtype=bf, device="cuda")
    qkv[-3:] = tail[:, :3 * h * 128]
    one = torch.ones(128, dtype=bf, device="cuda")
    ang = torch.rand(T, 64, device="cuda")
    got = cm.qk_norm_rope(qkv, h, one, one, ang.cos(), ang.sin())
    want = cm.qk_norm_rope(qkv[-3:].contiguous(), h, one, one, ang.cos()[-3:].contiguous(), ang.sin()[-3:].contiguous())
    for a, b in zip(got, want):
        assert torch.equal(a[-3:], b)


# ------------------------------------------------------------------ streams, graphs

def test_calls_on_another_stream_and_in_graphs(cm):
    import torch
    rng = np.random.default_rng(12)
    T, D, N = 70, 512, 264
    x = bf16(rows_of(rng, T, D))
    w = fp4_operand(cm, rng, N, D, "nvfp4")
    mod = bf16(rng.standard_normal((1, 2 * D)) * 0.3)

    def chain(x, **kw):
        _, h = cm.norm_residual(x, scale=mod[:, :D], shift=mod[:, D:], out_format="nvfp4", **kw)
        return cm.linear_fp4(x, w, act="gelu", **kw), cm.linear_fp4(h, w, **kw)

    ref = chain(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(x, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # both streams at once, each call with memory of its own
    a = [chain(x, stream=side), chain(x)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for got in a for u, v in zip(ref, got))
    # two captured chains, replayed on new inputs
    static = x.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain(static)
        graphs.append((g, outs))
    for seed in (1, 2):
        x2 = bf16(rows_of(np.random.default_rng(seed), T, D))
        want = chain(x2)
        static.copy_(x2)
        for g, outs in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, outs))


# ------------------------------------------------------------------ refusals and the status word

def test_refusals_of_device_tensors(cm):
    import torch
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")
    w = cm.quantize_fp4_rows(z(72, 64) + 1)
    with pytest.raises(cm.ChipmunkError, match="T=0"):
        cm.linear_fp4(z(0, 64), w)
    with pytest.raises(cm.ChipmunkError, match="T=0"):
        cm.norm_residual(z(0, 64))
    with pytest.raises(cm.ChipmunkError, match="N=12"):
        cm.linear_fp4(z(3, 64), cm.quantize_fp4_rows(z(12, 64)))
    with pytest.raises(cm.ChipmunkError, match="D=12"):
        cm.norm_residual(z(3, 12))
    with pytest.raises(cm.ChipmunkError, match="need y"):
        cm.norm_residual(z(3, 64), gate=z(1, 64))
    with pytest.raises(cm.ChipmunkError, match="ld_mod"):
        cm.norm_residual(z(3, 64), scale=z(1, 64).expand(2, 64), offsets=torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"))
    with pytest.raises(cm.ChipmunkError) as e:
        cm.linear_fp4(z(30, 64), w, workspace=z(16, dtype=torch.uint8))
    assert e.value.status == cm.ERR_WORKSPACE
    with pytest.raises(ValueError, match="contiguous"):
        cm.linear_fp4(z(64, 3).t(), w)
    with pytest.raises(ValueError, match="columns"):
        cm.linear_fp4(cm.quantize_fp4_rows(z(3, 64), "mxfp4"), w)
    with pytest.raises(ValueError, match="x must|shape"):
        cm.linear_fp4(z(3, 96), w)
    with pytest.raises(TypeError, match="one type"):
        cm.norm_residual(z(3, 64), scale=z(1, 64, dtype=torch.float32), shift=z(1, 64))
    with pytest.raises(ValueError, match="scale must be"):
        cm.norm_residual(z(3, 64), scale=z(2, 64))
    with pytest.raises(ValueError, match="multiple of 32"):
        cm.quantize_fp4_rows(z(3, 48))
    with pytest.raises(ValueError, match="384"):
        cm.qk_norm_rope(z(3, 100), 1, z(128), z(128), z(3, 64), z(3, 64))
    # no rows: nothing to quantise, and nothing comes back
    q = cm.quantize_fp4_rows(z(0, 64))
    assert q.rows == 0 and cm.dequantize_fp4_rows(q).shape == (0, 64)


def test_calls_are_skipped_while_the_status_word_is_set(cm):
    """A wait that ran out elsewhere: every later kernel returns without touching its outputs, the product's
    CTA pairs and the kernel launched behind a skipped quantiser included; cleared, all run again."""
    import torch
    rng = np.random.default_rng(40)
    sizes = [(1, 128, 96), (300, 264, 512), (2560, 2304, 512)]        # a few rows, single tiles, pairs
    ops = []
    for T, N, K in sizes:
        x, w = bf16(rows_of(rng, T, K)), fp4_operand(cm, rng, N, K, "nvfp4")
        out = torch.full((T, N), 3.0, dtype=torch.bfloat16, device="cuda")
        ops.append((out, lambda x=x, w=w, out=out: cm.linear_fp4(x, w, out=out)))
    x = bf16(rows_of(rng, 40, 512))
    h = torch.full_like(x, 3.0)
    ops.append((h, lambda: cm.norm_residual(x, out=h)))
    q, d = cm.quantize_fp4_rows(x), torch.full_like(x, 3.0)
    ops.append((d, lambda: cm.dequantize_fp4_rows(q, out=d)))
    q2 = cm.empty_fp4_rows(40, 512, "mxfp4", "cuda")
    q2.codes.fill_(3)
    ops.append((q2.codes, lambda: cm.quantize_fp4_rows(x, "mxfp4", out=q2)))
    hd = [torch.full((8, 1, 128), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    qkv, hw, ang = bf16(rng.standard_normal((8, 384))), bf16(np.ones(128)), f32(np.zeros((8, 64)))
    ops.append((hd[2], lambda: cm.qk_norm_rope(qkv, 1, hw, hw, ang, ang, q=hd[0], k=hd[1], v=hd[2])))
    lib = cm.load_library()
    assert lib.chipmunk_selftest_bounded_wait(torch.cuda.current_stream().cuda_stream) == 0
    for out, call in ops:
        call()
    torch.cuda.synchronize()
    for out, _ in ops:
        assert bool((out == 3).all())
    assert cm.read_device_status() == 1
    for out, call in ops:
        call()
    torch.cuda.synchronize()
    assert all(not bool((out == 3).all()) for out, _ in ops)
