"""Host side of the operators around a block's sparse layers: the 64-bit definitions pinned to
fixtures and identities, the structs' layout, and the refusals of the C ABI and of the binding
(none of which reach a device)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import block_ops as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cm():
    from dynamic_column_sparse_b200 import build, chipmunk
    build.build()
    chipmunk.load_library()
    return chipmunk


# ------------------------------------------------------------------ the definitions

def test_e2m1_rounding_ties_go_to_the_even_code():
    a = np.array([0, 0.25, 0.26, 0.5, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6, 100])
    want = [0, 0, 0.5, 0.5, 1, 0.5, 1, 1.5, 2, 2, 3, 4, 3, 4, 6, 6, 6]
    np.testing.assert_array_equal(R.E2M1[R.round_to(a, R.E2M1)], want)


def test_e4m3_table():
    t = R.e4m3_table()
    assert len(t) == 127 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[0x38] == 1 and t[126] == 448
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double(), torch.from_numpy(t))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantised_values_are_near_and_stable(fmt):
    x = np.random.default_rng(0).standard_normal((40, 256)).astype(np.float32)
    x = torch.from_numpy(x).bfloat16().double().numpy()
    codes, sb, rs = R.quantize_fp4(x, fmt)
    v = R.fp4_values(codes, sb, rs, fmt)
    n = R.BLOCK[fmt]
    amax = np.abs(x).reshape(40, -1, n).max(axis=2, keepdims=True)
    # at most one code step of a block whose top code is at least amax * 3 / 4 .. (saturation included)
    assert np.all(np.abs(v - x).reshape(40, -1, n) <= amax / 4 + 1e-12)
    again = R.fp4_values(*R.quantize_fp4(v, fmt), fmt)
    assert np.mean(again == v) > (0.99 if fmt == "mxfp4" else 0.5)
    # doubling the input doubles the values
    np.testing.assert_array_equal(R.fp4_values(*R.quantize_fp4(2 * x, fmt), fmt), 2 * v)


def test_quantise_special_rows():
    x = np.zeros((4, 32))
    x[1, 3], x[2, 0], x[3, :2] = np.nan, np.inf, (6.0, -0.2)
    codes, sb, rs = R.quantize_fp4(x, "nvfp4")
    assert rs[0] == 1 and np.isnan(rs[1]) and np.isnan(rs[2]) and rs[3] == 2.0 ** -8
    assert not sb[:3].any() and not codes[0].any()
    codes, sb, rs = R.quantize_fp4(x, "mxfp4")
    assert rs is None and list(sb[:, 0]) == [0, 255, 255, 127]
    assert codes[3, 0] == 7 and codes[3, 1] == 0


def test_norm_definition_identities():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((5, 48)) + 3, rng.standard_normal((5, 48))
    _, h = R.norm_residual(x, kind="layer", eps=0)
    np.testing.assert_allclose(h.mean(1), 0, atol=1e-12)
    np.testing.assert_allclose((h * h).mean(1), 1)
    np.testing.assert_allclose(h, torch.nn.functional.layer_norm(torch.from_numpy(x), (48,), eps=0).numpy())
    r, _ = R.norm_residual(x, y, gate=np.zeros(48), post="rms")
    np.testing.assert_array_equal(r, x)


def test_heads_definition_rotates_and_keeps_lengths():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 3 * 2 * 128))
    one = np.ones(128)
    ang = rng.uniform(-3, 3, (3, 64))
    for pairs in ("interleaved", "halves"):
        q, k, v = R.qk_norm_rope(x, 2, one, one, np.cos(ang), np.sin(ang), pairs, 0.0)
        np.testing.assert_allclose((q * q).sum(2), 128)
        back, _, _ = R.qk_norm_rope(np.concatenate([q.reshape(3, -1)] * 3, 1), 2, one, one, np.cos(ang), -np.sin(ang), pairs, 0.0)
        plain, _, _ = R.qk_norm_rope(x, 2, one, one, np.ones((3, 64)), np.zeros((3, 64)), pairs, 0.0)
        np.testing.assert_allclose(back, plain, atol=1e-12)
        np.testing.assert_array_equal(v.reshape(3, -1), x[:, 512:])


def test_scale_offsets_cover_the_tiles_once():
    for fmt, C in (("nvfp4", 288), ("mxfp4", 288), ("nvfp4", 32)):
        per_row = -(-C // 256) * 256 // R.BLOCK[fmt]
        seen = {R.scale_offset(r, b, C, fmt) for r in range(256) for b in range(per_row)}
        assert seen == set(range(256 * per_row))


# ------------------------------------------------------------------ the C ABI

def test_struct_layouts_match_the_header(cm, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    structs = {"chipmunk_fp4_rows": cm.Fp4Args, "chipmunk_linear_fp4_args": cm.LinearFp4Args,
               "chipmunk_norm_args": cm.NormArgs, "chipmunk_heads_args": cm.HeadsArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", "#include \"chipmunk.h\"", "int main(void) {"]
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        cname, field, val = line.split()
        py = structs[cname]
        assert int(val) == (ctypes.sizeof(py) if field == "sizeof" else getattr(py, field).offset), (cname, field)


def test_sizes_of_the_binding_match_the_library(cm):
    lib = cm.load_library()
    for fmt, f in (("nvfp4", cm.NVFP4), ("mxfp4", cm.MXFP4)):
        for rows in (1, 127, 128, 129, 4352, 118800):
            for cols in (32, 64, 224, 256, 288, 3072, 65536):
                assert cm.fp4_scale_bytes(rows, cols, fmt) == lib.chipmunk_fp4_scale_bytes(rows, cols, f)
                w = cm.Fp4Args(8, cols, f, 16, 16, 16)
                a = cm.LinearFp4Args(rows, 8, 0, 0, 16, cm.Fp4Args(), w, None, None)
                assert cm.linear_fp4_workspace_bytes(rows, cols, fmt) == cm.workspace_bytes(cm.OP_LINEAR_FP4, a)
    assert lib.chipmunk_fp4_scale_bytes(1, 48, 0) == 0


def test_scale_bytes(cm):
    assert cm.fp4_scale_bytes(1, 32, "nvfp4") == 4 * 512 and cm.fp4_scale_bytes(1, 32, "mxfp4") == 2 * 512
    assert cm.fp4_scale_bytes(129, 288, "nvfp4") == 2 * 8 * 512
    assert cm.fp4_scale_bytes(0, 64, "nvfp4") == 0
    for rows, cols in ((1, 0), (1, 48), (1, 65568), (-1, 64)):
        with pytest.raises(ValueError):
            cm.fp4_scale_bytes(rows, cols, "nvfp4")
    with pytest.raises(ValueError, match="fmt"):
        cm.fp4_scale_bytes(1, 64, "fp4")


def _fp4(cm, **kw):
    base = dict(rows=300, cols=256, format=0, codes=0x1000, scales=0x2000, row_scales=0x3000)
    base.update(kw)
    return cm.Fp4Args(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(cols=48), "ERR_SHAPE"), (dict(cols=0), "ERR_SHAPE"), (dict(cols=1 << 17), "ERR_SHAPE"),
    (dict(rows=-1), "ERR_SHAPE"), (dict(format=2), "ERR_INVALID_ARG"), (dict(codes=0), "ERR_INVALID_ARG"),
    (dict(row_scales=0), "ERR_INVALID_ARG"), (dict(scales=0x2004), "ERR_ALIGNMENT"), (dict(rows=0, codes=0), "OK"),
])
def test_quantise_refusals(cm, kw, status):
    lib = cm.load_library()
    q = _fp4(cm, **kw)
    assert lib.chipmunk_quantize_fp4_rows(0x4000, ctypes.byref(q), None) == getattr(cm, status)
    assert lib.chipmunk_dequantize_fp4_rows(ctypes.byref(q), 0, 0x4000, None) == getattr(cm, status)


def test_quantise_refuses_missing_pointers(cm):
    lib = cm.load_library()
    q = _fp4(cm)
    assert lib.chipmunk_quantize_fp4_rows(None, ctypes.byref(q), None) == cm.ERR_INVALID_ARG
    assert lib.chipmunk_quantize_fp4_rows(0x4008, ctypes.byref(q), None) == cm.ERR_ALIGNMENT
    assert lib.chipmunk_quantize_fp4_rows(0x4000, None, None) == cm.ERR_INVALID_ARG
    assert lib.chipmunk_dequantize_fp4_rows(ctypes.byref(q), 2, 0x4000, None) == cm.ERR_INVALID_ARG


def _linear(cm, **kw):
    base = dict(T=40, N=300 - 300 % 8, act=0, out_type=0, x=0x4000, xq=cm.Fp4Args(),
                w=_fp4(cm, rows=300 - 300 % 8), bias=0, out=0x5000)
    base.update(kw)
    return cm.LinearFp4Args(**base)


def test_linear_refusals(cm):
    lib = cm.load_library()
    call = lambda a, ws=0x6000, n=1 << 30: lib.chipmunk_linear_fp4(ctypes.byref(a), ws, n, None)
    assert lib.chipmunk_linear_fp4(None, None, 0, None) == cm.ERR_INVALID_ARG
    assert call(_linear(cm, T=0)) == cm.ERR_SHAPE
    assert call(_linear(cm, T=1 << 30, N=1 << 20, w=_fp4(cm, rows=1 << 20))) == cm.ERR_SHAPE
    assert call(_linear(cm, N=12, w=_fp4(cm, rows=12))) == cm.ERR_SHAPE
    assert call(_linear(cm, N=304)) == cm.ERR_SHAPE                    # w has 296 rows
    assert call(_linear(cm, act=2)) == cm.ERR_INVALID_ARG
    assert call(_linear(cm, out_type=5)) == cm.ERR_INVALID_ARG
    assert call(_linear(cm, out=0)) == cm.ERR_INVALID_ARG
    assert call(_linear(cm, out=0x5008)) == cm.ERR_ALIGNMENT
    assert call(_linear(cm, bias=0x5008)) == cm.ERR_ALIGNMENT
    a = _linear(cm)
    need = cm.workspace_bytes(cm.OP_LINEAR_FP4, a)
    # 40 rows of 128 bytes of codes, one tile row of scales, 40 row scales, each from a 256-byte boundary
    # (codes to a 256-byte boundary, row scales too)
    assert need == 40 * 128 + 4 * 512 + 256 == cm.linear_fp4_workspace_bytes(40, 256, "nvfp4")
    assert cm.linear_fp4_workspace_bytes(40, 256, "mxfp4") == 40 * 128 + 2 * 512
    assert call(a, None, 0) == cm.ERR_WORKSPACE and call(a, 0x6000, need - 1) == cm.ERR_WORKSPACE
    assert call(a, 0x6008, need) == cm.ERR_ALIGNMENT
    # quantised x: it has to fit, and needs no workspace
    a = _linear(cm, x=0, xq=_fp4(cm, rows=40, cols=288))
    assert cm.workspace_bytes(cm.OP_LINEAR_FP4, a) == 0 and call(a, None, 0) == cm.ERR_SHAPE
    assert call(_linear(cm, x=0, xq=_fp4(cm, rows=41)), None, 0) == cm.ERR_SHAPE
    assert call(_linear(cm, x=0, xq=_fp4(cm, rows=40, format=1)), None, 0) == cm.ERR_SHAPE
    assert call(_linear(cm, x=0), None, 0) == cm.ERR_SHAPE             # neither x nor xq


def _norm(cm, **kw):
    base = dict(T=40, D=256, B=1, norm=1, eps=1e-6, res_scale=1.0, res=0x1000, y=0x2000, gate=0x3000, res_out=0x4000,
                scale=0x5000, shift=0x6000, ld_mod=768, out=0x7000)
    base.update(kw)
    return cm.NormArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "ERR_SHAPE"), (dict(D=0), "ERR_SHAPE"), (dict(D=12), "ERR_SHAPE"), (dict(D=16392), "ERR_SHAPE"),
    (dict(B=0), "ERR_SHAPE"), (dict(B=2), "ERR_INVALID_ARG"), (dict(res_type=2), "ERR_INVALID_ARG"),
    (dict(mod_type=-1), "ERR_INVALID_ARG"), (dict(norm=0), "ERR_INVALID_ARG"), (dict(norm=3), "ERR_INVALID_ARG"),
    (dict(post_norm=3), "ERR_INVALID_ARG"), (dict(out_format=4), "ERR_INVALID_ARG"),
    (dict(eps=-1.0), "ERR_INVALID_ARG"), (dict(eps=float("nan")), "ERR_INVALID_ARG"),
    (dict(res_scale=float("inf")), "ERR_INVALID_ARG"), (dict(y=0), "ERR_INVALID_ARG"),
    (dict(y=0, gate=0, post_norm=1), "ERR_INVALID_ARG"), (dict(post_weight=0x8000), "ERR_INVALID_ARG"),
    (dict(out=0, res_out=0), "ERR_INVALID_ARG"), (dict(ld_mod=248), "ERR_SHAPE"), (dict(ld_mod=260), "ERR_SHAPE"),
    (dict(res=0), "ERR_INVALID_ARG"), (dict(res=0x1008), "ERR_ALIGNMENT"), (dict(shift=0x6002), "ERR_ALIGNMENT"),
    (dict(offsets=0x9002), "ERR_ALIGNMENT"), (dict(out_format=1), "ERR_INVALID_ARG"),
    (dict(out_format=2, out_row_scales=0xa000), "ERR_INVALID_ARG"),
    (dict(out_format=3, D=264, out_scales=0xa000), "ERR_SHAPE"), (dict(out_format=1, D=264, out_row_scales=0xa000), "ERR_SHAPE"),
])
def test_norm_refusals(cm, kw, status):
    lib = cm.load_library()
    a = _norm(cm, **kw)
    assert lib.chipmunk_norm_residual(ctypes.byref(a), None) == getattr(cm, status), lib.chipmunk_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "ERR_SHAPE"), (dict(h=0), "ERR_SHAPE"), (dict(h=1025), "ERR_SHAPE"), (dict(T=1 << 30, h=2), "ERR_SHAPE"),
    (dict(ld=760), "ERR_SHAPE"), (dict(ld=772), "ERR_SHAPE"), (dict(pairs=2), "ERR_INVALID_ARG"),
    (dict(eps=-1e-6), "ERR_INVALID_ARG"), (dict(cos=0), "ERR_INVALID_ARG"), (dict(v=0), "ERR_INVALID_ARG"),
    (dict(qkv=0x1008), "ERR_ALIGNMENT"),
])
def test_heads_refusals(cm, kw, status):
    lib = cm.load_library()
    base = dict(T=40, ld=768, h=2, pairs=0, eps=1e-6, qkv=0x1000, q_weight=0x2000, k_weight=0x3000, cos=0x4000, sin=0x5000,
                q=0x6000, k=0x7000, v=0x8000)
    base.update(kw)
    a = cm.HeadsArgs(**base)
    assert lib.chipmunk_qk_norm_rope(ctypes.byref(a), None) == getattr(cm, status), lib.chipmunk_last_error()


# ------------------------------------------------------------------ the binding

def test_binding_refuses_host_tensors_and_wrong_types(cm):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        cm.quantize_fp4_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        cm.norm_residual(x)
    with pytest.raises(ValueError, match="CUDA"):
        cm.qk_norm_rope(torch.zeros((4, 384), dtype=torch.bfloat16), 1, x[0], x[0], x, x)
    with pytest.raises(TypeError):
        cm.norm_residual(x.half())
    with pytest.raises(TypeError):
        cm.quantize_fp4_rows(x.float())
    with pytest.raises(ValueError, match="2-D"):
        cm.quantize_fp4_rows(x[0])
    with pytest.raises(ValueError, match="2-D"):
        cm.norm_residual(x[0])
    with pytest.raises(ValueError, match="fmt"):
        cm.Fp4Rows(None, None, None, "int4", 1, 64)
    with pytest.raises(TypeError, match="codes"):
        cm.Fp4Rows(None, None, None, "nvfp4", 1, 64)
