"""A whole block: norms, 4-bit projections, head split, sparse layers, gates, run as a model runs them.

Each stage is held to the 64-bit definition of that stage on the device's own input to it
(tolerances as for the operators alone; attention and MLP by the parity bar of their own tests), so
no error of one stage hides in another's."""
import math

import numpy as np
import pytest

import oracle as O
from helpers import assert_parity
from oracle import block_ops as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, slack, what):
    d = np.abs(got - ref)
    allowed = 2.0 ** -8 * np.abs(ref) + slack
    assert np.all(np.isfinite(got)) and np.all(d <= allowed), f"{what}: worst {np.max(d / allowed):.3g} of the bound"


def make_block(T, D, h, H, V, density, fmt, seed=0, x_dtype=None):
    import torch
    from dynamic_column_sparse_b200.layer import Fp4Linear, SparseDeltaAttention, SparseDeltaBlock, SparseDeltaMLP
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
    attn = SparseDeltaAttention(T, h, "cuda", density)
    mlp = SparseDeltaMLP(n(H, D, std=D ** -0.5), n(H, std=0.02), n(H, D, std=H ** -0.5), n(D, std=0.02), T, 128, density)
    mod = Fp4Linear(n(6 * D, V, std=0.3 * V ** -0.5), n(6 * D, std=0.1), 1, fmt)
    qkv = Fp4Linear(n(3 * h * 128, D, std=D ** -0.5), n(3 * h * 128, std=0.02), T, fmt)
    proj = Fp4Linear(n(D, h * 128, std=(h * 128) ** -0.5), n(D, std=0.02), T, fmt)
    block = SparseDeltaBlock(attn, mlp, mod, qkv, proj, 1 + n(128, std=0.1), 1 + n(128, std=0.1))
    ang = torch.rand(T, 64, generator=g, device="cuda") * 6
    x = n(T, D) + 0.3
    if x_dtype is not None:
        x = x.to(x_dtype)
    return block, x, n(1, V), ang.cos(), ang.sin(), n


def fp4_values(q):
    from dynamic_column_sparse_b200 import chipmunk as cm
    import torch
    return f64(cm.dequantize_fp4_rows(q, dtype=torch.float32))


def check_projection(lin, xv, out, what):
    wv = fp4_values(lin.w)
    ref = R.linear(xv, wv, f64(lin.bias))
    S = np.abs(xv) @ np.abs(wv).T + np.abs(f64(lin.bias))
    close(f64(out), ref, (xv.shape[1] / 64 + 8) * 2 * U * S, what)


@pytest.mark.parametrize("fmt,x32", [("nvfp4", False), ("mxfp4", True)])
def test_block_stages_match_their_definitions(fmt, x32):
    import torch
    from dynamic_column_sparse_b200 import chipmunk as cm
    T, D, h, H = 300, 256, 2, 512
    block, x, vec, cos, sin, n = make_block(T, D, h, H, 128, 400, fmt, x_dtype=torch.float32 if x32 else None)
    for dense in (True, False):
        if not dense:
            x += n(T, D, std=0.03).to(x.dtype)
        x0 = f64(x)
        (block.refresh if dense else block.step)(x, vec, cos, sin)
        torch.cuda.synchronize()
        assert cm.read_device_status() == 0
        m = f64(block.m)
        check_projection(block.mod, R.fp4_values(*R.quantize_fp4(f64(vec), fmt), fmt), block.m, "mod")
        sh1, sc1, g1, sh2, sc2, g2 = (m[0, i * D:(i + 1) * D] for i in range(6))
        # the quantised norm: the codes of a bf16 rounding of h, each value of h within 4 u-bounds of the definition
        _, h_ref = R.norm_residual(x0, scale=sc1, shift=sh1)
        hv = fp4_values(block.h_rows)
        blk = R.BLOCK[fmt]
        amax = np.abs(h_ref).reshape(T, -1, blk).max(axis=2).repeat(blk, axis=1)
        assert np.all(np.abs(hv - h_ref) <= 0.27 * amax + 1e-6)       # one code step of the block, at most
        check_projection(block.qkv, hv, block.qkv_out, "qkv")
        q, k, v = R.qk_norm_rope(f64(block.qkv_out), h, f64(block.q_weight), f64(block.k_weight), f64(cos), f64(sin),
                                 "interleaved", 1e-6)
        for name, got, ref in (("q", block.q, q), ("k", block.k, k)):
            pair = np.sqrt((ref * ref).reshape(T, h, 64, 2).sum(3).repeat(2, axis=2))
            close(f64(got), ref, 48 * U * pair, name)
        np.testing.assert_array_equal(f64(block.v), v)
        if dense:
            hf = lambda t: np.ascontiguousarray(f64(t).transpose(1, 0, 2))
            o_ref, _ = O.dense_attention(hf(block.q), hf(block.k), hf(block.v), block.attn.scale)
            assert_parity(hf(block.attn.o), o_ref, "attention", bf16_out=True)
            W1 = f64(block.mlp.w1t).T
            _, y_ref = O.dense_mlp(f64(block.h2), W1, f64(block.mlp.b1), f64(block.mlp.w2), f64(block.mlp.b2))
            assert_parity(f64(block.mlp.out), y_ref, "mlp", bf16_out=True)
        o = f64(block.attn.o).reshape(T, h * 128)
        check_projection(block.proj, R.fp4_values(*R.quantize_fp4(o, fmt), fmt), block.y, "proj")
        # the residual stream is rounded to x's type after each layer
        r1, h2_ref = R.norm_residual(x0, f64(block.y), gate=g1, scale=sc2, shift=sh2)
        c = r1 - r1.mean(axis=1, keepdims=True)
        rstd = 1 / np.sqrt((c * c).mean(axis=1, keepdims=True) + 1e-6)
        M = np.abs(x0) + np.abs(g1 * f64(block.y))
        M = ((M + M.mean(axis=1, keepdims=True)) * rstd + np.abs(c) * rstd * (1 + M.mean(axis=1, keepdims=True) * rstd)) * np.abs(1 + sc2)
        close(f64(block.h2), h2_ref, 256 * U * (M + np.abs(sh2)), "h2")
        half = U if x32 else 2.0 ** -8
        r2 = r1 + g2 * f64(block.mlp.out)
        mag = np.abs(x0) + np.abs(g1 * f64(block.y)) + np.abs(g2 * f64(block.mlp.out))
        d = np.abs(f64(x) - r2)
        assert np.all(d <= half * (np.abs(r1) + np.abs(r2)) * (1 + half) + 16 * U * mag)


def test_block_sparse_step_with_everything_selected_equals_the_dense_one():
    """All keys and columns selected: the sparse step recomputes everything and differs by rounding only."""
    import torch
    a, x, vec, cos, sin, n = make_block(200, 256, 2, 384, 64, 1000, "nvfp4")
    b, *_ = make_block(200, 256, 2, 384, 64, 1000, "nvfp4")
    xa, xb = x.clone(), x.clone()
    a.refresh(xa, vec, cos, sin)
    b.refresh(xb, vec, cos, sin)
    assert torch.equal(xa, xb)
    x2 = x + n(200, 256, std=0.05)
    xa, xb = x2.clone(), x2.clone()
    a.step(xa, vec, cos, sin)
    b.refresh(xb, vec, cos, sin)
    assert_parity(f64(xa), f64(xb), "sparse against dense", bf16_out=True)


def test_block_in_a_schedule_and_in_a_graph():
    """A captured sparse step, replayed, gives what the eager step gives, step after step."""
    import torch
    from dynamic_column_sparse_b200 import chipmunk as cm
    from dynamic_column_sparse_b200.layer import Schedule
    eager, x, vec, cos, sin, n = make_block(150, 128, 1, 256, 64, 300, "nvfp4")
    graphed, *_ = make_block(150, 128, 1, 256, 64, 300, "nvfp4")
    sched = Schedule({0, 3})
    static = x.clone()
    g = None
    for step in range(5):
        x1 = x + n(150, 128, std=0.03)
        xe = x1.clone()
        sched.run(eager, step, xe, vec, cos, sin)
        static.copy_(x1)
        if sched.is_dense(step):
            graphed.refresh(static, vec, cos, sin)
        else:
            if g is None:
                snapshot = [t.clone() for t in (static, graphed.mlp.a_cache, graphed.mlp.y_cache)]
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    graphed.step(static, vec, cos, sin)
                for t, s in zip((static, graphed.mlp.a_cache, graphed.mlp.y_cache), snapshot):
                    t.copy_(s)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(xe, static), step
    assert cm.read_device_status() == 0


def test_block_on_another_stream():
    import torch
    a, x, vec, cos, sin, n = make_block(130, 128, 1, 256, 64, 300, "mxfp4")
    b, *_ = make_block(130, 128, 1, 256, 64, 300, "mxfp4")
    xa, xb = x.clone(), x.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for f in ("refresh", "step"):
        getattr(a, f)(xa, vec, cos, sin)
        getattr(b, f)(xb, vec, cos, sin, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(xa, xb)


def test_block_refuses_parts_that_do_not_fit():
    import torch
    from dynamic_column_sparse_b200.layer import Fp4Linear, SparseDeltaBlock
    block, *_ , n = make_block(130, 128, 1, 256, 64, 300, "nvfp4")
    parts = lambda **kw: SparseDeltaBlock(**{**dict(attn=block.attn, mlp=block.mlp, mod=block.mod, qkv=block.qkv,
                                                     proj=block.proj, q_weight=block.q_weight, k_weight=block.k_weight), **kw})
    parts()
    with pytest.raises(ValueError, match="proj"):
        parts(proj=Fp4Linear(n(128, 256), None, 130))
    with pytest.raises(ValueError, match="proj"):
        parts(proj=Fp4Linear(n(128, 128), None, 100))
    with pytest.raises(ValueError, match="qkv"):
        parts(qkv=block.proj)
    with pytest.raises(ValueError, match="rows"):
        block.proj(torch.zeros((131, 128), dtype=torch.bfloat16, device="cuda"))
