"""Per-layer state for the column-sparse delta method: caches, selections, schedule.

A diffusion transformer calls each layer once per denoising step. On a dense
(refresh) step the layer runs fully, scores every intermediate column, picks
the columns to recompute per token block and rebuilds its caches; on the
sparse steps in between it recomputes only those columns against the caches
(Chipmunk blog post, "Activation Deltas Across Diffusion Steps are Very
Sparse"; the HunyuanVideo table footnote runs 6 of 50 steps denser).

``SparseDeltaBlock`` puts the two layers into the block they belong to, with its
norms, gates, 4-bit projections (``Fp4Linear``) and head split.

These classes own the device buffers and call the C ABI through
``dynamic_column_sparse_b200.chipmunk``; all arithmetic runs in the library's
CUDA kernels.
"""
from __future__ import annotations

import math

import torch

from . import chipmunk as cm


def k_from_density(n: int, density_permille: int) -> int:
    """Selected count per block for a kept fraction in per mille, rounded down."""
    return (int(n) * int(density_permille)) // 1000


class SparseDeltaMLP:
    """MLP ``gelu(x W1 + b1) W2 + b2`` with an activation / output cache.

    Weights: ``w1t`` [H][D] (W1 transposed), ``b1`` [H], ``w2`` [H][D],
    ``b2`` [D], all bf16 on one CUDA device. ``density_permille`` is the
    kept fraction of hidden columns per ``Bt``-token block.
    """

    def __init__(self, w1t, b1, w2, b2, T: int, Bt: int = 128, density_permille: int = 300):
        H, D = w1t.shape
        dev = w1t.device
        self.w1t, self.b1, self.w2, self.b2 = w1t, b1, w2, b2
        self.T, self.D, self.H, self.Bt = T, D, H, Bt
        self.nb = (T + Bt - 1) // Bt
        self.k = k_from_density(H, density_permille)
        self.a_cache = torch.zeros((self.nb, H, Bt), dtype=torch.bfloat16, device=dev)
        self.y_cache = torch.zeros((T, D), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
        self.idx = torch.zeros((self.nb, self.k), dtype=torch.int32, device=dev)
        self.scores = torch.empty((self.nb, H), dtype=torch.float32, device=dev)
        self.workspace = torch.empty(cm.mlp_workspace_bytes(T, H, self.k, Bt), dtype=torch.uint8, device=dev)
        self.has_cache = False

    def refresh(self, x, stream=None):
        """Dense step: output, column scores, new selection, rebuilt caches."""
        cm.mlp_refresh(x, self.w1t, self.b1, self.w2, self.b2, self.a_cache, self.y_cache, self.idx, self.scores,
                       self.out, Bt=self.Bt, first_step=not self.has_cache, stream=stream)
        self.has_cache = True
        return self.out

    def step(self, x, stream=None):
        """Sparse step: recompute the selected columns against the caches."""
        if not self.has_cache:
            raise RuntimeError("a sparse step needs a refresh first")
        cm.mlp_delta(x, self.w1t, self.b1, self.w2, self.idx, self.a_cache, self.y_cache, self.out, Bt=self.Bt,
                     workspace=self.workspace, stream=stream)
        return self.out


class SparseDeltaAttention:
    """Attention ``softmax(scale q k^T) v`` per head with a cached complement partial.

    ``q, k, v`` are [T][h][128] bf16. ``density_permille`` is the kept
    fraction of keys per (head, 128-query block). With ``compact`` the
    complement is cached as ``lse_c`` (fp32) and the normalised ``o_c`` (bf16)
    instead of ``m_c``, ``l_c``, ``acc_c`` (fp32): half the bytes. With
    ``keep_mass`` the refresh also keeps the attention mass ``scores``
    [h][nb][T] (fp32); otherwise the mass never leaves the refresh kernel's
    row buffers.
    """

    def __init__(self, T: int, h: int, device, density_permille: int = 165, scale: float | None = None,
                 compact: bool = False, keep_mass: bool = False):
        d = 128
        self.T, self.h, self.d = T, h, d
        self.nb = (T + 127) // 128
        self.k = k_from_density(T, density_permille)
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        f32 = torch.float32
        self.idx = torch.zeros((h, self.nb, self.k), dtype=torch.int32, device=device)
        self.compact = compact
        if compact:
            self.lse_c = torch.empty((h, T), dtype=f32, device=device)
            self.o_c = torch.empty((h, T, d), dtype=torch.bfloat16, device=device)
            self.m_c = self.l_c = self.acc_c = None
        else:
            self.m_c = torch.empty((h, T), dtype=f32, device=device)
            self.l_c = torch.empty((h, T), dtype=f32, device=device)
            self.acc_c = torch.empty((h, T, d), dtype=f32, device=device)
            self.lse_c = self.o_c = None
        self.o = torch.empty((T, h, d), dtype=torch.bfloat16, device=device)
        self.scores = torch.empty((h, self.nb, T), dtype=f32, device=device) if keep_mass else None
        self.workspace = torch.empty(cm.attn_refresh_workspace_bytes(T, h, self.k, keep_mass), dtype=torch.uint8,
                                     device=device)
        self.has_cache = False

    def refresh(self, q, k, v, stream=None):
        """Dense step: output, attention mass, new key selection, complement cache."""
        cm.attn_refresh(q, k, v, self.idx, self.m_c, self.l_c, self.acc_c, self.o, self.scores, scale=self.scale,
                        workspace=self.workspace, stream=stream, lse_c=self.lse_c, o_c=self.o_c)
        self.has_cache = True
        return self.o

    def step(self, q, k, v, stream=None):
        """Sparse step: selected keys with the current q, k, v, merged with the cached complement."""
        if not self.has_cache:
            raise RuntimeError("a sparse step needs a refresh first")
        if self.compact:
            cm.attn_delta_compact(q, k, v, self.idx, self.lse_c, self.o_c, self.o, scale=self.scale, stream=stream)
        else:
            cm.attn_delta(q, k, v, self.idx, self.m_c, self.l_c, self.acc_c, self.o, scale=self.scale, stream=stream)
        return self.o


class Fp4Linear:
    """Dense projection ``act(x W^T + bias)`` with its weight kept as 4-bit microscaled rows.

    ``weight`` [N][K] and ``bias`` [N] bf16 on one CUDA device; the weight is quantised once, here. ``T`` rows at
    most per call (the scratch for the quantised x is sized for them; calls that run at the same time need
    an object each)."""

    def __init__(self, weight, bias=None, T: int = 1, fmt: str = "nvfp4", act: str = "none"):
        self.w = cm.quantize_fp4_rows(weight, fmt)
        self.bias, self.fmt, self.act = bias, fmt, act
        self.T = T
        self.workspace = torch.empty(cm.linear_fp4_workspace_bytes(T, self.w.cols, fmt), dtype=torch.uint8,
                                     device=weight.device)

    def __call__(self, x, out=None, stream=None):
        """x: bf16 [t][K], t <= T, or ``Fp4Rows``; out bf16 [t][N]."""
        if not isinstance(x, cm.Fp4Rows) and x.shape[0] > self.T:
            raise ValueError(f"{x.shape[0]} rows, the scratch is sized for {self.T}")
        return cm.linear_fp4(x, self.w, self.bias, out=out, act=self.act, workspace=self.workspace, stream=stream)


class SparseDeltaBlock:
    """A diffusion-transformer block around the two sparse-delta layers, on this library's kernels alone:

        shift1, scale1, gate1, shift2, scale2, gate2 = mod(vec)
        x += gate1 * proj(attn(heads(qkv(norm(x) * (1 + scale1) + shift1))))
        x += gate2 * mlp(norm(x) * (1 + scale2) + shift2)

    ``attn`` and ``mlp`` are the block's layers (same T); ``mod`` [6 D][...], ``qkv`` [3 h 128][D] and
    ``proj`` [D][h 128] are ``Fp4Linear`` of one format, built for 1, T and T rows; ``q_weight``, ``k_weight`` [128]
    bf16 weigh the norm of the q and k heads. ``refresh`` and ``step`` take x [T][D] (bf16 or fp32, updated
    in place), the activated conditioning ``vec`` [1][...] bf16 and the rotation's ``cos``, ``sin``
    [T][64] fp32, and return x, so that ``Schedule.run`` drives a block as it drives a layer."""

    def __init__(self, attn: SparseDeltaAttention, mlp: SparseDeltaMLP, mod: Fp4Linear, qkv: Fp4Linear, proj: Fp4Linear,
                 q_weight, k_weight, pairs: str = "interleaved", eps: float = 1e-6):
        T, D, h, dev = attn.T, mlp.D, attn.h, q_weight.device
        if mlp.T != T:
            raise ValueError(f"attention is built for {T} tokens, the MLP for {mlp.T}")
        want = {"mod": (mod, 6 * D, mod.w.cols), "qkv": (qkv, 3 * h * 128, D), "proj": (proj, D, h * 128)}
        for name, (lin, rows, cols) in want.items():
            if (lin.w.rows, lin.w.cols) != (rows, cols):
                raise ValueError(f"{name} has a weight of {lin.w.rows} x {lin.w.cols}, expected {rows} x {cols}")
        if proj.T < T:
            raise ValueError(f"proj is built for {proj.T} rows, the block has {T}")
        self.attn, self.mlp, self.mod, self.qkv, self.proj = attn, mlp, mod, qkv, proj
        self.q_weight, self.k_weight, self.pairs, self.eps = q_weight, k_weight, pairs, eps
        self.T, self.D, self.h = T, D, h
        bf = torch.bfloat16
        self.m = torch.empty((1, 6 * D), dtype=bf, device=dev)
        self.h_rows = cm.empty_fp4_rows(T, D, qkv.fmt, dev)
        self.qkv_out = torch.empty((T, 3 * h * 128), dtype=bf, device=dev)
        self.q, self.k, self.v = (torch.empty((T, h, 128), dtype=bf, device=dev) for _ in range(3))
        self.y = torch.empty((T, D), dtype=bf, device=dev)
        self.h2 = torch.empty((T, D), dtype=bf, device=dev)

    def _run(self, x, vec, cos, sin, dense, stream):
        D = self.D
        m = self.mod(vec, out=self.m, stream=stream)
        shift1, scale1, gate1, shift2, scale2, gate2 = (m[:, i * D:(i + 1) * D] for i in range(6))
        cm.norm_residual(x, scale=scale1, shift=shift1, eps=self.eps, out=self.h_rows, out_format=self.qkv.fmt,
                         stream=stream)
        self.qkv(self.h_rows, out=self.qkv_out, stream=stream)
        cm.qk_norm_rope(self.qkv_out, self.h, self.q_weight, self.k_weight, cos, sin, pairs=self.pairs, eps=self.eps,
                        q=self.q, k=self.k, v=self.v, stream=stream)
        attn = self.attn.refresh if dense else self.attn.step
        o = attn(self.q, self.k, self.v, stream=stream)
        self.proj(o.view(self.T, self.h * 128), out=self.y, stream=stream)
        cm.norm_residual(x, self.y, gate=gate1, res_out=x, scale=scale2, shift=shift2, eps=self.eps, out=self.h2,
                         stream=stream)
        mlp = self.mlp.refresh if dense else self.mlp.step
        cm.norm_residual(x, mlp(self.h2, stream=stream), gate=gate2, res_out=x, out_format=None, stream=stream)
        return x

    def refresh(self, x, vec, cos, sin, stream=None):
        """Dense step of both layers; x is updated in place."""
        return self._run(x, vec, cos, sin, True, stream)

    def step(self, x, vec, cos, sin, stream=None):
        """Sparse step of both layers; x is updated in place."""
        return self._run(x, vec, cos, sin, False, stream)


class Schedule:
    """Which denoising steps run dense: ``dense_steps`` (e.g. {0, 5} of 10)."""

    def __init__(self, dense_steps=(0,)):
        self.dense_steps = frozenset(dense_steps)

    def is_dense(self, step: int) -> bool:
        return step in self.dense_steps

    def run(self, layer, step: int, *inputs, stream=None):
        return layer.refresh(*inputs, stream=stream) if self.is_dense(step) else layer.step(*inputs, stream=stream)
