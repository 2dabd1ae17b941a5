"""The 4-bit product in each form of its kernel against its 64-bit definition, all outputs compared.

Values and weights are quantised by the 64-bit definition or read back exactly; the product itself is
summed in 64 bits on the device. Tolerance: (K / 64 + 8) * 2u * S with S = sum |x w| + |bias| for the
fp32 sums and the epilogue (u = 2^-24, as for the smaller products), and half a step of the stored type."""
import math

import numpy as np
import pytest

from linear_forms import NAMES, PAIR, SINGLE, SIZES, WIDE
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


class Product:
    """Inputs of a T x N x K product and its definition in 64 bits."""

    def __init__(self, cm, T, N, K, fmt, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + N + K)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.cm, self.shape = cm, (T, N, K)
        x = n(T, K) * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device="cuda").float())
        x[:, torch.randint(0, K, (max(1, K // 100),), generator=g, device="cuda")] *= 30
        self.x = x.bfloat16()
        # every row of w its own row scale
        self.w = cm.quantize_fp4_rows((n(N, K) * K ** -0.5 * torch.exp2(torch.randint(-4, 5, (N, 1), generator=g, device="cuda").float())).bfloat16(), fmt)
        self.bias = n(N).bfloat16()
        self.xq = cm.quantize_fp4_rows(self.x, fmt)
        xv = torch.from_numpy(R.fp4_values(*R.quantize_fp4(f64(self.x), fmt), fmt)).cuda()
        wv = cm.dequantize_fp4_rows(self.w, dtype=torch.float32).double()
        self.sums, self.mag = xv @ wv.t(), xv.abs() @ wv.abs().t()

    def check(self, bias=True, act="none", out_dtype=None, quantised=False, out=None):
        import torch
        out_dtype = out_dtype or torch.bfloat16
        T, N, K = self.shape
        out = self.cm.linear_fp4(self.xq if quantised else self.x, self.w, self.bias if bias else None, act=act,
                                 out_dtype=out_dtype, out=out)
        u, S = self.sums, self.mag
        if bias:
            u, S = u + self.bias.double(), S + self.bias.double().abs()
        ref, slack = u, (K / 64 + 8) * 2 * U * S
        if act == "gelu":     # slope below 1.13, its own evaluation a few 2^-21 of its argument
            ref = 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
            slack = 1.13 * slack + 2.0 ** -19 * u.abs()
        d, allowed = (out.double() - ref).abs(), (2.0 ** -8 if out.dtype == torch.bfloat16 else U) * ref.abs() + slack
        bad = ~(d <= allowed)
        assert not bool(bad.any()), (f"{self.shape} act={act} {out.dtype}: {int(bad.sum())} outside, first at "
                                     f"{bad.nonzero()[0].tolist()}, worst {float((d / allowed).max()):.3g} of the bound")
        return out


CASES = [(form, *size) for form, sizes in SIZES.items() for size in sizes]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("form,T,N,K", CASES, ids=[f"{NAMES[c[0]]}-{c[1]}x{c[2]}x{c[3]}" for c in CASES])
def test_every_form_matches_the_definition(cm, form, T, N, K, fmt):
    import torch
    assert cm.load_library().chipmunk_selftest_linear_fp4_form(T, N, K, 0) == form
    p = Product(cm, T, N, K, fmt)
    first = p.check()
    assert torch.equal(first, p.check())                      # the same from run to run
    p.check(bias=False, quantised=True)
    p.check(out_dtype=torch.float32)
    p.check(act="gelu")
    p.check(act="gelu", out_dtype=torch.float32, quantised=True, bias=False)


@pytest.mark.parametrize("form", [PAIR, WIDE], ids=NAMES.get)
def test_large_forms_leave_the_rows_behind_theirs(cm, form):
    """Output rows behind the last one keep what they held, the output's last tile being ragged both ways."""
    import torch
    T, N, K = SIZES[form][0]
    p = Product(cm, T, N, K, "nvfp4")
    for dtype in (torch.bfloat16, torch.float32):
        big = torch.full((T + 300, N), 7.0, dtype=dtype, device="cuda")
        p.check(out=big[:T])
        assert bool((big[T:] == 7).all())


@pytest.mark.parametrize("form", [SINGLE, PAIR, WIDE], ids=NAMES.get)
def test_rows_that_are_not_finite_stay_in_their_rows_in_every_form(cm, form):
    """A row with a NaN or an infinity gives a row of NaN; the rest of its tile and of the next is untouched."""
    import torch
    T, N, K = SIZES[form][0]
    for fmt in ("nvfp4", "mxfp4"):
        p = Product(cm, T, N, K, fmt)
        clean = cm.linear_fp4(p.x, p.w, p.bias)
        x = p.x.clone()
        rows = [0, 130, 255, T - 1]
        for i, r in enumerate(rows):
            x[r, (37 * i) % K] = float("nan") if i % 2 else float("inf")
        got = cm.linear_fp4(x, p.w, p.bias)
        good = torch.ones(T, dtype=torch.bool, device="cuda")
        good[rows] = False
        assert bool(got[rows].isnan().all()) and torch.equal(got[good], clean[good])


@pytest.mark.parametrize("form", [SINGLE, PAIR, WIDE], ids=NAMES.get)
def test_every_form_is_skipped_while_the_status_word_is_set(cm, form):
    """A wait that ran out elsewhere: the product returns without touching its output, behind its own (skipped)
    quantiser and on quantised x; with the word cleared the same calls match the definition."""
    import torch
    T, N, K = SIZES[form][0]
    lib = cm.load_library()
    assert lib.chipmunk_selftest_linear_fp4_form(T, N, K, 0) == form == lib.chipmunk_selftest_linear_fp4_form(T, N, K, 1)
    p = Product(cm, T, N, K, "nvfp4")
    outs = [torch.full((T, N), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    assert lib.chipmunk_selftest_bounded_wait(torch.cuda.current_stream().cuda_stream) == 0
    cm.linear_fp4(p.x, p.w, p.bias, out=outs[0])
    cm.linear_fp4(p.xq, p.w, p.bias, out=outs[1])
    torch.cuda.synchronize()
    for out in outs:
        assert bool((out == 3).all())
    assert cm.read_device_status() == 1
    p.check(out=outs[0])
    p.check(out=outs[1], quantised=True)


@pytest.mark.parametrize("form", [PAIR, WIDE], ids=NAMES.get)
def test_large_forms_in_a_graph_and_on_two_streams(cm, form):
    """A captured norm and product replayed on other inputs, and two products at once, give the eager results."""
    import torch
    T, N, K = SIZES[form][0]
    p = Product(cm, T, N, K, "nvfp4")

    def chain(x, **kw):
        _, h = cm.norm_residual(x, out_format="nvfp4", **kw)
        return cm.linear_fp4(h, p.w, p.bias, **kw), cm.linear_fp4(x, p.w, p.bias, act="gelu", **kw)

    want = [chain(p.x), chain(-2 * p.x)]
    static = p.x.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    both = [chain(static, stream=side), chain(static)]
    side.synchronize()
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(a, b) for a, b in zip(want[0], got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = chain(static)
    for x, ref in ((p.x, want[0]), (-2 * p.x, want[1])):
        static.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))


@pytest.mark.parametrize("T", [1, 40], ids=["rows", "single"])
def test_gelu_over_its_range(cm, T):
    """Products of zero rows are the bias, exactly: GELU alone. With 2z the exponent (within 7u of its value in
    fp32), the result's relative error is at most 2 |z| 7u, and 2^-20 for exp2, the sum and the division."""
    import torch
    u = torch.linspace(-9.5, 9.5, 4096, device="cuda").bfloat16()
    w = cm.quantize_fp4_rows(torch.ones(u.numel(), 32, device="cuda").bfloat16())
    x = torch.zeros(T, 32, device="cuda").bfloat16()
    got = cm.linear_fp4(x, w, u, act="gelu", out_dtype=torch.float32).double()
    u = u.double()
    z2 = 2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)
    ref = (u / (1 + torch.exp(-z2))).expand(T, -1)
    assert bool(((got - ref).abs() <= (z2.abs() * 7 * U + 2.0 ** -20) * ref.abs()).all())
