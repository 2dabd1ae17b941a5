"""Cases that measure the operators around a layer's sparse attention and MLP.

A diffusion-transformer block wraps the two sparse-delta layers of this library
in norms, gates, projections and a head split. The operators measured here are

* ``norm``:   r = res_scale * res + gate * post_norm(y);  h = pre_norm(r) * (1 + scale) + shift
* ``quant``:  rows to 4-bit microscaled codes and back to the values they stand for
* ``linear``: x W^T + b with both operands in a 4-bit microscaled format (``entry``
              cases take x through the modulated norm first, as a block's first
              projection does)
* ``heads``:  a fused projection split into q, k, v, with the norm of every q and k
              head and the rotation by position

``own`` chooses between the plain torch form and the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # text tokens of one prompt entering a block: modulated norm only, latency counts
        {"name": "norm_text_512", "op": "norm", "T": 512, "D": 3072, "B": 1, "kind": "layer", "post": "none",
         "res": "bf16", "y": False},
        # the image + text rows of the 1280x768 layer between attention and MLP
        {"name": "norm_mid_4352", "op": "norm", "T": 4352, "D": 3072, "B": 1, "kind": "layer", "post": "none",
         "res": "bf16", "y": True},
        # the 720p video layer as packed samples: sandwich norms on an fp32 residual stream, ragged sample ends
        {"name": "norm_video_118800", "op": "norm", "T": 118800, "D": 3072, "B": 5, "kind": "rms", "post": "rms",
         "res": "fp32", "y": True},
        # hidden activations of the 1280x768 layer's MLP
        {"name": "quant_hidden_4352", "op": "quant", "T": 4352, "D": 12288, "fmt": "nvfp4"},
        # a video layer's rows, power-of-two scales
        {"name": "quant_video_118800", "op": "quant", "T": 118800, "D": 3072, "fmt": "mxfp4"},
        # one step's modulation vectors from its time embedding: one row against the whole weight
        {"name": "linear_mod_1", "op": "linear", "T": 1, "D": 3072, "N": 18432, "fmt": "nvfp4", "act": "none"},
        # a ragged prompt through the first MLP projection
        {"name": "linear_text_333", "op": "linear", "T": 333, "D": 3072, "N": 12288, "fmt": "mxfp4", "act": "gelu"},
        # second MLP projection of the 1280x768 layer's dense rows (long sum)
        {"name": "linear_down_4352", "op": "linear", "T": 4352, "D": 12288, "N": 3072, "fmt": "nvfp4", "act": "none"},
        # norm, quantisation and the fused q, k, v projection of the 1280x768 layer
        {"name": "entry_qkv_4352", "op": "entry", "T": 4352, "D": 3072, "N": 9216, "fmt": "nvfp4", "act": "none"},
        # attention's output projection over a whole video layer
        {"name": "linear_video_118800", "op": "linear", "T": 118800, "D": 3072, "N": 3072, "fmt": "nvfp4",
         "act": "none"},
        # 24 heads of the 1280x768 layer out of its fused projection
        {"name": "heads_4352", "op": "heads", "T": 4352, "h": 24, "extra": 0, "pairs": "interleaved"},
        # the 2304x1280 layer, heads read out of a projection that also carries the MLP's hidden columns
        {"name": "heads_wide_12032", "op": "heads", "T": 12032, "h": 24, "extra": 12288, "pairs": "interleaved"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "linear", "linear", "entry", "heads"])
    T = _log(rng, 1, 29000)
    if op == "norm":
        y = rng.random() < 0.75
        return {"op": op, "T": T, "D": 8 * _log(rng, 8, 1024), "B": rng.randint(1, min(T, 7)),
                "kind": rng.choice(["layer", "rms"]), "post": rng.choice(["none", "rms", "layer"]) if y else "none",
                "res": rng.choice(["bf16", "fp32"]), "y": y}
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    if op == "quant":
        return {"op": op, "T": T, "D": 32 * _log(rng, 2, min(512, 11000000 // T)), "fmt": fmt}
    if op == "heads":
        h = _log(rng, 1, 48)
        return {"op": op, "T": min(T, 12000), "h": h, "extra": rng.choice([0, 0, 8 * rng.randint(1, 1000)]),
                "pairs": rng.choice(["interleaved", "interleaved", "halves"])}
    return {"op": op, "T": T, "D": 32 * _log(rng, 2, 128), "N": 8 * _log(rng, 8, 1152), "fmt": fmt,
            "act": rng.choice(["none", "none", "gelu"])}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    t = torch.randn(*shape, generator=g, device=DEV)
    return t.mul_(std).to(dtype)


def _offsets(T, B, seed):
    """Sample boundaries 0 <= ... <= T' of B packed samples; with several samples the last rows may belong to none."""
    if B == 1:
        return [0, T]
    g = torch.Generator().manual_seed(seed)
    end = T - (T % 7 if T > 16 else 0)
    cuts = torch.randint(0, end + 1, (B - 1,), generator=g).sort().values.tolist()
    return [0] + cuts + [end]


def _rows_in(g, T, D):
    """Rows as a block sees them: normal values, a scale for each row, some channels much larger than the rest."""
    x = torch.randn(T, D, generator=g, device=DEV)
    x *= torch.rand(T, 1, generator=g, device=DEV).mul_(2).add_(0.25)
    loud = torch.randint(0, D, (max(1, D // 256),), generator=g, device=DEV)
    x[:, loud] *= 8.0
    return x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "norm":
        T, D, B = case["T"], case["D"], case["B"]
        s["x"] = _rows_in(g, T, D).add_(0.3).to(torch.float32 if case["res"] == "fp32" else torch.bfloat16)
        s["y_in"] = _normal(g, T, D, std=0.7) if case["y"] else None
        mod = _normal(g, B, 3 * D, std=0.3)  # one projection gives gate, scale and shift of a sample
        s["gate"], s["scale"], s["shift"] = mod[:, :D], mod[:, D:2 * D], mod[:, 2 * D:]
        s["post_w"] = _normal(g, D, std=0.2).add_(1) if case["post"] != "none" else None
        off = _offsets(T, B, seed)
        s["end"] = off[-1]
        s["off"] = torch.tensor(off, dtype=torch.int32, device=DEV) if B > 1 else None
        s["res_out"] = torch.zeros_like(s["x"]) if case["y"] else None
        s["h"] = torch.zeros(T, D, dtype=torch.bfloat16, device=DEV)
        return s
    if op == "heads":
        T, h = case["T"], case["h"]
        s["qkv"] = _normal(g, T, 3 * h * 128 + case["extra"])
        s["qw"], s["kw"] = (_normal(g, 128, std=0.2).add_(1) for _ in range(2))
        ang = torch.rand(T, 64, generator=g, device=DEV) * (2 * math.pi)
        s["cos"], s["sin"] = ang.cos(), ang.sin()
        s["q"], s["k"], s["v"] = (torch.empty(T, h, 128, dtype=torch.bfloat16, device=DEV) for _ in range(3))
        return s
    T, D = case["T"], case["D"]
    s["x"] = _rows_in(g, T, D).to(torch.bfloat16)
    if op == "quant":
        return s
    N = case["N"]
    w = _normal(g, N, D, std=D ** -0.5)
    codes, bs, rs = _quantize(w, case["fmt"])
    s["codes"], s["bs"], s["rs"] = _pack(codes), _tiled(bs, case["fmt"]), rs
    s["bias"] = _normal(g, N, std=0.1)
    s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    if op == "entry":
        mod = _normal(g, 1, 2 * D, std=0.3)
        s["scale"], s["shift"] = mod[:, :D], mod[:, D:]
    return s


# ------------------------------------------------------------------ the plain forms

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _code(a):
    """e2m1 code of a magnitude: nearest, ties to the even code, 6 at most."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _pow2(e):
    """2^e in fp32 for e in [-127, 127], by its bits."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantize(x, fmt):
    """Codes [R][C] (sign in bit 3), block-scale bytes [R][C / block], row scales [R] (nvfp4)."""
    R, C = x.shape
    b = x.float().view(R, C // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(2)
    if fmt == "mxfp4":
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)  # floor(log2 amax) - 2
        e = torch.where(amax > 0, e, -127)
        bs, rs = (e + 127).to(torch.uint8), None
        step = _pow2(e)
    else:
        row = amax.amax(1)
        e = (torch.frexp(row)[1] - 11).clamp(-110, 117)  # floor(log2 row) - 10
        rs = torch.where(row > 0, _pow2(e), 1.0)
        f8 = (amax / (6.0 * rs[:, None])).to(torch.float8_e4m3fn)
        bs = f8.view(torch.uint8)
        step = f8.float() * rs[:, None]
    t = torch.where(step[:, :, None] > 0, b / step[:, :, None], 0.0)
    codes = _code(t.abs()) + (torch.signbit(t) & (t != 0)).to(torch.uint8) * 8
    return codes.view(R, C), bs, rs


def _values(codes, bs, rs, fmt):
    """The fp32 values that codes and scales stand for."""
    R, C = codes.shape
    mag = torch.tensor(_E2M1, device=codes.device)[(codes & 7).long()]
    v = torch.where(codes >= 8, -mag, mag).view(R, C // BLOCK[fmt], BLOCK[fmt])
    if fmt == "mxfp4":
        step = _pow2(bs.int() - 127)
    else:
        step = bs.view(torch.float8_e4m3fn).float() * rs[:, None]
    return (v * step[:, :, None]).view(R, C)


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1)


def _tiled(bs, fmt):
    """Block scales in the tensor core's order: tiles of 128 rows x 4 scales, byte (r % 32) * 16 + (r / 32) * 4 + c."""
    R, n = bs.shape
    per = 256 // BLOCK[fmt]
    rt, ct = -(-R // 128), -(-n // per) * (per // 4)
    p = torch.zeros(rt * 128, ct * 4, dtype=torch.uint8, device=bs.device)
    p[:R, :n] = bs
    return p.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous().view(rt, ct, 512)


def _untiled(t, R, n):
    rt, ct, _ = t.shape
    return t.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:R, :n]


def _norm(x, kind, eps=1e-6):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(1, keepdim=True) + eps)


def _per_row(v, off, T):
    """Rows of a per-sample vector [B][D] for every row of the samples."""
    if off is None:
        return v.float()
    row = torch.arange(T, device=v.device, dtype=torch.int32)
    return v.float()[torch.searchsorted(off[1:], row, right=True)]


def _plain_norm(s):
    end = s["end"]
    r = s["x"][:end].float()
    if s["y"]:
        y = s["y_in"][:end].float()
        if s["post"] != "none":
            y = _norm(y, s["post"]) * s["post_w"].float()
        r = r + _per_row(s["gate"], s["off"], end) * y
        s["res_out"][:end] = r.to(s["x"].dtype)
    h = _norm(r, s["kind"]) * (1 + _per_row(s["scale"], s["off"], end)) + _per_row(s["shift"], s["off"], end)
    s["h"][:end] = h.to(torch.bfloat16)
    return {"res": s["res_out"], "h": s["h"]} if s["y"] else {"h": s["h"]}


def _plain_linear(s, x):
    fmt, N, D = s["fmt"], s["N"], s["D"]
    a = _values(*_quantize(x, fmt), fmt)
    w = _values(_unpack(s["codes"]), _untiled(s["bs"], N, D // BLOCK[fmt]), s["rs"], fmt)
    o = a @ w.t() + s["bias"].float()
    if s["act"] == "gelu":
        o = 0.5 * o * (1 + torch.tanh(math.sqrt(2 / math.pi) * (o + 0.044715 * o * o * o)))
    return o.to(torch.bfloat16)


def _rotate(x, cos, sin, pairs):
    c, n = cos[:, None, :], sin[:, None, :]
    if pairs == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * n, a * n + b * c), 3).flatten(2)
    a, b = x[..., :64], x[..., 64:]
    return torch.cat((a * c - b * n, a * n + b * c), 2)


def _plain_heads(s):
    T, h = s["T"], s["h"]
    q, k, v = s["qkv"][:, :3 * h * 128].view(T, 3, h, 128).unbind(1)

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w.float()
        return _rotate(x, s["cos"], s["sin"], s["pairs"]).to(torch.bfloat16)

    return {"q": one(q, s["qw"]), "k": one(k, s["kw"]), "v": v.contiguous()}


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "heads":
        return _plain_heads(s)
    if op == "quant":
        return _values(*_quantize(s["x"], s["fmt"]), s["fmt"]).to(torch.bfloat16)
    x = s["x"]
    if op == "entry":
        x = (_norm(x.float(), "layer") * (1 + s["scale"].float()) + s["shift"].float()).to(torch.bfloat16)
    return _plain_linear(s, x)


def _own(s):
    from dynamic_column_sparse_b200 import chipmunk as cm
    op = s["op"]
    if op == "norm":
        if s["y"]:
            r, h = cm.norm_residual(s["x"], s["y_in"], gate=s["gate"], post_norm=s["post"], post_weight=s["post_w"],
                                    res_out=s["res_out"], norm=s["kind"], scale=s["scale"], shift=s["shift"],
                                    offsets=s["off"], out=s["h"])
            return {"res": r, "h": h}
        _, h = cm.norm_residual(s["x"], norm=s["kind"], scale=s["scale"], shift=s["shift"], offsets=s["off"],
                                out=s["h"])
        return {"h": h}
    if op == "heads":
        q, k, v = cm.qk_norm_rope(s["qkv"], s["h"], s["qw"], s["kw"], s["cos"], s["sin"], pairs=s["pairs"], q=s["q"],
                                  k=s["k"], v=s["v"])
        return {"q": q, "k": k, "v": v}
    if op == "quant":
        return cm.dequantize_fp4_rows(cm.quantize_fp4_rows(s["x"], s["fmt"]))
    w = cm.Fp4Rows(s["codes"], s["bs"], s["rs"], s["fmt"], s["N"], s["D"])
    x = s["x"]
    if op == "entry":
        _, x = cm.norm_residual(x, norm="layer", scale=s["scale"], shift=s["shift"], out_format=s["fmt"])
    return cm.linear_fp4(x, w, s["bias"], out=s["out"], act=s["act"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "norm":
        T, D = case["T"], case["D"]
        r = 4 if case["res"] == "fp32" else 2
        per = r + 2 + ((2 + r) if case["y"] else 0)  # residual in, h out; y in and residual out
        return {"bytes": T * D * per + case["B"] * D * 2 * (3 if case["y"] else 2), "flops": T * D * 12}
    if op == "heads":
        T, h = case["T"], case["h"]
        return {"bytes": T * (3 * h * 128 * 4 + 512), "flops": T * h * 256 * 7}
    T, D = case["T"], case["D"]
    if op == "quant":
        return {"bytes": 4 * T * D, "flops": 4 * T * D}
    N = case["N"]
    w_bytes = N * D // 2 + N * (D // BLOCK[case["fmt"]])
    return {"bytes": 2 * T * D + w_bytes + 2 * T * N + 2 * N, "flops": 2 * T * D * N}


# ------------------------------------------------------------------ the definition in 64 bits

def _x_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _x_round(a, bits, emin, top):
    """`a` (>= 0, 64 bits) to the nearest number of `bits` significant bits, ties to even, exponents from emin, top at most."""
    e = (torch.frexp(a)[1] - 1).clamp(min=emin) - (bits - 1)
    return (torch.round(a * _x_pow2(-e)) * _x_pow2(e)).clamp(max=top)


def _x_fp4(x, fmt):
    """The values that 4-bit rows of x stand for."""
    R, C = x.shape
    v = x.double().view(R, -1, BLOCK[fmt])
    big = v.abs().max(2, keepdim=True).values
    if fmt == "mxfp4":
        unit = _x_pow2((torch.frexp(big)[1] - 3).clamp(-127, 127))
    else:
        row = big.max(1, keepdim=True).values
        rs = _x_pow2((torch.frexp(row)[1] - 11).clamp(-110, 117))
        unit = _x_round(big / (6 * rs), 4, -6, 448.0) * rs
    q = _x_round((v / unit).abs().nan_to_num(0.0, 0.0, 0.0), 2, 0, 6.0)
    return (torch.sign(v) * q * unit).view(R, C)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _x_fp4(s["x"], s["fmt"])
    if op == "heads":
        T, h = case["T"], case["h"]
        x = s["qkv"][:, :3 * h * 128].double().view(T, 3, h, 128)
        rot = torch.complex(s["cos"].double(), s["sin"].double())

        def one(i, w):
            t = x[:, i]
            t = t / torch.sqrt(t.square().sum(2, keepdim=True) / 128 + 1e-6) * w.double()
            if case["pairs"] == "interleaved":
                z = torch.view_as_complex(t.reshape(T, h, 64, 2).contiguous())
                return torch.view_as_real(z * rot[:, None]).reshape(T, h, 128)
            z = torch.complex(t[..., :64].contiguous(), t[..., 64:].contiguous()) * rot[:, None]
            return torch.cat((z.real, z.imag), 2)

        return {"q": one(0, s["qw"]), "k": one(1, s["kw"]), "v": x[:, 2].contiguous()}

    def norm(t, kind):
        if kind == "layer":
            return torch.nn.functional.layer_norm(t, t.shape[1:], eps=1e-6)
        return t / torch.sqrt(t.square().sum(1, keepdim=True) / t.shape[1] + 1e-6)

    if op == "norm":
        T, D, end = case["T"], case["D"], s["end"]
        h = torch.zeros(T, D, dtype=torch.float64, device=DEV)
        res = torch.zeros(T, D, dtype=torch.float64, device=DEV)
        off = [0, T] if s["off"] is None else s["off"].tolist()
        for b in range(case["B"]):
            lo, hi = off[b], off[b + 1]
            if lo == hi:
                continue
            r = s["x"][lo:hi].double()
            if case["y"]:
                y = s["y_in"][lo:hi].double()
                if case["post"] != "none":
                    y = norm(y, case["post"]) * s["post_w"].double()
                r = r + y * s["gate"][b].double()
            res[lo:hi] = r
            h[lo:hi] = norm(r, case["kind"]) * (s["scale"][b].double() + 1) + s["shift"][b].double()
        return {"res": res, "h": h} if case["y"] else {"h": h}
    x = s["x"]
    if op == "entry":
        x = (norm(x.double(), "layer") * (s["scale"].double() + 1) + s["shift"].double()).to(torch.bfloat16)
    w = _normal_weights(case, seed)
    o = _x_fp4(x, case["fmt"]) @ _x_fp4(w, case["fmt"]).t() + s["bias"].double()
    if case["act"] == "gelu":
        o = torch.nn.functional.gelu(o, approximate="tanh")
    return o


def _normal_weights(case, seed):
    """The bf16 weights that prepare() quantises."""
    g = _gen(seed)
    _rows_in(g, case["T"], case["D"])
    return _normal(g, case["N"], case["D"], std=case["D"] ** -0.5)
