"""The layer operators around the NVFP4 product, as measured cases.

Operators: the root-mean-square norm with the residual's addition (bf16, fp32 or MXFP8 output) and its
gradient; the W4 product with bias, activation, gate and residual in its epilogue and its gradient; and the
MXFP8 form (E4M3 codes, one power-of-two scale per 32 values of a row) that activations are kept in.

``run`` computes a case in elementary torch operations, or, where ``own`` is set, by the framework's calls.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "fp32": F32}
EPS = 1e-6
MX = 32  # values per MXFP8 scale
GELU_C = math.sqrt(2.0 / math.pi)


# ---------------------------------------------------------------------------------------------- cases

def _norm(name, rows, cols, dtype="bf16", residual=True, out="bf16"):
    return dict(name=name, op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, out=out)


def _norm_grad(name, rows, cols, dtype="bf16", kept="plain", ds=True):
    return dict(name=name, op="norm_grad", rows=rows, cols=cols, dtype=dtype, kept=kept, ds=ds)


def _linear(name, rows, k, n, x="bf16", bias=False, act="none", gated=False, residual=False, out="bf16", keep="none"):
    return dict(name=name, op="linear", rows=rows, k=k, n=n, x=x, bias=bias, act=act, gated=gated,
                residual=residual, out=out, keep=keep)


def _linear_grad(name, rows, k, n, act="none", gated=False, kept="none", bias=False):
    return dict(name=name, op="linear_grad", rows=rows, k=k, n=n, act=act, gated=gated, kept=kept, bias=bias)


def _codec(name, op, rows, cols, dtype="bf16"):
    return dict(name=name, op=op, rows=rows, cols=cols, dtype=dtype)


def listed():
    return [
        # one token of a decoding step: the residual's addition and the norm of one row
        _norm("norm, one token", 1, 4096),
        # a long prompt: the norm writes the 8-bit input of the next products
        _norm("norm, prompt to 8 bits", 8192, 4096, out="mxfp8"),
        # a training step's backward pass through a norm, with the residual stream's own gradient
        _norm_grad("norm gradient", 8192, 4096),
        # the same from a kept 8-bit input, over a wide layer and an odd number of tokens
        _norm_grad("norm gradient from 8 bits", 777, 14336, kept="mxfp8"),
        # one token through a projection that adds to the residual stream
        _linear("product, one token", 1, 4096, 4096, residual=True),
        # a decoding batch through a gated up-projection, its 8-bit input from the norm
        _linear("product, batch, gated", 24, 4096, 11008, x="mxfp8", act="silu", gated=True),
        # a short prompt through an up-projection with a bias, odd sizes, its pre-activation kept for a backward pass
        _linear("product, short prompt", 333, 4112, 11000, bias=True, act="gelu", keep="bf16"),
        # training: a gated up-projection over 4096 tokens, its pre-activation kept in 8 bits
        _linear("product, training, gated", 4096, 4096, 11008, act="silu", gated=True, keep="mxfp8"),
        # the backward pass of an attention projection with a bias
        _linear_grad("product gradient", 4096, 4096, 4096, bias=True),
        # the backward pass of a gated up-projection over a short batch, from the kept 8 bits
        _linear_grad("product gradient, gated", 512, 4096, 11008, act="silu", gated=True, kept="mxfp8"),
        # a checkpoint of a layer's activations, written
        _codec("checkpoint, written", "to_mxfp8", 8192, 4096),
        # and a small odd one read back
        _codec("checkpoint, read", "from_mxfp8", 250, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2.0 * 4096 * 4096 * 22016


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "to_mxfp8", "from_mxfp8"])
    if op in ("norm", "norm_grad", "to_mxfp8", "from_mxfp8"):
        cols = _log(rng, 64, 16384)
        rows = min(_log(rng, 1, 16384), (1 << 26) // cols)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if op == "norm":
            c = _norm("", rows, cols, dtype, rng.random() < 0.7, rng.choice([dtype, "mxfp8"]))
        elif op == "norm_grad":
            c = _norm_grad("", rows, cols, dtype, rng.choice(["plain", "mxfp8"]), rng.random() < 0.6)
        else:
            c = _codec("", op, rows, cols, dtype)
    else:
        k = 16 * _log(rng, 16, 768)
        n = _log(rng, 256, 12288)
        rows = _log(rng, 1, 6144)
        act = rng.choice(["none", "silu", "gelu"])
        gated = act != "none" and rng.random() < 0.5
        if gated:
            n = max(32, n // 32 * 32)
        rows = max(1, min(rows, int(MOST_FLOPS / (2.0 * k * n * (1 + gated)))))
        kept = rng.choice(["bf16", "mxfp8"])
        if op == "linear":
            c = _linear("", rows, k, n, rng.choice(["bf16", "mxfp8"]), rng.random() < 0.4, act, gated,
                        rng.random() < 0.4, rng.choice(["bf16", "bf16", "fp32"]), kept if rng.random() < 0.4 else "none")
        else:
            c = _linear_grad("", rows, k, n, act, gated, kept if act != "none" else "none", rng.random() < 0.5)
    del c["name"]
    return c


# --------------------------------------------------------------------------------------------- inputs

def _make_weights(g, n, k):
    """NVFP4 codes, E4M3 scales and alpha of a random [n, k] matrix by the max rule."""
    w = torch.randn(n, k, generator=g, device="cuda").mul_(0.02)
    alpha = (w.abs().max() / 2688.0).reshape(1)
    amax = w.view(n, k // 16, 16).abs().amax(-1)
    s8 = (amax / (6.0 * alpha)).clamp_(max=448.0).to(torch.float8_e4m3fn)
    d = (s8.float() * alpha).clamp_min_(1e-30)
    x = w.view(n, k // 16, 16).div_(d[..., None]).view(n, k)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    idx = torch.bucketize(x.abs(), edges).to(torch.uint8)
    idx += ((x < 0) & (idx > 0)).to(torch.uint8) * 8
    codes = (idx[:, 0::2] | (idx[:, 1::2] << 4)).contiguous()
    return codes, s8.view(torch.uint8).contiguous(), alpha


def _acts(g, rows, cols, std=1.0):
    """Activations: normal, with a few columns far larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device="cuda").mul_(std)
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    x[:, big] *= 8.0
    return x


def _mx_inputs(v):
    codes, scales = _to_mx(v.float())
    return codes.contiguous(), scales.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)
    c, s = case, {"case": case}
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op = c["op"]
    if op in ("norm", "norm_grad", "to_mxfp8", "from_mxfp8"):
        dt = DTYPES[c["dtype"]]
        x = _acts(g, c["rows"], c["cols"]).to(dt)
        if op == "to_mxfp8":
            return s | {"x": x}
        if op == "from_mxfp8":
            return s | {"x": _mx_inputs(x)}
        s["w"] = (1.0 + 0.1 * rand(c["cols"])).to(dt)
        if op == "norm":
            return s | {"x": x, "r": _acts(g, c["rows"], c["cols"], 2.0).to(dt) if c["residual"] else None}
        return s | {"s": _mx_inputs(x) if c["kept"] == "mxfp8" else x, "dy": rand(c["rows"], c["cols"]).to(dt),
                    "ds": rand(c["rows"], c["cols"]).to(dt) if c["ds"] else None}
    n = c["n"] * (2 if c["gated"] else 1)
    s["W"] = _make_weights(g, n, c["k"])
    if op == "linear":
        x = _acts(g, c["rows"], c["k"]).to(BF16)
        s["x"] = _mx_inputs(x) if c["x"] == "mxfp8" else x
        s["b"] = rand(n).mul_(0.5).to(BF16) if c["bias"] else None
        s["r"] = rand(c["rows"], c["n"]).to(BF16) if c["residual"] else None
    else:
        s["dy"] = rand(c["rows"], c["n"]).to(BF16)
        z = rand(c["rows"], n).mul_(1.5).to(BF16) if c["act"] != "none" else None
        s["z"] = _mx_inputs(z) if c["kept"] == "mxfp8" else z
    return s


# ----------------------------------------------------------------------------------------- plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _weights(W):
    """q * Delta in fp32 (exact), without alpha."""
    codes, scales, _ = W
    n, half = codes.shape
    table = torch.tensor(E2M1, device=codes.device)
    q = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(n, half // 8, 16)
    return (q * scales.view(torch.float8_e4m3fn).float()[..., None]).view(n, 2 * half)


def _pow2(e):
    """2^e in fp32, e from -127 to 127, from its bits (pow rounds)."""
    return torch.where(e > -127, (e.int() + 127) << 23, 1 << 22).view(F32)


def _to_mx(v):
    """fp32 rows -> E4M3 codes and E8M0 scales: the smallest power of two with max|v| <= 448 * scale."""
    rows, cols = v.shape
    nb = -(-cols // MX)
    p = torch.nn.functional.pad(v, (0, nb * MX - cols)).view(rows, nb, MX)
    m, e = torch.frexp(p.abs().amax(-1))  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m == 0, -127, e - 9 + (m > 0.875).int()).clamp(-127, 127)
    codes = (p / _pow2(e)[..., None]).to(torch.float8_e4m3fn).view(rows, nb * MX)[:, :cols]
    return codes.contiguous(), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _from_mx(t):
    """The fp32 values of MXFP8 rows, or of plain rows."""
    if isinstance(t, torch.Tensor):
        return t.float()
    codes, scales = t
    rows, cols = codes.shape
    s = _pow2(scales.view(torch.uint8).int() - 127)
    return codes.float() * s.repeat_interleave(MX, 1)[:, :cols]


def _act(z, kind):
    if kind == "none":
        return z
    return z * torch.sigmoid(z if kind == "silu" else 2 * GELU_C * (z + 0.044715 * z * z * z))


def _act_grad(z, kind):
    if kind == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    s = torch.sigmoid(2 * GELU_C * (z + 0.044715 * z * z * z))
    return s + z * s * (1 - s) * 2 * GELU_C * (1 + 3 * 0.044715 * z * z)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "to_mxfp8":
        return _to_mx(s["x"].float())
    if op == "from_mxfp8":
        return _from_mx(s["x"]).to(DTYPES[c["dtype"]])
    if op == "norm":
        h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w"].float()
        y = _to_mx(y) if c["out"] == "mxfp8" else y.to(DTYPES[c["out"]])
        return (y,) if s["r"] is None else (y, h.to(s["x"].dtype))
    if op == "norm_grad":
        h, dy, w = _from_mx(s["s"]), s["dy"].float(), s["w"].float()
        q = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
        g = dy * w
        dx = q * (g - h * (q * q * (g * h).mean(-1, keepdim=True)))
        if s["ds"] is not None:
            dx = dx + s["ds"].float()
        return dx.to(s["dy"].dtype), (dy * h * q).sum(0)
    W, alpha = _weights(s["W"]), s["W"][2]
    if op == "linear":
        z = (_from_mx(s["x"]) @ W.T) * alpha
        if s["b"] is not None:
            z = z + s["b"].float()
        a = _act(z[:, :c["n"]], c["act"]) * z[:, c["n"]:] if c["gated"] else _act(z, c["act"])
        if s["r"] is not None:
            a = a + s["r"].float()
        y = a.to(DTYPES[c["out"]])
        return (y,) if c["keep"] == "none" else (y, _to_mx(z) if c["keep"] == "mxfp8" else z.to(BF16))
    dy = s["dy"].float()
    if c["act"] == "none":
        dz = dy
    else:
        z = _from_mx(s["z"])
        if c["gated"]:
            zg, zu = z[:, :c["n"]], z[:, c["n"]:]
            dz = torch.cat((dy * zu * _act_grad(zg, c["act"]), dy * _act(zg, c["act"])), 1)
        else:
            dz = dy * _act_grad(z, c["act"])
    return ((dz @ W) * alpha).to(BF16), dz.to(BF16) if c["act"] != "none" else None, dz.sum(0) if c["bias"] else None


# --------------------------------------------------------------------------------------- the framework

def _own(s):
    import nvfp4_block_scaled_elem_amd as nv

    c = s["case"]
    op = c["op"]
    if op == "to_mxfp8":
        return nv.quantize_mxfp8(s["x"])
    if op == "from_mxfp8":
        return nv.dequantize_mxfp8(*s["x"], DTYPES[c["dtype"]])
    if op == "norm":
        out = "mxfp8" if c["out"] == "mxfp8" else DTYPES[c["out"]]
        r = nv.rms_norm(s["x"], s["w"], EPS, residual=s["r"], out_dtype=out)
        return (r,) if s["r"] is None else r
    if op == "norm_grad":
        return nv.rms_norm_grad(s["dy"], s["s"], s["w"], EPS, dS=s["ds"])
    act = None if c["act"] == "none" else c["act"]
    if op == "linear":
        keep = {"none": None, "bf16": BF16, "mxfp8": "mxfp8"}[c["keep"]]
        r = nv.linear(s["x"], *s["W"], bias=s["b"], activation=act, gated=c["gated"], residual=s["r"],
                      out_dtype=DTYPES[c["out"]], keep=keep)
        return (r,) if keep is None else r
    return nv.linear_grad(s["dy"], *s["W"], Z=s["z"], activation=act, gated=c["gated"], bias=c["bias"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work

def _mx_bytes(rows, cols):
    return rows * (cols + -(-cols // MX))


def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "norm_grad", "to_mxfp8", "from_mxfp8"):
        rows, cols, b = c["rows"], c["cols"], 2 if c["dtype"] == "bf16" else 4
        e = rows * cols
        mx = _mx_bytes(rows, cols)
        if op in ("to_mxfp8", "from_mxfp8"):
            return {"bytes": e * b + mx, "flops": 2 * e}
        if op == "norm":
            out = mx if c["out"] == "mxfp8" else e * b
            return {"bytes": e * b * (3 if c["residual"] else 1) + cols * b + out, "flops": 5 * e}
        kept = mx if c["kept"] == "mxfp8" else e * b
        return {"bytes": e * b * (3 if c["ds"] else 2) + kept + cols * (b + 4), "flops": 12 * e}
    rows, k, n = c["rows"], c["k"], c["n"] * (2 if c["gated"] else 1)
    total = n * k // 2 + n * k // 16 + 4
    if op == "linear":
        total += _mx_bytes(rows, k) if c["x"] == "mxfp8" else rows * k * 2
        total += (n * 2 if c["bias"] else 0) + (rows * c["n"] * 2 if c["residual"] else 0)
        total += rows * c["n"] * (2 if c["out"] == "bf16" else 4)
        total += {"none": 0, "bf16": rows * n * 2, "mxfp8": _mx_bytes(rows, n)}[c["keep"]]
    else:
        total += rows * c["n"] * 2 + rows * k * 2 + (n * 4 if c["bias"] else 0)
        total += {"none": 0, "bf16": rows * n * 2, "mxfp8": _mx_bytes(rows, n)}[c["kept"]]
        total += rows * n * 2 if c["act"] != "none" else 0
    return {"bytes": total, "flops": 2 * rows * n * k}


# ----------------------------------------------------------------------------------------------- exact

def _x_pow2(e):
    """2^e in binary64 for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _x_values(t):
    """MXFP8 or plain rows as binary64."""
    if not isinstance(t, (tuple, list)):
        return t.to(F64)
    rows, cols = t[0].shape
    scale = _x_pow2(t[1].view(torch.uint8).to(torch.int64) - 127)
    col = torch.arange(cols, device=t[0].device) // MX
    return t[0].to(F64) * scale[:, col]


def _x_round_mx(v):
    """The E4M3 codes (as values) and scales of binary64 rows, rounded once."""
    rows, cols = v.shape
    nb = (cols + MX - 1) // MX
    big = torch.zeros(rows, nb * MX, dtype=F64, device=v.device)
    big[:, :cols] = v.abs()
    top = big.view(rows, nb, MX).max(-1).values
    m, e = torch.frexp(top / 448.0)
    e = torch.where(m == 0.5, e - 1, e)  # top / 448 <= 2^e, the least such e
    e = torch.where(top <= 448.0 * _x_pow2(e), e, e + 1)
    scale = _x_pow2(torch.where(top > 0, e, -127).clamp(-127, 127))
    u = v / scale[:, torch.arange(cols, device=v.device) // MX]
    step = _x_pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(u / step) * step, scale


def _x_weights(W):
    codes, scales, alpha = W
    nib = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    nib[:, 0::2], nib[:, 1::2] = codes % 16, codes // 16
    e, m = (nib % 8) // 2, (nib % 2).to(F64)
    mag = torch.where(e == 0, 0.5 * m, _x_pow2(e - 1) * (1.0 + 0.5 * m))
    q = torch.where(nib >= 8, -mag, mag)
    del nib, e, m, mag
    q *= scales.view(torch.float8_e4m3fn).to(F64).repeat_interleave(16, 1)
    return q * alpha.to(F64)


def _x_act(z, kind):
    """An activation and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s + z * s * (1.0 - s)
    t = torch.tanh(GELU_C * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_C * (1.0 + 0.134145 * z * z)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "to_mxfp8":
        return _x_round_mx(s["x"].to(F64))
    if op == "from_mxfp8":
        return _x_values(s["x"])
    if op == "norm":
        h = s["x"].to(F64)
        if s["r"] is not None:
            h = h + s["r"].to(F64)
        y = s["w"].to(F64) * h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["cols"] + EPS)
        y = _x_round_mx(y) if c["out"] == "mxfp8" else y
        return (y,) if s["r"] is None else (y, h)
    if op == "norm_grad":
        h, dy, w = _x_values(s["s"]), s["dy"].to(F64), s["w"].to(F64)
        var = (h * h).sum(-1, keepdim=True) / c["cols"] + EPS
        unit = h / torch.sqrt(var)
        g = w * dy
        dx = (g - unit * (g * unit).sum(-1, keepdim=True) / c["cols"]) / torch.sqrt(var)
        if s["ds"] is not None:
            dx = dx + s["ds"].to(F64)
        return dx, (dy * unit).sum(0)
    W = _x_weights(s["W"])
    n = c["n"]
    if op == "linear":
        z = _x_values(s["x"]) @ W.t()
        if s["b"] is not None:
            z = z + s["b"].to(F64)
        y = _x_act(z[:, :n], c["act"])[0]
        if c["gated"]:
            y = y * z[:, n:]
        if s["r"] is not None:
            y = y + s["r"].to(F64)
        return (y,) if c["keep"] == "none" else (y, _x_round_mx(z) if c["keep"] == "mxfp8" else z)
    dy = s["dy"].to(F64)
    if c["act"] == "none":
        dz = dy
    else:
        z = _x_values(s["z"])
        a, da = _x_act(z[:, :n], c["act"])
        dz = torch.cat((dy * z[:, n:] * da, dy * a), 1) if c["gated"] else dy * da
    return dz @ W, dz if c["act"] != "none" else None, dz.sum(0) if c["bias"] else None
