"""Plain binary64 forms of the layer operators, for the tests: no library code, one formula per line."""
import math

import torch

GELU_C = math.sqrt(2.0 / math.pi)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value
U = 2.0 ** -24  # one binary32 rounding
# Binary32's smallest normal number: the hardware reciprocal gives 0 for results below it, so a logistic
# function below 2^-126 (arguments under -87) may read as 0, and what is formed from it is off by 2^-126 times
# its factor, however small the exact value is.
TINY = 2.0 ** -126


def pow2(e):
    """2^e in binary64 for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def mx_scale_exp(amax):
    """The exponent of the smallest power of two, 2^-127 at least, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax.double())  # amax = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def mx_blocks(v, fill=0.0):
    rows, cols = v.shape
    nb = -(-cols // 32)
    out = torch.full((rows, nb * 32), fill, dtype=v.dtype, device=v.device)
    out[:, :cols] = v
    return out.view(rows, nb, 32)


def mx_quantize(v):
    """(codes' values, scale bytes) of finite binary64 rows, each value rounded once, ties to even."""
    b = mx_blocks(v.double())
    e = mx_scale_exp(b.abs().amax(-1))
    u = b / pow2(e)[..., None]
    step = pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)
    q = torch.round(u / step) * step
    return q.view(v.shape[0], -1)[:, :v.shape[1]], (e + 127).to(torch.uint8)


def mx_values(codes, scales):
    """The binary64 values of an MXFP8 pair."""
    b = scales.view(torch.uint8).to(torch.int64)
    s = torch.where(b == 255, torch.full(b.shape, float("nan"), dtype=torch.float64, device=b.device), pow2(b - 127))
    return codes.view(torch.float8_e4m3fn).double() * s.repeat_interleave(32, 1)[:, :codes.shape[1]]


def value(t):
    return mx_values(*t) if isinstance(t, tuple) else t.double()


def rms_norm(x, w, eps, r=None):
    h = x.double() + (0 if r is None else r.double())
    q = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    return h * q * w.double(), h


def norm_depth(cols):
    """Additions on the longest path of a row's sum: a thread's own, a wave's six, the waves' sixteen."""
    return max(64, 8 * -(-cols // 8192)) + 22


def rms_norm_grad(dy, h, w, eps, dh=None):
    """(dx, dweight, a bound of the binary32 error of each)."""
    dy, h, w = dy.double(), h.double(), w.double()
    rows, cols = h.shape
    q = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = dy * w
    c = q * q * (g * h).mean(-1, keepdim=True)
    d = torch.zeros_like(h) if dh is None else dh.double()
    dx = q * (g - h * c) + d
    depth = norm_depth(cols)
    spread = q * q * (g * h).abs().mean(-1, keepdim=True)
    ex = U * ((depth + 10) * (q * g.abs() + q * h.abs() * (c.abs() + spread)) + 2 * d.abs())
    ew = U * (depth + 10 + rows) * (dy * h * q).abs().sum(0)
    return dx, (dy * h * q).sum(0), ex, ew


# ------------------------------------------------------------------------------------------- products

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def weights(codes, scales):
    """q * Delta of NVFP4 weights, binary64, without alpha."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    n = codes.shape[0]
    q = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).view(n, -1)
    return q * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def logistic_arg(z, act):
    return z if act == "silu" else 2 * GELU_C * (z + 0.044715 * z ** 3)


def act_value(z, act):
    return z if act is None else z * torch.sigmoid(logistic_arg(z, act))


def act_slope(z, act):
    if act is None:
        return torch.ones_like(z)
    s = torch.sigmoid(logistic_arg(z, act))
    dv = 1.0 if act == "silu" else 2 * GELU_C * (1 + 3 * 0.044715 * z * z)
    return s + z * s * (1 - s) * dv


def act_error(z, act):
    """Binary32 error of act(z) for a given z: e^-v is off by |v| 2^-24 (v rounded) and a few units, and so is
    the logistic function; a dozen roundings in all."""
    if act is None:
        return torch.zeros_like(z)
    return U * (12 + 2 * logistic_arg(z, act).abs()) * act_value(z, act).abs() + TINY * z.abs()


def act_slope_error(z, act):
    """The same for act'(z): sums of terms up to (1 + |z|) dv, each with the logistic function's error."""
    if act is None:
        return torch.zeros_like(z)
    v = logistic_arg(z, act)
    dv = 1.0 if act == "silu" else 2 * GELU_C * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(v)
    return U * (16 + 4 * v.abs()) * (s + s * (1 - s) * z.abs() * dv) + TINY * (1 + z.abs() * dv)


def product_error(x, W, alpha, length):
    """fp32 sums of `length` exact products in any order, the factor and one rounding more."""
    return (length * 2.0 ** -23 + 2.0 ** -22) * alpha * (x.abs() @ W.abs().T)


def linear(x, codes, scales, alpha, bias=None, act=None, gated=False, res=None):
    """(y, z, a bound of the binary32 error of each) of values x (binary64)."""
    W, alpha = weights(codes, scales), float(alpha)
    z, ez = alpha * (x @ W.T), product_error(x, W, alpha, x.shape[1])
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * z.abs()
    F = z.shape[1] // 2 if gated else z.shape[1]
    g, eg = z[:, :F], ez[:, :F]
    y = act_value(g, act)
    ey = 1.13 * eg + act_error(g, act)  # |act'| <= 1.13
    if gated:
        u, eu = z[:, F:], ez[:, F:]
        ey = ey * (u.abs() + eu) + y.abs() * eu + U * (y * u).abs()
        y = y * u
    if res is not None:
        y = y + res.double()
        ey = ey + U * y.abs()
    return y, z, ey, ez


def linear_dz(dy, z, act, gated):
    """(dz, a bound of its binary32 error) for given z."""
    if act is None:
        return dy, torch.zeros_like(dy)
    if not gated:
        return dy * act_slope(z, act), dy.abs() * (act_slope_error(z, act) + U * act_slope(z, act).abs())
    F = z.shape[1] // 2
    g, u = z[:, :F], z[:, F:]
    s, es = act_slope(g, act), act_slope_error(g, act)
    a, ea = act_value(g, act), act_error(g, act)
    return (torch.cat((dy * u * s, dy * a), 1),
            torch.cat(((dy * u).abs() * (es + 2 * U * s.abs()), dy.abs() * (ea + U * a.abs())), 1))
