"""Plain binary64 forms of the layer operators, for the tests: no library code, one formula per line."""
import math

import torch

GELU_C = math.sqrt(2.0 / math.pi)
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value
U = 2.0 ** -24  # one binary32 rounding


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
