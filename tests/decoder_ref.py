"""Plain binary64 forms of a decoder layer's operators between its products, for the tests: no library code."""
import math

import torch

from tests import layer_ref as ref

PAGE = 64
F64 = torch.float64


def rotary(x, pos, sections, base, inverse=False):
    """(y, a bound of the binary32 error): the angle's fraction of a turn is rounded to binary32 (2^-26 turns), the sine
    and cosine are within two units, the products and the sum round once each; the angle itself is off by some
    2^-53 of its size on both sides."""
    x = x.double()
    half = sum(sections)
    axis = torch.cat([torch.full((n,), i, dtype=torch.long) for i, n in enumerate(sections)]).to(x.device)
    p = pos.view(-1, x.shape[0])[axis].T.double()
    w = p * torch.pow(torch.tensor(base, dtype=F64), -torch.arange(half, dtype=F64) / half).to(x.device)
    c, s = torch.cos(w)[:, None], (-torch.sin(w) if inverse else torch.sin(w))[:, None]
    a, b = x[..., :half], x[..., half:2 * half]
    err = (a.abs() + b.abs()) * (2.0 ** -21 + w.abs()[:, None] * 2.0 ** -50)
    return (torch.cat((a * c - b * s, b * c + a * s, x[..., 2 * half:]), -1),
            torch.cat((err, err, torch.zeros_like(x[..., 2 * half:])), -1))


def to_codes(u):
    """Nearest E4M3 values, ties to even, of |u| <= 448."""
    step = ref.pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(u / step) * step


class Cache:
    """A cache in binary64: the values of the codes [pages, heads, 64, dim] of keys and values, and scale exponents."""

    def __init__(self, cache):
        k, v, ks, vs = cache
        self.codes = [k.view(torch.float8_e4m3fn).double(), v.view(torch.float8_e4m3fn).double().transpose(2, 3).contiguous()]
        self.byte = [t.view(torch.uint8).long() for t in (ks, vs)]

    def append(self, kv, table, spans):
        """kv: K and V [tokens, heads, dim]; spans: (first row, new tokens, length) of each sequence."""
        for which, x in enumerate(kv):
            codes, byte = self.codes[which], self.byte[which]
            for s, (first, n, length) in enumerate(spans):
                for pos in range(max(length - n, 0), length):
                    if pos % PAGE and pos != max(length - n, 0):
                        continue
                    lo, hi = pos % PAGE, min(PAGE, length - pos + pos % PAGE)
                    page = int(table[s, pos // PAGE])
                    if not 0 <= page < codes.shape[0]:
                        continue
                    row = first + n - (length - pos)
                    rows = x[row:row + hi - lo].double().transpose(0, 1)
                    top = rows.abs().amax((1, 2))
                    need = torch.where(torch.isfinite(top), ref.mx_scale_exp(torch.nan_to_num(top, 1, 1, 1)) + 127, 255)
                    if lo:
                        need = torch.maximum(need, byte[page])
                        down = ref.pow2((byte[page] - need).clamp_min(-300))[:, None, None]
                        codes[page, :, :lo] = to_codes(codes[page, :, :lo] * down)
                    scale = ref.pow2(127 - need)[:, None, None]
                    codes[page, :, lo:hi] = to_codes(torch.nan_to_num(rows, 0, 0, 0) * scale)
                    bad = need == 255
                    codes[page, :, :hi][bad] = math.nan
                    byte[page] = need


def attention(q, cache, table, spans, scale, causal):
    """(o, a bound of its error) of the rows in spans; rows of no sequence are NaN. Binary32 scores are off by dim 2^-23
    of sum |q k| and by 2^-22 of themselves, which is the relative error of a probability; a probability is rounded to
    bf16 (2^-8) before the second product, whose sums are binary32."""
    k, v, ks, vs = cache
    heads, kv_heads, dim = q.shape[1], k.shape[1], q.shape[2]
    out = torch.full(q.shape, math.nan, dtype=F64, device=q.device)
    err = torch.zeros_like(out)
    value = [t.view(torch.float8_e4m3fn).double() for t in (k, v)]
    exps = [torch.where(b == 255, math.nan, ref.pow2(b - 127)) for b in (t.view(torch.uint8).long() for t in (ks, vs))]
    for s, (first, n, length) in enumerate(spans):
        if n == 0:
            continue
        if length == 0:
            out[first:first + n] = 0.0
            continue
        pages = table[s, :-(-length // PAGE)].long()
        there = ((pages >= 0) & (pages < k.shape[0])).repeat_interleave(PAGE)[:length]
        pages = pages.clamp(0, k.shape[0] - 1)
        K = (value[0][pages] * exps[0][pages][:, :, None, None]).permute(1, 0, 2, 3).flatten(1, 2)[:, :length]
        V = (value[1][pages] * exps[1][pages][:, :, None, None]).permute(1, 0, 3, 2).flatten(1, 2)[:, :length]
        nan = (torch.isnan(exps[0]) | torch.isnan(exps[1]))[pages].T.repeat_interleave(PAGE, 1)[:, :length]  # [kv_heads, length]
        at = torch.arange(length, device=q.device)
        for h in range(heads):
            g = h * kv_heads // heads
            x = q[first:first + n, h].double()
            last = length - n + 1 + torch.arange(n, device=q.device) if causal else torch.full((n,), length, device=q.device)
            seen = (at[None] < last[:, None]) & there
            score = torch.nan_to_num(x @ K[g].T, 0, 0, 0) * scale
            mag = torch.nan_to_num(x.abs() @ K[g].abs().T, 0, 0, 0) * abs(scale)
            score = score.masked_fill(~seen, -math.inf)
            none = ~seen.any(1)
            p = torch.softmax(score.masked_fill(none[:, None], 0.0), -1) * ~none[:, None]
            Vg = torch.nan_to_num(V[g], 0, 0, 0)
            o = p @ Vg
            spread = p @ Vg.abs()
            es = (mag * seen).amax(1) * (dim * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -20
            e = spread * (2.0 ** -8 + 2 * es[:, None] + (length + 64) * 2.0 ** -23)
            o[(seen & nan[g]).any(1)] = math.nan
            out[first:first + n, h], err[first:first + n, h] = o, e
    return out, err


# ------------------------------------------------------------------------------------------- experts

def route(logits, top_k, sigmoid, normalize):
    """(chosen [tokens, experts] bool, weights, their relative error): the binary32 exponential of a difference d of
    logits is off by |d| 2^-23 (d and d log2(e) rounded) and a few units; sums of up to 512 terms in six steps."""
    l = logits.double()
    T, E = l.shape
    lower = torch.arange(E, device=l.device)
    before = ((l[:, None, :] > l[:, :, None]) | ((l[:, None, :] == l[:, :, None]) & (lower[None, :] < lower[:, None]))).sum(-1)
    chosen = (before < top_k) & (l > -math.inf)
    p = torch.sigmoid(l) if sigmoid else torch.softmax(l.masked_fill(~(l > -math.inf).any(1)[:, None], 0.0), -1)
    if normalize:
        e = torch.where(chosen, p, 0.0)
        p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    top = l.amax(1, keepdim=True).clamp_min(-1e30)
    err = 2.0 ** -19 + 2.0 ** -21 * torch.nan_to_num((top - l).abs() + l.abs(), 0, 0, 0)
    return chosen, torch.where(chosen, p, 0.0), err


def moe(x, logits, up, down, top_k, act, gated, sigmoid, normalize, res=None):
    """(y, a bound of the error before y's own rounding): the first product and its activation as in layer_ref.linear,
    a half step of bf16 on h, the second product's sums, the weights."""
    chosen, w, ew = route(logits, top_k, sigmoid, normalize)
    y = torch.zeros(x.shape, dtype=F64, device=x.device) if res is None else res.double()
    err = ref.U * y.abs()
    total = torch.zeros_like(y)
    for e in range(logits.shape[1]):
        mine = chosen[:, e].nonzero()[:, 0]
        if len(mine) == 0:
            continue
        h, _, eh, _ = ref.linear(x[mine].double(), up[0][e], up[1][e], up[2][e], act=act, gated=gated)
        eh = eh + (h.abs() + eh) * ref.HALF[torch.bfloat16]
        W, alpha = ref.weights(down[0][e], down[1][e]), float(down[2][e])
        o = alpha * (h @ W.T)
        eo = alpha * (eh @ W.abs().T) + ref.product_error(h.abs() + eh, W, alpha, h.shape[1])
        share = w[mine, e, None]
        y[mine] += share * o
        total[mine] += (share * o).abs()
        err[mine] += share * (eo + (ew[mine, e, None] + 4 * ref.U) * (o.abs() + eo))
    return y, err + (top_k + 1) * ref.U * total
