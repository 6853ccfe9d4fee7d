"""The operators of a decoder layer that stand between and beside its products, as measured cases.

Operators: rotary positions of one or several axes; a paged cache of keys and values in 8 bits, written
(`kv_append`) and attended to (`attention`: one token of each sequence, or whole prompts); and a layer of
experts with NVFP4 weights for a few tokens (`moe`).

``run`` computes a case in elementary torch operations, or, where ``own`` is set, by the framework's calls.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DTYPES = {"bf16": BF16, "fp32": F32}
BASE = 10000.0
BLOCK = 64  # tokens of a cache's block: one scale per block and head


# ---------------------------------------------------------------------------------------------- cases

def _rotary(name, tokens, heads, dim, axes=1, rotated=None, dtype="bf16"):
    return dict(name=name, op="rotary", tokens=tokens, heads=heads, dim=dim, axes=axes, rotated=rotated or dim, dtype=dtype)


def _append(name, seqs, kv_heads, dim, most, old_lo, old_hi, dtype="bf16"):
    """`most`: new tokens of a sequence, from most // 2 (at least 1) up; old_lo .. old_hi: tokens it has already."""
    return dict(name=name, op="append", seqs=seqs, kv_heads=kv_heads, dim=dim, most=most, old_lo=old_lo, old_hi=old_hi,
                dtype=dtype)


def _attention(name, seqs, heads, kv_heads, dim, most, old_lo, old_hi, causal=True):
    return dict(name=name, op="attention", seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, most=most, old_lo=old_lo,
                old_hi=old_hi, causal=causal)


def _moe(name, tokens, experts, top_k, width, inner, act="silu", gated=True, scoring="softmax", normalize=True,
         residual=False, logits="fp32"):
    return dict(name=name, op="moe", tokens=tokens, experts=experts, top_k=top_k, width=width, inner=inner, act=act,
                gated=gated, scoring=scoring, normalize=normalize, residual=residual, logits=logits)


def listed():
    return [
        # one token of a decoding step: the positions of its query and key heads
        _rotary("rotary: one token", 1, 40, 128),
        # a prompt with images: three axes (time, height, width)
        _rotary("rotary: images", 8191, 40, 128, axes=3),
        # a decoding step of a batch: a token of each sequence goes into the cache
        _append("cache: a token each", 64, 8, 128, 1, 100, 8000),
        # prompts of odd lengths, some after earlier turns, go into the cache
        _append("cache: prompts", 5, 8, 128, 3001, 0, 700),
        # a decoding step of one user's long conversation
        _attention("attention: one sequence", 1, 32, 8, 128, 1, 7999, 7999),
        # a decoding step of a batch of conversations of very different lengths
        _attention("attention: batch", 64, 32, 8, 128, 1, 300, 16000),
        # a few drafted tokens of each sequence are verified: seven query heads to a key head of 64
        _attention("attention: drafts", 16, 28, 4, 64, 6, 500, 5000),
        # prompts of odd lengths, one after an earlier turn
        _attention("attention: prompts", 2, 32, 8, 128, 5003, 0, 3333),
        # a token through a layer of many small experts
        _moe("experts: one token", 1, 128, 8, 2048, 768),
        # a small decoding batch through the same kind of layer, the experts' sum added to the residual stream
        _moe("experts: small batch", 8, 64, 6, 4096, 1408, scoring="sigmoid", residual=True),
        # a short batch through a layer of few wide experts
        _moe("experts: wide", 33, 8, 2, 4096, 14336),
        # a larger decoding batch
        _moe("experts: batch", 150, 128, 8, 2048, 768, act="gelu", normalize=False, logits="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_BYTES, MOST_FLOPS = 5.0e8, 3.0e11


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "moe", "moe"])
    if op == "rotary":
        axes = rng.choice([1, 1, 3])
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.randint(1, 64)
        tokens = min(_log(rng, 1, 16384), (1 << 26) // (heads * dim))
        c = _rotary("", tokens, heads, dim, axes, rng.choice([dim, dim, dim // 2]), rng.choice(["bf16", "bf16", "fp32"]))
    elif op == "append":
        seqs, kv_heads, dim = _log(rng, 1, 256), rng.randint(1, 16), rng.choice([64, 80, 96, 128, 256])
        most = rng.choice([1, 1, _log(rng, 2, 4096)])
        most = max(1, min(most, (1 << 23) // (seqs * kv_heads * dim)))
        c = _append("", seqs, kv_heads, dim, most, rng.randint(0, 200), rng.randint(200, 2000), rng.choice(["bf16", "bf16", "fp32"]))
    elif op == "attention":
        kv_heads, dim = rng.randint(1, 12), rng.choice([64, 80, 96, 128, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 12])
        most = rng.choice([1, 1, 1, rng.randint(2, 16), _log(rng, 16, 4096)])
        hi = _log(rng, 64, 32768)
        seqs = _log(rng, 1, 128)
        seqs = max(1, min(seqs, int(MOST_BYTES / (2 * hi * kv_heads * dim)),
                          int(MOST_FLOPS / (4.0 * most * (hi + most) * heads * dim))))
        while 4.0 * most * (hi + most) * heads * dim > MOST_FLOPS:
            most //= 2
        c = _attention("", seqs, heads, kv_heads, dim, most, max(1, hi // rng.randint(1, 40)), hi, rng.random() < 0.85)
    else:
        experts = rng.choice([8, 16, 60, 64, 128, 256])
        top_k = rng.randint(1, 8)
        width, inner = 16 * _log(rng, 16, 384), 16 * _log(rng, 8, 256)
        gated = rng.random() < 0.8
        while 0.5625 * experts * width * inner * (3 if gated else 2) > MOST_BYTES:
            inner = inner // 32 * 16
        c = _moe("", _log(rng, 1, 256), experts, top_k, width, max(16, inner), rng.choice(["silu", "gelu"]), gated,
                 rng.choice(["softmax", "sigmoid"]), rng.random() < 0.7, rng.random() < 0.4, rng.choice(["bf16", "fp32"]))
    del c["name"]
    return c


def _spread(n, lo, hi, start):
    """n whole numbers spread over lo .. hi by their logarithm, in no order."""
    a, b = math.log(max(lo, 0.5)), math.log(max(hi, 0.5))
    return [min(hi, max(lo, int(round(math.exp(a + (b - a) * ((start + 0.6180339887 * i) % 1.0)))))) for i in range(n)]


def _lengths(c):
    """(tokens that each sequence has before, new ones) of an append or attention case."""
    old = _spread(c["seqs"], c["old_lo"], c["old_hi"], 0.98)
    new = [1] * c["seqs"] if c["most"] == 1 else _spread(c["seqs"], max(1, c["most"] // 2), c["most"], 0.99)
    return old, new


def _sections(c):
    pairs = c["rotated"] // 2
    return [pairs] if c["axes"] == 1 else [pairs - 2 * (3 * pairs // 8), 3 * pairs // 8, 3 * pairs // 8]


# --------------------------------------------------------------------------------------------- inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, lengths):
    """A table of shuffled pages for sequences of these lengths, and the number of pages."""
    need = [-(-n // BLOCK) for n in lengths]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(need + [1]), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages


def _filled(g, pages, kv_heads, dim):
    """A cache whose every block is filled: keys with a few far larger channels, values; blocks of 64 tokens."""
    k = torch.empty(pages, kv_heads, BLOCK, dim, dtype=E4M3, device="cuda")
    v = torch.empty(pages, kv_heads, dim, BLOCK, dtype=E4M3, device="cuda")
    ks = torch.empty(pages, kv_heads, dtype=E8M0, device="cuda")
    vs = torch.empty(pages, kv_heads, dtype=E8M0, device="cuda")
    big = 1.0 + 3.0 * (torch.rand(kv_heads, 1, dim, generator=g, device="cuda") < 0.05)
    step = max(1, (1 << 25) // (kv_heads * BLOCK * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, kv_heads, BLOCK, dim, generator=g, device="cuda") * big
        e = _scale_exp(x.abs().amax((-1, -2)))
        k[p:p + n] = (x / _pow2(e)[..., None, None]).to(E4M3)
        ks[p:p + n] = (e + 127).to(torch.uint8).view(E8M0)
        x = torch.randn(n, kv_heads, dim, BLOCK, generator=g, device="cuda")
        e = _scale_exp(x.abs().amax((-1, -2)))
        v[p:p + n] = (x / _pow2(e)[..., None, None]).to(E4M3)
        vs[p:p + n] = (e + 127).to(torch.uint8).view(E8M0)
    return k, v, ks, vs


def _make_experts(g, experts, n, k):
    """NVFP4 codes, E4M3 scales and alphas of random [n, k] matrices by the max rule."""
    codes = torch.empty(experts, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, n, k // 16, dtype=torch.uint8, device="cuda")
    alphas = torch.empty(experts, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    for i in range(experts):
        w = torch.randn(n, k // 16, 16, generator=g, device="cuda").mul_(k ** -0.5)
        amax = w.abs().amax(-1)
        alpha = amax.max() / 2688.0
        s8 = (amax / (6.0 * alpha)).clamp_(max=448.0).to(E4M3)
        x = w.div_((s8.float() * alpha).clamp_min_(1e-30)[..., None]).view(n, k)
        q = torch.bucketize(x.abs(), edges, out_int32=True)
        q += ((x < 0) & (q > 0)) * 8
        codes[i] = (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8)
        scales[i], alphas[i] = s8.view(torch.uint8), alpha
    return codes, scales, alphas


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    c, s = case, {"case": case}
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    whole = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")  # noqa: E731
    if c["op"] == "rotary":
        t = c["tokens"]
        # the query and key heads of a product whose output holds value heads too
        s["x"] = rand(t, c["heads"] + 8, c["dim"]).to(DTYPES[c["dtype"]])[:, :c["heads"]]
        first = whole(0, 100000, 1)
        if c["axes"] == 1:
            s["pos"] = first + torch.arange(t, device="cuda")
        else:  # frames of 64 x 64 patches
            i = torch.arange(t, device="cuda")
            s["pos"] = first + torch.stack((i // 4096, i // 64 % 64, i % 64))
        return s
    if c["op"] == "moe":
        t, e = c["tokens"], c["experts"]
        x = rand(t, c["width"])
        x[:, whole(0, c["width"], max(1, c["width"] // 512))] *= 8.0
        s["x"] = x.to(BF16)
        s["logits"] = rand(t, e).mul_(1.5).to(DTYPES[c["logits"]])
        s["up"] = _make_experts(g, e, c["inner"] * (2 if c["gated"] else 1), c["width"])
        s["down"] = _make_experts(g, e, c["width"], c["inner"])
        s["r"] = rand(t, c["width"]).to(BF16) if c["residual"] else None
        return s
    old, new = _lengths(c)
    total = [a + b for a, b in zip(old, new)]
    tokens = sum(new)
    s["table"], pages = _table(g, total)
    s["lengths"] = _ints(total)
    s["starts"] = None if c["most"] == 1 else _ints([sum(new[:i]) for i in range(len(new) + 1)])
    s["cache"] = _filled(g, pages, c["kv_heads"], c["dim"])
    if c["op"] == "append":
        dt = DTYPES[c["dtype"]]
        qkv = rand(tokens, 6 * c["kv_heads"], c["dim"]).to(dt)  # one buffer, as a product leaves it
        s["k"], s["v"] = qkv[:, 4 * c["kv_heads"]:5 * c["kv_heads"]], qkv[:, 5 * c["kv_heads"]:]
    else:
        s["q"] = rand(tokens, c["heads"], c["dim"]).mul_(1.5).to(BF16)
    return s


# ----------------------------------------------------------------------------------------- plain forms

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
GELU_C = math.sqrt(2.0 / math.pi)


def _pow2(e):
    """2^e in fp32, e from -127 to 127, from its bits."""
    return torch.where(e > -127, (e.int() + 127) << 23, 1 << 22).view(F32)


def _scale_exp(amax):
    """The exponent of the smallest power of two, 2^-127 at least, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.where(m == 0, -127, e - 9 + (m > 0.875).int()).clamp(-127, 127)


def _scale_of(scales):
    return _pow2(scales.view(torch.uint8).int() - 127)


def _plain_rotary(s):
    c, x = s["case"], s["x"]
    r, half = c["rotated"], c["rotated"] // 2
    axis = torch.arange(c["axes"], device=x.device).repeat_interleave(torch.tensor(_sections(c), device=x.device), output_size=half)
    pos = s["pos"].view(c["axes"], -1)[axis].T.double()  # [tokens, half]
    angle = pos * torch.exp(torch.arange(half, device=x.device, dtype=F64) * (-2.0 * math.log(BASE) / r))
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:r].float()
    return torch.cat(((a * cos - b * sin).to(x.dtype), (b * cos + a * sin).to(x.dtype), x[..., r:]), -1)


def _owner(s, tokens):
    """For each token: its sequence, and its place among the sequence's new tokens counted from the end (0: the last)."""
    at = torch.arange(tokens, device="cuda")
    if s["starts"] is None:
        return at, torch.zeros_like(at)
    seq = torch.searchsorted(s["starts"][1:].long(), at, right=True)
    return seq, s["starts"].long()[seq + 1] - 1 - at


def _plain_append_one(x, codes, scales, page, place, first_page, first_place, turned):
    """Keys or values x [tokens, heads, dim] into codes [pages, heads, 64, dim] (turned: [.., dim, 64])."""
    # Slots of a block behind its sequence's end are left as they are.
    x = x.float()
    heads = x.shape[1]
    amax = torch.zeros(codes.shape[0], heads, device=x.device).index_reduce_(0, page, x.abs().amax(-1), "amax")
    need = _scale_exp(amax)
    # the block that a sequence's first new token goes into may hold earlier tokens; all others start empty
    older = first_place > 0
    had = scales.view(torch.uint8)[first_page].int() - 127
    first = torch.where(older[:, None], torch.maximum(had, need[first_page]), need[first_page])
    need[first_page] = first
    block = codes[first_page]
    moved = ((block.float() * _pow2(had)[..., None, None]) / _pow2(first)[..., None, None]).to(E4M3).view(torch.uint8)
    earlier = (torch.arange(BLOCK, device=x.device) < first_place[:, None])[:, None]
    earlier = earlier[..., None, :] if turned else earlier[..., None]
    codes.view(torch.uint8)[first_page] = torch.where(earlier, moved, block.view(torch.uint8))
    scales.view(torch.uint8)[page] = (need[page] + 127).to(torch.uint8)
    code = (x / _pow2(need[page])[..., None]).to(E4M3).view(torch.uint8)
    head = torch.arange(heads, device=x.device)
    if turned:
        codes.view(torch.uint8)[page[:, None], head, :, place[:, None]] = code
    else:
        codes.view(torch.uint8)[page[:, None], head, place[:, None]] = code


def _plain_append(s):
    tokens, seqs = s["k"].shape[0], s["table"].shape[0]
    seq, behind = _owner(s, tokens)
    pos = s["lengths"].long()[seq] - 1 - behind
    page, place = s["table"].long()[seq, pos // BLOCK], pos % BLOCK
    first = torch.arange(seqs, device="cuda") if s["starts"] is None else s["starts"][:-1].long()
    k, v, ks, vs = s["cache"]
    _plain_append_one(s["k"], k, ks, page, place, page[first], place[first], False)
    _plain_append_one(s["v"], v, vs, page, place, page[first], place[first], True)
    return k, v, ks, vs


def _plain_attention(s):
    c, q = s["case"], s["q"]
    k, v, ks, vs = s["cache"]
    seqs, width = s["table"].shape
    group, n, length = c["heads"] // c["kv_heads"], c["most"], width * BLOCK
    pages = s["table"].long()
    # [seqs, kv_heads, tokens, dim]
    keys = (k[pages].float() * _scale_of(ks[pages])[..., None, None]).transpose(1, 2).reshape(seqs, c["kv_heads"], length, c["dim"])
    values = (v[pages].float() * _scale_of(vs[pages])[..., None, None]).transpose(3, 4).transpose(1, 2).reshape(keys.shape)
    seq, behind = _owner(s, q.shape[0])
    place = n - 1 - behind  # queries end at the same place of a padded row
    padded = torch.zeros(seqs, n, c["heads"], c["dim"], device=q.device)
    padded[seq, place] = q.float()
    rows = padded.view(seqs, n, c["kv_heads"], group, c["dim"]).permute(0, 2, 3, 1, 4).reshape(seqs, c["kv_heads"], group * n, c["dim"])
    score = (rows @ keys.transpose(2, 3)) * c["dim"] ** -0.5
    at = torch.arange(length, device=q.device)
    last = s["lengths"][:, None] - (torch.arange(n - 1, -1, -1, device=q.device) if c["causal"] else 0)  # tokens that a query sees
    seen = at < last[:, :, None] if c["causal"] else (at < last[:, :, None]).expand(seqs, n, length)
    score = score.view(seqs, c["kv_heads"], group, n, length).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp_min(-3e38))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-38)
    o = (p.view(seqs, c["kv_heads"], group * n, length) @ values).view(seqs, c["kv_heads"], group, n, c["dim"])
    return o.permute(0, 3, 1, 2, 4).reshape(seqs, n, c["heads"], c["dim"])[seq, place].to(BF16)


def _expert_values(W, which=None):
    """fp32 weights (with alpha) of all experts, or of those asked for."""
    codes, scales, alphas = W if which is None else (t[which] for t in W)
    table = torch.tensor(E2M1, device=codes.device)
    q = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(*scales.shape, 16)
    return (q * (scales.view(E4M3).float())[..., None]).flatten(-2) * alphas[:, None, None]


def _act(z, kind):
    return z * torch.sigmoid(z if kind == "silu" else 2 * GELU_C * (z + 0.044715 * z * z * z))


def _plain_moe(s):
    c, x, n = s["case"], s["x"].float(), s["case"]["inner"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    l = s["logits"].float()
    p = torch.softmax(l, -1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    ids = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    w = w / w.sum(-1, keepdim=True) if c["normalize"] else w
    mid = lambda z: _act(z[..., :n], c["act"]) * z[..., n:] if c["gated"] else _act(z, c["act"])  # noqa: E731
    if t * k <= e:  # the chosen experts of each token
        which = ids.reshape(-1)
        z = (_expert_values(s["up"], which) @ x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        o = (_expert_values(s["down"], which) @ mid(z)[:, :, None])[..., 0]
        y = (o.view(t, k, -1) * w[:, :, None]).sum(1)
    else:  # every expert over every token
        share = torch.zeros(t, e, device=x.device).scatter_(1, ids, w)
        z = x @ _expert_values(s["up"]).transpose(1, 2)
        o = mid(z) @ _expert_values(s["down"]).transpose(1, 2)
        y = (o * share.T[:, :, None]).sum(0)
    return (y if s["r"] is None else y + s["r"].float()).to(BF16)


PLAIN = {"rotary": _plain_rotary, "append": _plain_append, "attention": _plain_attention, "moe": _plain_moe}


# --------------------------------------------------------------------------------------- the framework

def _own(s):
    import nvfp4_block_scaled_elem_amd as nv

    c = s["case"]
    if c["op"] == "rotary":
        return nv.rotary(s["x"], s["pos"], sections=_sections(c), base=BASE)
    if c["op"] == "append":
        return tuple(nv.kv_append(s["cache"], s["k"], s["v"], s["table"], s["lengths"], s["starts"]))
    if c["op"] == "attention":
        return nv.attention(s["q"], s["cache"], s["table"], s["lengths"], s["starts"], causal=c["causal"])
    return nv.moe(s["x"], s["logits"], s["up"], s["down"], c["top_k"], activation=c["act"], gated=c["gated"],
                  scoring=c["scoring"], normalize=c["normalize"], residual=s["r"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "rotary":
        e, b = c["tokens"] * c["heads"] * c["dim"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2 * e * b + 8 * c["axes"] * c["tokens"], "flops": 3 * e}
    if c["op"] == "moe":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        per = c["width"] * c["inner"] * (3 if c["gated"] else 2)
        used = e * (1.0 - (1.0 - k / e) ** t)  # experts that some token takes
        io = t * c["width"] * 2 * (3 if c["residual"] else 2) + t * e * (2 if c["logits"] == "bf16" else 4)
        return {"bytes": int(used * (per * 0.5625 + 8)) + io, "flops": 2 * t * k * per}
    old, new = _lengths(c)
    tokens, seqs = sum(new), len(new)
    if c["op"] == "append":
        e = tokens * c["kv_heads"] * c["dim"] * 2
        blocks = sum((a + b - 1) // BLOCK - a // BLOCK + 1 for a, b in zip(old, new))
        return {"bytes": e * ((2 if c["dtype"] == "bf16" else 4) + 1) + blocks * (4 + 2 * c["kv_heads"]) + 8 * seqs,
                "flops": 2 * e}
    cached = sum(a + b for a, b in zip(old, new))
    if c["causal"]:
        seen = sum(b * a + b * (b + 1) // 2 for a, b in zip(old, new))
    else:
        seen = sum(b * (a + b) for a, b in zip(old, new))
    blocks = sum(-(-(a + b) // BLOCK) for a, b in zip(old, new))
    return {"bytes": cached * c["kv_heads"] * c["dim"] * 2 + blocks * (4 + 2 * c["kv_heads"]) + 8 * seqs
            + tokens * c["heads"] * c["dim"] * 4, "flops": 4 * seen * c["heads"] * c["dim"]}


# ----------------------------------------------------------------------------------------------- exact

def _x_pow2(e):
    """2^e in binary64 for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _x_cache_rows(s, i, length):
    """Keys and values [length, kv_heads, dim] of sequence i, in binary64."""
    k, v, ks, vs = s["cache"]
    pages = s["table"][i, :-(-length // BLOCK)].long()
    x = k[pages].to(F64) * _x_pow2(ks.view(torch.uint8)[pages].long() - 127)[:, :, None, None]
    y = v[pages].to(F64) * _x_pow2(vs.view(torch.uint8)[pages].long() - 127)[:, :, None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:length], y.permute(0, 3, 1, 2).flatten(0, 1)[:length]


def _x_least_scale(top):
    """The least power of two, 2^-127 at least, that keeps `top` within 448 of it (binary64, by its exponent)."""
    e = torch.floor(torch.log2(top.clamp_min(1e-300) / 448.0))
    e = torch.where(top <= 448.0 * _x_pow2(e - 1), e - 1, torch.where(top <= 448.0 * _x_pow2(e), e, e + 1))
    return torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(-127, 127)


def _x_to_codes(u):
    """Values in steps of E4M3, ties to even."""
    step = _x_pow2(torch.frexp(u.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(u / step) * step


def _x_append(c, s):
    old, new = _lengths(c)
    out = []
    for x, codes, scales, turned in ((s["k"], s["cache"][0], s["cache"][2], False), (s["v"], s["cache"][1], s["cache"][3], True)):
        codes, byte = codes.to(F64), scales.view(torch.uint8).to(torch.int64)
        if turned:
            codes = codes.transpose(2, 3)
        codes, at = codes.contiguous(), 0
        for i, (a, b) in enumerate(zip(old, new)):
            pos = a
            while pos < a + b:
                place, n = pos % BLOCK, min(BLOCK - pos % BLOCK, a + b - pos)
                page = int(s["table"][i, pos // BLOCK])
                rows = x[at:at + n].to(F64).transpose(0, 1)  # [heads, n, dim]
                e = _x_least_scale(rows.abs().amax((1, 2)))
                if place:
                    e = torch.maximum(e, (byte[page] - 127).to(F64))
                    codes[page, :, :place] = _x_to_codes(codes[page, :, :place] * _x_pow2(byte[page] - 127 - e.long())[:, None, None])
                codes[page, :, place:place + n] = _x_to_codes(rows * _x_pow2(-e.long())[:, None, None])
                byte[page] = e.long() + 127
                pos, at = pos + n, at + n
        out.append((codes.transpose(2, 3) if turned else codes, _x_pow2(byte - 127)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        x, half = s["x"].to(F64), c["rotated"] // 2
        y = x.clone()
        pos = s["pos"].view(c["axes"], -1).to(F64)
        j = 0
        for a, n in enumerate(_sections(c)):
            for _ in range(n):
                turn = pos[a] / BASE ** (2.0 * j / c["rotated"])
                z = torch.complex(x[..., j], x[..., half + j]) * torch.polar(torch.ones_like(turn), turn)[:, None]
                y[..., j], y[..., half + j] = z.real, z.imag
                j += 1
        return y
    if c["op"] == "append":
        return _x_append(c, s)
    if c["op"] == "attention":
        old, new = _lengths(c)
        group, at, out = c["heads"] // c["kv_heads"], 0, []
        for i, (a, b) in enumerate(zip(old, new)):
            k, v = _x_cache_rows(s, i, a + b)
            q = s["q"][at:at + b].to(F64)
            rows = []
            for h in range(c["heads"]):
                w = q[:, h] @ k[:, h // group].T / math.sqrt(c["dim"])
                if c["causal"]:
                    w = w + torch.full_like(w, -math.inf).triu_(a + 1)
                rows.append(torch.softmax(w, -1) @ v[:, h // group])
            out.append(torch.stack(rows, 1))
            at += b
        return torch.cat(out)
    x, l, n = s["x"].to(F64), s["logits"].to(F64), c["inner"]
    y = torch.zeros_like(x) if s["r"] is None else s["r"].to(F64)
    p = torch.exp(l - torch.logsumexp(l, -1, keepdim=True)) if c["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    # an expert is chosen where fewer than top_k come before it: larger logits, or equal ones of a lower index
    lower = torch.arange(c["experts"], device=l.device)
    before = ((l[:, None, :] > l[:, :, None]) | ((l[:, None, :] == l[:, :, None]) & (lower[None, :] < lower[:, None]))).sum(-1)
    share = torch.where(before < c["top_k"], p, torch.zeros_like(p))
    if c["normalize"]:
        share = share / share.sum(-1, keepdim=True)
    levels = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=F64, device=x.device) / 2.0
    for e in range(c["experts"]):
        mine = (share[:, e] > 0).nonzero()[:, 0]
        if not len(mine):
            continue
        W = []
        for codes, scales, alphas in (s["up"], s["down"]):
            b = codes[e].long()
            nib = torch.stack((b % 16, b // 16), -1).flatten(1)
            q = levels[nib % 8] * torch.where(nib >= 8, -1.0, 1.0)
            W.append(q * scales[e].view(E4M3).to(F64).repeat_interleave(16, 1) * alphas[e].to(F64))
        z = x[mine] @ W[0].T
        f = z[:, :n]
        if c["act"] == "silu":
            f = f / (1.0 + torch.exp(-f))
        else:
            f = 0.5 * f * (1.0 + torch.tanh(GELU_C * (f + 0.044715 * f ** 3)))
        y[mine] += share[mine, e, None] * ((f * z[:, n:] if c["gated"] else f) @ W[1].T)
    return y
