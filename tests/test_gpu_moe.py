"""The layer of experts on the GPU against binary64 (tests/decoder_ref.py), and a decoder layer's operators together."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import decoder_ref as dref
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def say(msg):
    print(msg, flush=True)


def rand(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def experts(seed, e, n, k):
    """Every code and a wide range of scales, not the quantiser's alone; an alpha of its own for each expert."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (e, n, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(0x10, 0x60, (e, n, k // 16), generator=g, device="cuda").to(torch.uint8)
    return codes, scales, (0.5 + torch.rand(e, generator=g, device="cuda")) * 0.05 / k ** 0.5


def layer(seed, e, width, inner, gated):
    return experts(seed, e, inner * (1 + gated), width), experts(seed + 1, e, width, inner)


def check(y, want, err):
    bound = err + want.abs() * ref.HALF[y.dtype] + 1e-38
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    bad = torch.nan_to_num((y.double() - want).abs() - bound, -1.0)
    assert (bad <= 0).all(), float(bad.max())


# tokens, experts, top_k, width, inner
MOE = [(1, 1, 1, 16, 16), (1, 8, 2, 128, 48), (1, 128, 8, 512, 192), (2, 60, 4, 272, 80), (5, 7, 7, 144, 1040), (8, 64, 6, 1040, 32),
       (9, 16, 1, 48, 2064), (17, 3, 2, 400, 160), (33, 8, 2, 256, 784), (64, 512, 32, 64, 16), (130, 20, 3, 112, 176),
       (257, 2, 1, 64, 64), (1024, 32, 8, 32, 48), (8192, 4, 1, 16, 16)]


@pytest.mark.parametrize("tokens,count,top_k,width,inner", MOE)
def test_moe_matches_binary64(tokens, count, top_k, width, inner):
    say(f"moe tokens={tokens} experts={count} top_k={top_k} width={width} inner={inner}")
    x = rand(1, tokens, width + 8)[:, 3:3 + width]  # rows that are not aligned
    logits = rand(2, tokens, count + 5, dtype=F32, std=2.0)[:, 1:count + 1]
    r = rand(3, tokens, width + 16)[:, :width]
    for act, gated, scoring, normalize, res, l in (
            ("silu", True, "softmax", True, None, logits), ("gelu", True, "sigmoid", False, r, logits.bfloat16()),
            ("gelu", False, "softmax", False, r, logits), (None, False, "sigmoid", True, None, logits.bfloat16())):
        up, down = layer(5, count, width, inner, gated)
        y = nv.moe(x, l, up, down, top_k, activation=act, gated=gated, scoring=scoring, normalize=normalize, residual=res)
        want, err = dref.moe(x, l, up, down, top_k, act, gated, scoring == "sigmoid", normalize, res)
        assert y.dtype == BF16 and y.shape == (tokens, width)
        check(y, want, err)


# The forms of the kernel for many weight rows: routing inside it (5 and 8 tokens), X of two slices held over
# column tiles, whole and with a short last slice, two tiles of pairs with a last one of either, the second product's sum in
# parts; a last column tile that is not whole
FORMS = [(5, 32, 4, 512, 1040), (8, 64, 6, 1040, 1408), (40, 64, 4, 2048, 1024), (40, 64, 4, 1040, 1040), (40, 64, 4, 2576, 784),
         (40, 64, 4, 1024, 2064), (100, 4, 2, 528, 3200), (70, 4, 2, 4112, 2064), (33, 8, 2, 4096, 2064), (40, 4, 1, 4096, 4112),
         (17, 8, 2, 4096, 8208), (16, 8, 2, 4096, 2064), (256, 8, 2, 1040, 1408), (200, 16, 4, 528, 528), (100, 2, 2, 2064, 400)]


@pytest.mark.parametrize("tokens,count,top_k,width,inner", FORMS)
def test_moe_of_many_rows(tokens, count, top_k, width, inner):
    say(f"moe rows tokens={tokens} experts={count} top_k={top_k} width={width} inner={inner}")
    x, logits, r = rand(1, tokens, width), rand(2, tokens, count, dtype=F32, std=2.0), rand(3, tokens, width)
    logits[0, :] = -INF  # a token of no experts
    logits[-1, 1:] = -INF  # and one of a single one
    for gated in (True, False):
        up, down = layer(7, count, width, inner, gated)
        y = nv.moe(x, logits, up, down, top_k, gated=gated, residual=r)
        want, err = dref.moe(x, logits, up, down, top_k, "silu", gated, False, True, r)
        check(y, want, err)


@pytest.mark.parametrize("width,inner", [(1024, 528), (2064, 784)])
def test_moe_of_uneven_choices(width, inner):
    """Experts that all tokens choose, beside others that few or none do: entries of one expert in several work-groups."""
    x, logits = rand(1, 150, width), rand(2, 150, 64, dtype=F32)
    logits[:, 7] += 20.0
    logits[40:, 63] += 15.0
    logits[:, 20:40] -= 30.0
    up, down = layer(9, 64, width, inner, True)
    y = nv.moe(x, logits, up, down, 3, scoring="sigmoid")
    want, err = dref.moe(x, logits, up, down, 3, "silu", True, True, True)
    check(y, want, err)


# more rows, wide sums, and weights as the quantiser writes them
@pytest.mark.parametrize("tokens,count,top_k,width,inner", [(1, 4, 2, 4096, 1408), (6, 8, 2, 2048, 5632), (70, 12, 4, 1024, 4112)])
def test_moe_of_quantised_weights(tokens, count, top_k, width, inner):
    say(f"moe quantised {tokens} {count} {top_k} {width} {inner}")
    def stack(n, k, seed):
        parts = [nv.quantize(rand(seed + i, n, k, std=k ** -0.5), "4o6") for i in range(count)]
        return tuple(torch.stack(t) if i < 2 else torch.cat(t) for i, t in enumerate(zip(*parts)))
    up, down = stack(2 * inner, width, 10), stack(width, inner, 50)
    x, logits = rand(1, tokens, width), rand(2, tokens, count, dtype=F32)
    y = nv.moe(x, logits, up, down, top_k)
    want, err = dref.moe(x, logits, up, down, top_k, "silu", True, False, True)
    check(y, want, err)


@pytest.mark.parametrize("tokens", [1, 3, 8, 20])
def test_choices(tokens):
    """Experts as one-hot rows: y shows which experts were taken, with which weights. Ties, -inf, all alike, signed zeros."""
    count, width = 16, 16
    codes = torch.zeros(count, 16, 8, dtype=torch.uint8, device="cuda")
    scales = torch.full((count, 16, 1), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    up = codes.clone()
    up[:, 0, 0] = 0x02  # h[0] = x[0]
    down = codes.clone()
    for e in range(count):
        down[e, e, 0] = 0x02  # y[e] = h[0]
    one = torch.ones(count, device="cuda")
    x = torch.zeros(tokens, width, dtype=BF16, device="cuda")
    x[:, 0] = 1.0
    rows = [[1.0] * count, [0.0, -0.0] * 8, [-INF] * count, [-INF] * 5 + [2.0] + [-INF] * 10, [float(i % 3) for i in range(count)],
            [-300.0 - i for i in range(count)], [300.0 + i for i in range(count)], [float(-i) for i in range(count)]]
    logits = torch.tensor([rows[i % len(rows)] for i in range(tokens)], device="cuda")
    for first in range(len(rows)):
        l = torch.roll(logits, first, 0) if tokens > 1 else torch.tensor([rows[first]], device="cuda")
        for sigmoid in (False, True):
            for normalize in (False, True):
                y = nv.moe(x, l, (up, scales, one), (down, scales, one), 4, activation=None, gated=False,
                           scoring="sigmoid" if sigmoid else "softmax", normalize=normalize)
                chosen, w, ew = dref.route(l, 4, sigmoid, normalize)
                assert torch.equal(y != 0, (w > 2.0 ** -126) & chosen) or not normalize
                assert (y[~chosen] == 0).all()
                check(y, w, w * ew + 2.0 ** -126)


def test_values_that_are_not_finite():
    """A NaN among a token's logits or inputs makes NaN of its row alone."""
    up, down = layer(1, 8, 64, 32, True)
    x, logits = rand(1, 6, 64), rand(2, 6, 8, dtype=F32)
    clean = nv.moe(x, logits, up, down, 2)
    for normalize in (True, False):
        for scoring in ("softmax", "sigmoid"):
            bad = logits.clone()
            bad[2, 5] = float("nan")
            y = nv.moe(x, bad, up, down, 2, normalize=normalize, scoring=scoring)
            same = nv.moe(x, logits, up, down, 2, normalize=normalize, scoring=scoring)
            assert torch.isnan(y[2]).all()
            y[2] = same[2]
            assert torch.equal(y, same)
    bad = x.clone()
    bad[4, 3] = float("nan")
    y = nv.moe(bad, logits, up, down, 2)
    assert torch.isnan(y[4]).all()
    y[4] = clean[4]
    assert torch.equal(y, clean)


def test_only_chosen_experts_are_read():
    """Experts that no token chose may hold anything."""
    up, down = layer(1, 40, 128, 64, True)
    x, logits = rand(1, 5, 128), rand(2, 5, 40, dtype=F32)
    y = nv.moe(x, logits, up, down, 3)
    chosen, _, _ = dref.route(logits, 3, False, True)
    idle = ~chosen.any(0)
    for W in (up, down):
        W[0][idle], W[1][idle], W[2][idle] = 0xFF, 0x7F, float("nan")
    assert torch.equal(nv.moe(x, logits, up, down, 3), y)


def test_buffers_and_reproducibility():
    up, down = layer(1, 16, 256, 112, True)
    x, logits, r = rand(1, 40, 256), rand(2, 40, 16, dtype=F32), rand(3, 40, 256)
    y = nv.moe(x, logits, up, down, 4, residual=r)
    ws = torch.full((nv.moe_workspace_bytes(40, 256, 112, 16, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(y)
    for _ in range(3):
        assert nv.moe(x, logits, up, down, 4, residual=r, workspace=ws, out=out) is out and torch.equal(out, y)
    both = r.clone()
    assert torch.equal(nv.moe(x, logits, up, down, 4, residual=both, out=both), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = nv.moe(x, logits, up, down, 4, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(z, y)
    # parts of the tokens, each by the kernels that its size takes
    want, err = dref.moe(x, logits, up, down, 4, "silu", True, False, True, r)
    check(y, want, err)
    for lo, hi in ((0, 1), (3, 8), (3, 15), (20, 40)):
        check(nv.moe(x[lo:hi], logits[lo:hi], up, down, 4, residual=r[lo:hi]), want[lo:hi], err[lo:hi])
    assert nv.moe(x[:0], logits[:0], up, down, 4).shape == (0, 256)


@pytest.mark.parametrize("tokens", [1, 8, 40])
def test_graph(tokens):
    up, down = layer(1, 16, 256, 112, True)
    x, logits = rand(1, tokens, 256), rand(2, tokens, 16, dtype=F32)
    ws = torch.empty(nv.moe_workspace_bytes(tokens, 256, 112, 16, 4), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    nv.moe(x, logits, up, down, 4, workspace=ws, out=out)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = [torch.empty_like(x) for _ in graphs]
    for graph, o in zip(graphs, outs):
        with torch.cuda.graph(graph):
            nv.moe(x, logits, up, down, 4, workspace=ws, out=o)
    for i in range(4):
        x.copy_(rand(30 + i, tokens, 256))
        logits.copy_(rand(60 + i, tokens, 16, dtype=F32))
        want = nv.moe(x, logits, up, down, 4)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want)
        torch.randn(1000, device="cuda").sum().item()


def test_refusals():
    up, down = layer(1, 8, 64, 32, True)
    x, logits = rand(1, 6, 64), rand(2, 6, 8, dtype=F32)
    E = nv.NVFP4Error
    good = (x, logits, up, down, 2)
    swap = lambda W, i, t: tuple(t if k == i else v for k, v in enumerate(W))  # noqa: E731
    for at, bad in ((0, x.float()), (0, x[0]), (0, x[:, :32]), (0, x[:5]), (1, logits.half()), (1, logits[:, :7]), (1, logits[:5]),
                    (2, up[:2]), (2, down), (2, swap(up, 0, up[0][:7])), (2, swap(up, 1, up[1][:, :, :3])),
                    (2, swap(up, 2, up[2][:7])), (2, swap(up, 2, up[2].double())), (2, swap(up, 0, up[0].cpu())),
                    (2, swap(up, 0, up[0].transpose(1, 2).contiguous().transpose(1, 2))), (3, up), (3, down[:2]),
                    (4, 0), (4, -1), (4, 9)):
        args = list(good)
        args[at] = bad
        with pytest.raises(E):
            nv.moe(*args)
    for kw in (dict(activation=None), dict(activation="relu"), dict(scoring="top"), dict(residual=x.float()),
               dict(residual=x[:5]), dict(out=x.float()), dict(out=x[:, ::2]), dict(gated=False),
               dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(E):
            nv.moe(*good, **kw)
    many = rand(1, 4097, 64)
    with pytest.raises(E):
        nv.moe(many, rand(2, 4097, 8, dtype=F32), up, down, 2)
    with torch.enable_grad(), pytest.raises(E):
        nv.moe(x.clone().requires_grad_(), logits, up, down, 2)


def test_a_decoder_layer():
    """A layer's operators in a row, a prompt and then single tokens: norm, product, rotary positions, cache, attention,
    product with the residual, norm, experts. Each call is held to binary64 on what the call before it gave."""
    width, heads, kv_heads, dim, count, top_k, inner = 256, 4, 2, 64, 8, 2, 96
    wqkv = nv.quantize(rand(1, (heads + 2 * kv_heads) * dim, width, std=0.06), "4o6")
    wo = nv.quantize(rand(2, width, heads * dim, std=0.06), "4o6")
    up, down = layer(3, count, width, inner, True)
    router = rand(5, count, width, std=0.1)
    n1, n2 = (1.0 + 0.1 * rand(i, width, dtype=F32) for i in (6, 7))
    lengths = [70, 3, 129]
    table = torch.randperm(12, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(3, 4).cuda()
    cache = nv.kv_cache(12, kv_heads, dim)
    state = dref.Cache(cache)
    for turn in range(3):
        new = lengths if turn == 0 else [1] * 3
        total = [a + turn for a in lengths]
        spans, first = [], 0
        for n, length in zip(new, total):
            spans.append((first, n, length))
            first += n
        x = rand(10 + turn, first, width)
        pos = torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).cuda()
        lens = torch.tensor(total, dtype=torch.int32, device="cuda")
        starts = torch.tensor([s[0] for s in spans] + [first], dtype=torch.int32, device="cuda") if turn == 0 else None
        h = nv.rms_norm(x, n1)
        qkv = nv.linear(h, *wqkv).view(first, heads + 2 * kv_heads, dim)
        qk = qkv[:, :heads + kv_heads]
        want, err = dref.rotary(qk, pos, (dim // 2,), 10000.0)
        nv.rotary(qk, pos, out=qk)
        check(qk, want, err)
        K, V = qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        state.append((K, V), table, spans)
        nv.kv_append(cache, K, V, table, lens, starts)
        got = dref.Cache(cache)
        assert all(torch.equal(a, b) for a, b in zip(got.codes + got.byte, state.codes + state.byte))
        o = nv.attention(qkv[:, :heads], cache, table, lens, starts)
        want, err = dref.attention(qkv[:, :heads], cache, table, spans, dim ** -0.5, True)
        check(o, want, err)
        s = nv.linear(o.view(first, heads * dim), *wo, residual=x)
        want, _, err, _ = ref.linear(o.view(first, heads * dim).double(), *wo, res=x)
        check(s, want, err)
        h = nv.rms_norm(s, n2)
        logits = (h.float() @ router.float().T)
        y = nv.moe(h, logits, up, down, top_k, residual=s)
        want, err = dref.moe(h, logits, up, down, top_k, "silu", True, False, True, s)
        check(y, want, err)
