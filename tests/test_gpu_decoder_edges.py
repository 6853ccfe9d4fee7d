"""Calls at the edges of the decoder operators, on the GPU: what is not finite beside what is, values at the end of a type's range,
caches and lists far longer than those of tests/test_gpu_decoder.py, streams and graphs of their own."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import decoder_ref as dref
from tests import test_gpu_decoder as dec
from tests import test_gpu_moe as moe_of
from tests.test_gpu_decoder import SPLIT, ints, rand, spans, starts_of, u8

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print(msg, flush=True)


# ----------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("dim", [64, 80])
@pytest.mark.parametrize("new", [[1, 1], [5, 3], [20, 9], [600, 90]])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_queries_of_infinities(dim, new, width):
    """softmax of scores that are all -inf is NaN, as of any with +inf among them: a row with an infinite query is NaN where it sees
    a token, zeros where it sees none, and the other rows are what they are without it, bit for bit."""
    say(f"infinite queries {dim} {new} {width}")
    lengths = [700, 90]
    cache, table = dec.ready(12, lengths, 2, dim, width=width)
    u8(cache.k)[:, :, :, 3] = 0x38  # all keys' column 3 is positive
    q = rand(3, sum(new), 8, dim)
    args = (cache, table, ints(lengths), starts_of(spans(lengths, new)))
    for causal in (True, False):
        clean = nv.attention(q, *args, causal=causal)
        bad = q.clone()
        rows = [(0, 1, -1.0), (sum(new) - 1, 6, -1.0), (new[0] - 1, 7, 1.0), (sum(new) // 2, 2, -1.0)]
        for row, head, sign in rows:
            bad[row, head, 3] = sign * float("inf")
        o = nv.attention(bad, *args, causal=causal)
        for row, head, _ in rows:
            assert torch.isnan(o[row, head]).all(), (row, head)
            o[row, head] = clean[row, head]
        assert torch.equal(o, clean)
    # rows that see none: no pages, no tokens, more new tokens than tokens
    nowhere = torch.full_like(table, -1)
    assert (nv.attention(bad, cache, nowhere, *args[2:]) == 0).all()
    assert (nv.attention(bad, cache, table, ints([0, 0]), args[3]) == 0).all()
    if new[0] > 1:
        o = nv.attention(bad, cache, table, ints([new[0] - 1, new[1] - 1]), args[3])
        assert (o[0] == 0).all() and (o[new[0]] == 0).all()


def held(lengths, new, heads, kv_heads, dim, width=None, bad=()):
    """Attention of such sequences against binary64, causal and not, twice the same, and with blocks (sequence, block, key head) of
    NaN in keys or values or, without a head, missing."""
    table, pages = dec.layout(6, lengths, width=width)
    cache = nv.kv_cache(pages, kv_heads, dim)
    dec.fill(cache, 6)
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    args = (q, cache, table, ints(lengths), starts_of(sp))
    for causal in (True, False):
        o = nv.attention(*args, causal=causal)
        dec.check(o, *dref.attention(q, cache, table, sp, dim ** -0.5, causal))
        assert torch.equal(nv.attention(*args, causal=causal), o)
    if all(n == 1 for n in new):
        assert torch.equal(nv.attention(*args[:4]), nv.attention(*args))
    for i, (s, block, head) in enumerate(bad):
        if head is None:
            table[s, block] = -1 if i % 2 else 1 << 30
        else:
            u8(cache[2 + i % 2])[int(table[s, block]), head] = 255
    if bad:
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, True)
        assert torch.isnan(want).any()
        dec.check(nv.attention(*args), want, err)


# Tiles in more than 16, 64 and 256 parts, joined by a work-group or by a wave; shares of more than 256 blocks (a wave looks its pages up
# more than once), with a work-group for each CU instead of two, padded to whole shares (two sequences) and not (five)
FAR = [
    ([8000], [1], 4, 1, 64, None, [(0, 101, None), (0, 120, 0)]),
    ([20011], [2], 7, 1, 32, None, [(0, 250, None), (0, 301, 0)]),
    ([80003], [1], 2, 1, 16, None, [(0, 700, None), (0, 1249, 0)]),
    ([80003] + [30 + i for i in range(79)], [1] * 80, 3, 1, 16, None, [(0, 800, None), (0, 1100, 0), (40, 0, 0)]),
    ([40000, 39001], [1, 1], 128, 64, 16, None, [(0, 290, None), (1, 600, None), (0, 300, 5), (1, 607, 63)]),
    ([20000, 19000, 21000, 64, 18001], [1, 3, 1, 2, 1], 64, 64, 16, None, [(2, 3, None), (0, 312, 7), (4, 280, None), (2, 310, 9)]),
    ([30000, 35000, 31, 33333], [6, 5, 3, 2], 192, 32, 32, None, [(1, 400, None), (3, 333, 31), (0, 111, 4)]),
]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim,width,bad", FAR, ids=[f"{len(c[0])}x{c[0][0]}-{c[3]}x{c[4]}" for c in FAR])
def test_attention_far(lengths, new, heads, kv_heads, dim, width, bad):
    say(f"far {lengths[:5]} {new[:5]} {heads} {kv_heads} {dim}")
    held(lengths, new, heads, kv_heads, dim, width, bad)


# A single token over more than 256 blocks beside a prompt, in the kernel of many rows
@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim,width", [([500, 20000], [300, 1], 4, 1, 64, None), ([30001, 700], [2, 600], 6, 2, 128, None),
                                                                  ([17000, 90, 400], [1, 1, 400], 2, 1, 256, 300)])
def test_attention_far_beside_prompts(lengths, new, heads, kv_heads, dim, width):
    say(f"far beside prompts {lengths} {new} {heads} {kv_heads} {dim}")
    far = lengths.index(max(lengths))
    held(lengths, new, heads, kv_heads, dim, width, [(far, 257, None), (1 - far if far < 2 else 0, 1, 0), (far, 260, kv_heads - 1)])


# Chunks of hundreds of rows beside so many single tokens that the call goes by blocks: many tiles of a sequence among the shares, of 16
# rows and, over wide tables, of 32
@pytest.mark.parametrize("chunk,singles,heads,kv_heads,dim,width", [
    (200, 40, 4, 1, 64, SPLIT), (200, 40, 4, 1, 64, 200), (301, 90, 7, 1, 80, 100), (512, 128, 4, 1, 128, 170), (100, 70, 8, 4, 256, SPLIT),
    (250, 30, 6, 2, 192, SPLIT), (64, 70, 16, 1, 48, 100)])
def test_attention_of_chunks_among_single_tokens(chunk, singles, heads, kv_heads, dim, width):
    say(f"chunks {chunk} {singles} {heads} {kv_heads} {dim} {width}")
    lengths = [20 + 61 * i % 1500 for i in range(singles)]
    new = [1] * singles
    lengths[singles // 2:singles // 2], new[singles // 2:singles // 2] = [chunk + 190], [chunk]
    rows = -(-sum(new) * heads // kv_heads // len(new))
    assert 4 < rows <= 32 and width > 64
    held(lengths, new, heads, kv_heads, dim, width, [(singles // 2, 3, 0), (3, 1, None), (singles // 2, 1, None), (singles, 0, kv_heads - 1)])


@pytest.mark.parametrize("lengths,new", [([900, 70, 3000], [1, 1, 1]), ([700, 64, 300], [300, 64, 2]), ([4000, 3000], [30, 50])])
def test_attention_on_a_stream_of_its_own(lengths, new):
    """Rotary positions, cache and attention on a stream, each result compared; scratch of the call's own and the caller's."""
    heads, kv_heads, dim = 8, 2, 64
    table, pages = dec.layout(1, lengths, width=SPLIT)
    sp = spans(lengths, new)
    qkv, pos = rand(1, sum(new), heads + 2 * kv_heads, dim), torch.arange(sum(new), device="cuda")
    caches = [nv.kv_cache(pages, kv_heads, dim) for _ in range(2)]
    for c in caches:
        dec.fill(c, 5)
    ws = torch.empty(nv.attention_workspace_bytes(sum(new), len(new), SPLIT, heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
    lens, starts = ints(lengths), starts_of(sp)

    def step(cache, stream, workspace):
        x = nv.rotary(qkv, pos, sections=(16,), stream=stream)
        nv.kv_append(cache, x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], table, lens, starts, stream=stream)
        return x, nv.attention(x[:, :heads], cache, table, lens, starts, workspace=workspace, stream=stream)

    x, o = step(caches[0], None, None)
    want, err = dref.attention(x[:, :heads], caches[0], table, sp, dim ** -0.5, True)
    dec.check(o, want, err)
    side = torch.cuda.Stream()
    for workspace in (None, ws):
        dec.fill(caches[1], 5)
        side.wait_stream(torch.cuda.current_stream())
        on_side = step(caches[1], side, workspace)
        side.synchronize()
        assert torch.equal(on_side[0], x) and torch.equal(on_side[1], o)
        assert all(torch.equal(u8(a), u8(b)) for a, b in zip(*caches))
        with torch.cuda.stream(side):  # the current stream
            again = step(caches[1], None, workspace)
        side.synchronize()
        assert torch.equal(again[0], x) and torch.equal(again[1], o)


@pytest.mark.parametrize("lengths,new", [([3000, 20, 700], [1, 1, 1]), ([4000, 3000], [30, 50])])
def test_two_graphs_share_a_workspace(lengths, new):
    """Attention captured twice over one workspace, replayed in turn with other queries, lengths and pages."""
    heads, kv_heads, dim, width = 8, 2, 128, SPLIT
    cache, table = dec.ready(4, lengths, kv_heads, dim, width=width)
    q, lens, starts = rand(1, sum(new), heads, dim), ints(lengths), starts_of(spans(lengths, new))
    ws = torch.empty(nv.attention_workspace_bytes(sum(new), len(new), width, heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    tables, outs = [table.clone(), table.flip(1).contiguous()], [torch.empty_like(q) for _ in range(2)]
    nv.attention(q, cache, table, lens, starts, workspace=ws, out=outs[0])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, t, o in zip(graphs, tables, outs):
        with torch.cuda.graph(graph):
            nv.attention(q, cache, t, lens, starts, workspace=ws, out=o)
    for i in range(4):
        q.copy_(rand(30 + i, *q.shape))
        lens.add_(-7)
        for graph, t, o in zip(graphs, tables, outs):
            want = nv.attention(q, cache, t, lens, starts)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)
            torch.randn(1000, device="cuda").sum().item()
        assert not torch.equal(*outs)


@pytest.mark.parametrize("last", [64, 0])
def test_starts_that_run_backwards(last):
    """Starts that give many sequences the same rows: the blocks of all tiles are 2^32 and a few (or 2^32, which is none to 32
    bits). What the rows get is open, but nothing beside the output is written, and the next call is right."""
    say(f"starts that run backwards {last}")
    seqs, tokens, width, heads, dim = 1026, 1024, 8192, 16, 16
    cache = nv.kv_cache(4, 1, dim)
    dec.fill(cache, 1)
    table = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    lengths = [width * 64] * 1024 + [last, 0]
    starts = [0 if i % 2 == 0 else tokens for i in range(seqs)] + [0]
    need = nv.attention_workspace_bytes(tokens, seqs, width, heads, 1, dim)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((tokens + 64, heads, dim), 7.0, dtype=BF16, device="cuda")
    q = rand(2, tokens, heads, dim)
    nv.attention(q, cache, table, ints(lengths), ints(starts), workspace=ws[:need], out=out[32:-32])
    torch.cuda.synchronize()
    assert (ws[need:] == 0xA5).all() and (out[:32] == 7.0).all() and (out[-32:] == 7.0).all()
    table, lengths, q = table[:100, :SPLIT], [1 + 7 * i % 130 for i in range(100)], q[:100]
    o = nv.attention(q, cache, table, ints(lengths))
    want, err = dref.attention(q, cache, table, spans(lengths, [1] * 100), dim ** -0.5, True)
    dec.check(o, want, err)


# ------------------------------------------------------------------------------------------- the cache

def bits(pattern):
    return torch.tensor(pattern, dtype=torch.int32).view(F32).item()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", [0, 1])
def test_append_of_the_largest_values(dtype, which):
    """248 * 2^120 is half way between the codes of 240 and 256 at scale 2^120 and goes to 256 * 2^120 = 2^128, which is no binary32 number: from
    there on a value makes its block one of NaNs as an infinity does, below it is held."""
    table, pages = dec.layout(3, [130])
    below = [bits(0x7F770000)] if dtype == BF16 else [bits(0x7F770000), bits(0x7F77FFFF)]  # 247 * 2^120, and the last below 248
    beyond = [bits(0x7F780000), bits(0x7F7F0000)] + ([] if dtype == BF16 else [bits(0x7F7FFFFF)])  # 248 and 255 * 2^120, the last
    for value in below + [-v for v in below] + beyond + [-v for v in beyond]:
        cache = nv.kv_cache(pages, 2, 32)
        x = [rand(i, 130, 2, 32, dtype=dtype) for i in (1, 2)]
        x[which][70, 1, 9] = value
        nv.kv_append(cache, *x, table, ints([130]), ints([0, 130]))
        page = int(table[0, 1])
        byte, codes = u8(cache[2 + which])[page], u8(cache[which])[page, 1]
        assert byte[0] != 255 and all((u8(s)[int(table[0, b])] != 255).all() for s in cache[2:] for b in (0, 2))
        if abs(value) < bits(0x7F780000):
            at = codes[6, 9] if which == 0 else codes[9, 6]
            assert byte[1] == 247 and at == (0x77 if value > 0 else 0xF7)  # 240 * 2^120
        else:
            assert byte[1] == 255 and (codes == 0x7F).all()


@pytest.mark.parametrize("new,behind", [(6, 3), (20, 10), (100, 60)])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_rows_that_do_not_see_the_largest_values(new, behind, width):
    """Rows whose tokens end in front of a block with such a value are what they are without it, beside rows that see it."""
    heads, dim, length = 2, 64, 64 + behind
    table, pages = dec.layout(3, [length], width=width)
    q = rand(5, new, 4, dim)
    out = []
    for value in (1.0, bits(0x7F7F0000)):
        cache = nv.kv_cache(pages, heads, dim)
        K, V = rand(1, length, heads, dim), rand(2, length, heads, dim)
        V[-1, 1, 9] = value
        nv.kv_append(cache, K, V, table, ints([length]), ints([0, length]))
        out.append(nv.attention(q, cache, table, ints([length]), ints([0, new])))
    apart = new - behind  # row i sees length - new + i + 1 tokens: these at most 64
    assert torch.equal(out[0][:apart], out[1][:apart])
    assert torch.equal(out[0][:, :2], out[1][:, :2])  # the other key head's
    assert torch.isnan(out[1][apart:, 2:]).all()


def test_outputs_that_share_memory_with_an_operand():
    """The operand itself is fine, and so is memory between its rows; anything else is refused."""
    E = nv.NVFP4Error
    buf = rand(1, 12 * 40 * 64)
    at = lambda first, tokens, heads, stride: buf[first:first + 40 * 64 * 4].as_strided((tokens, heads, 64), (stride, 64, 1))  # noqa: E731
    x, pos = at(64, 5, 8, 40 * 64), torch.arange(5, device="cuda")
    for first in (0, 64 + 8, 64 + 2 * 40 * 64, 64 + 7 * 64, 64 + 4 * 40 * 64 + 7 * 64 + 63):
        with pytest.raises(E):
            nv.rotary(x, pos, out=buf[first:first + 5 * 8 * 64].view(5, 8, 64))
    small = at(0, 2, 4, 40 * 64)
    between = buf[4 * 64:4 * 64 + 2 * 4 * 64].view(2, 4, 64)  # behind the first row's heads, in front of the second's
    y = nv.rotary(small, pos[:2])
    with torch.device("cuda"):  # (the check does its sums on the host whatever the default device is)
        with pytest.raises(E):
            nv.rotary(x, pos, out=buf[64 + 8:64 + 8 + 5 * 8 * 64].view(5, 8, 64))
        assert torch.equal(nv.rotary(small, pos[:2], out=between), y)
    want = nv.rotary(x, pos)
    assert torch.equal(nv.rotary(x, pos, out=x), want)
    # attention: in place over each of its kernels; the first heads of a wider product are not a contiguous output
    for lengths, new, width in (([900, 70], [1, 1], SPLIT), ([900, 70], [1, 1], None), ([900, 70], [20, 9], SPLIT), ([2000, 300], [600, 300], None),
                                ([5000, 64], [40, 30], 160)):
        cache, table = dec.ready(2, lengths, 2, 64, width=width)
        args = (cache, table, ints(lengths), starts_of(spans(lengths, new)))
        wide = rand(3, sum(new), 12, 64)
        q = wide[:, :8].contiguous()
        o = nv.attention(q, *args)
        with pytest.raises(E):
            nv.attention(wide[:, :8], *args, out=wide.view(-1)[:q.numel()].view(q.shape))
        assert torch.equal(nv.attention(q, *args, out=q), o) and torch.equal(q, o)
    one = wide[:1, :8]  # a single row is the same memory whatever its stride
    o = nv.attention(one, cache, table[:1], ints([64]))
    assert torch.equal(nv.attention(one, cache, table[:1], ints([64]), out=wide.view(-1)[:512].view(1, 8, 64)), o)
    # experts: the residual, and the inputs
    up, down = moe_of.layer(1, 8, 64, 32, True)
    for tokens in (4, 40):
        both, logits = moe_of.rand(3, 2 * tokens, 64), moe_of.rand(2, tokens, 8, dtype=F32)
        x = moe_of.rand(1, tokens, 64)
        for residual, out in ((both[::2], both[:tokens]), (both[1:tokens + 1], both[:tokens]), (both[:tokens], both[1:tokens + 1])):
            with pytest.raises(E):
                nv.moe(x, logits, up, down, 2, residual=residual, out=out)
        y = nv.moe(x, logits, up, down, 2, residual=both[:tokens])
        assert torch.equal(nv.moe(x, logits, up, down, 2, residual=both[:tokens], out=both[:tokens]), y)
        y = nv.moe(x, logits, up, down, 2)
        assert torch.equal(nv.moe(x, logits, up, down, 2, out=x), y)


def test_a_cache_without_heads_is_refused():
    cache = (torch.zeros(2, 0, 64, 16, dtype=torch.uint8, device="cuda"), torch.zeros(2, 0, 16, 64, dtype=torch.uint8, device="cuda"),
             torch.zeros(2, 0, dtype=torch.uint8, device="cuda"), torch.zeros(2, 0, dtype=torch.uint8, device="cuda"))
    table, lengths = ints([[0]]), ints([1])
    for heads in (0, 2):
        with pytest.raises(nv.NVFP4Error):
            nv.attention(rand(1, 1, heads, 16), cache, table, lengths)
    with pytest.raises(nv.NVFP4Error):
        nv.kv_append(cache, rand(1, 1, 0, 16), rand(1, 1, 0, 16), table, lengths)


# ------------------------------------------------------------------------------------------- experts

# More than 2048 pairs, which the kernel of many rows lists in several loads of its ids, to the most that there may be; experts that most
# tokens choose beside others of few; one tile of pairs an expert and two, X held and not
@pytest.mark.parametrize("tokens,count,top_k,width,inner", [(600, 16, 8, 256, 256), (1024, 16, 8, 128, 1040), (2047, 8, 4, 1040, 144),
                                                            (8192, 64, 1, 256, 128), (260, 512, 31, 128, 128)])
def test_moe_of_many_pairs(tokens, count, top_k, width, inner):
    say(f"many pairs {tokens} {count} {top_k} {width} {inner}")
    x, logits, r = moe_of.rand(1, tokens, width), moe_of.rand(2, tokens, count, dtype=F32), moe_of.rand(3, tokens, width)
    logits[:, 1] += 4.0
    logits[:, count // 2] -= 4.0
    logits[tokens // 2] = -moe_of.INF
    for gated in (True, False):
        up, down = moe_of.layer(7, count, width, inner, gated)
        y = nv.moe(x, logits, up, down, top_k, gated=gated, scoring="sigmoid", residual=r)
        want, err = dref.moe(x, logits, up, down, top_k, "silu", gated, True, True, r)
        moe_of.check(y, want, err)
        assert torch.equal(nv.moe(x, logits, up, down, top_k, gated=gated, scoring="sigmoid", residual=r), y)


@pytest.mark.parametrize("tokens", [2, 3, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("which", ["up", "down"])
@pytest.mark.parametrize("bad", ["scale", "alpha"])
def test_weights_that_are_not_finite_stay_with_their_tokens(tokens, which, bad):
    """A NaN scale byte or an infinite alpha of an expert reaches the tokens that chose it, and no others: they are what they
    are with sound weights, bit for bit."""
    say(f"not finite weights {tokens} {which} {bad}")
    up, down = moe_of.layer(1, 8, 256, 160, True)
    x, logits = moe_of.rand(1, tokens, 256), moe_of.rand(2, tokens, 8, dtype=F32)
    logits[0, 5], logits[1, 5] = 30.0, -30.0  # chosen by the first, not by the second
    clean = nv.moe(x, logits, up, down, 2)
    chosen, _, _ = dref.route(logits, 2, False, True)
    W = up if which == "up" else down
    if bad == "scale":
        W[1][5] = 0x7F
    else:
        W[2][5] = float("inf")
    y = nv.moe(x, logits, up, down, 2)
    mine = chosen[:, 5]
    assert mine[0] and not mine[1]
    assert not torch.isfinite(y[mine]).any() if bad == "scale" else not torch.isfinite(y[mine]).all()
    assert torch.equal(y[~mine], clean[~mine])
