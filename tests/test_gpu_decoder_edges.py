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
