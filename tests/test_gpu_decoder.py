"""Rotary positions, the cache in 8 bits and attention over it, on the GPU against binary64 (tests/decoder_ref.py)."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import decoder_ref as dref
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
PAGE = 64


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(seed, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * std).to(dtype)


def u8(t):
    return t.view(torch.uint8)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(y, want, err):
    bound = err + want.abs() * ref.HALF[y.dtype] + 1e-38
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    bad = torch.nan_to_num((y.double() - want).abs() - bound, -1.0)
    assert (bad <= 0).all(), float(bad.max())


# ------------------------------------------------------------------------------------------- rotary

# (tokens, heads, dim, sections)
ROTARY = [(1, 1, 2, (1,)), (1, 40, 128, (64,)), (3, 5, 64, (32,)), (7, 3, 80, (8, 16, 16)), (130, 2, 256, (128,)),
          (5, 33, 96, (12,)), (33, 4, 37, (3, 0, 5)), (600, 9, 128, (16, 24, 24)), (2, 2, 200, (10, 20, 30, 40))]


@pytest.mark.parametrize("tokens,heads,dim,sections", ROTARY)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotary(tokens, heads, dim, sections, dtype):
    say(f"rotary {tokens} {heads} {dim} {sections}")
    wide = rand(tokens + dim, tokens, heads + 2, dim, dtype=dtype)
    x = wide[:, 1:heads + 1]
    for ptype, top in ((torch.int64, 2 ** 33), (torch.int32, 2 ** 20)):
        pos = torch.randint(-top // 4, top, (len(sections), tokens), generator=gen(5), device="cuda").to(ptype)
        for base, inverse in ((10000.0, False), (500000.0, True)):
            want, err = dref.rotary(x, pos, sections, base, inverse)
            check(nv.rotary(x, pos, sections=sections, base=base, inverse=inverse), want, err)
            before = wide.clone()
            assert nv.rotary(x, pos, sections=sections, base=base, inverse=inverse, out=x) is x
            check(x, want, err)
            assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, -1], before[:, -1])
            assert torch.equal(x[..., 2 * sum(sections):], before[:, 1:-1, 2 * sum(sections):])
            wide.copy_(before)


def test_rotary_of_one_axis_and_other_layouts():
    x = rand(1, 6, 4, 64, dtype=F32)
    pos = torch.arange(6, device="cuda")
    y = nv.rotary(x, pos)
    want, err = dref.rotary(x, pos, (32,), 10000.0)
    check(y, want, err)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)  # heads are the outer dimension in memory
    assert torch.equal(nv.rotary(heads_first, pos), y)
    out = torch.empty_like(x)
    assert nv.rotary(x, pos, out=out) is out and torch.equal(out, y)
    assert torch.equal(nv.rotary(x, torch.zeros_like(pos)), x)
    assert nv.rotary(x[:0], pos[:0]).shape == (0, 4, 64)
    back = nv.rotary(y, pos, inverse=True)  # two roundings and the sines' errors, twice
    assert ((back - x).abs() <= 2.0 ** -19 * x.abs().amax()).all()


def test_rotary_gradient():
    """The gradient is the inverse call: against autograd of the formula in binary64, and against differences."""
    x = rand(3, 5, 3, 48, dtype=F32)
    pos = torch.randint(0, 5000, (2, 5), device="cuda", generator=gen(2))
    dy = rand(4, 5, 3, 48, dtype=F32)
    xd = x.double().requires_grad_()
    (dref.rotary(xd, pos, (7, 9), 100.0)[0] * dy.double()).sum().backward()
    dx = nv.rotary(dy, pos, sections=(7, 9), base=100.0, inverse=True)
    _, err = dref.rotary(dy, pos, (7, 9), 100.0, True)
    check(dx, xd.grad, err)
    step = rand(6, 5, 3, 48, dtype=F32)
    f = lambda t: (nv.rotary(t, pos, sections=(7, 9), base=100.0).double() * dy.double()).sum()  # noqa: E731
    # linear: a difference is exact but for the roundings, each at most 2^-21 of a term
    slack = 2.0 ** -19 * float((dy.double().abs() * (x.abs() + step.abs()).double()).sum()) * 2
    assert abs(float(f(x + step) - f(x)) - float((dx.double() * step.double()).sum())) <= slack


# --------------------------------------------------------------------------------- caches and sequences

def fill(cache, seed):
    """Every byte of the cache: finite codes and scales of moderate size, as earlier sequences leave them."""
    g = gen(seed)
    for t in cache[:2]:
        c = torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8)
        u8(t).copy_(torch.where((c & 127) == 127, c - 1, c))
    for t in cache[2:]:
        u8(t).copy_(torch.randint(115, 121, t.shape, generator=g, device="cuda").to(torch.uint8))


def layout(seed, lengths, extra=2, width=None):
    """A table of shuffled pages (unused entries far outside the cache) and the number of pages."""
    need = [-(-n // PAGE) for n in lengths]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lengths), (width or max(need + [1])) + 3), 1 << 30, dtype=torch.int32)
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return table.cuda()[:, :-3], pages  # rows of the table are not contiguous


def spans(lengths, new, first=0):
    out = []
    for length, n in zip(lengths, new):
        out.append((first, n, length))
        first += n
    return out


def starts_of(sp):
    return ints([s[0] for s in sp] + [sp[-1][0] + sp[-1][1]])


# ------------------------------------------------------------------------------------------- append

APPEND = [
    # lengths (with the new tokens), new tokens, heads, dim
    ([1, 64, 65, 100, 128, 129, 7], [1] * 7, 3, 128),
    ([1], [1], 1, 16),
    ([64, 300, 1, 0, 77, 200], [64, 37, 1, 0, 77, 3], 2, 80),
    ([1000, 130], [1000, 66], 2, 256),
    ([63, 64, 65, 66, 190], [2, 2, 2, 2, 128], 5, 48),
]


@pytest.mark.parametrize("lengths,new,heads,dim", APPEND)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_is_exact(lengths, new, heads, dim, dtype):
    say(f"append {lengths} {new} {heads} {dim}")
    table, pages = layout(7, lengths)
    cache = nv.kv_cache(pages, heads, dim)
    lens = ints(lengths)
    for trial, std in enumerate((1.0, 30.0, 1e-30)):  # scales below, above and far below those of the cache
        fill(cache, trial)
        sp = spans(lengths, new, first=2)
        rows = sum(new) + 5  # two rows in front, three behind
        K, V = (rand(trial * 10 + i, rows, 2 * heads, dim, dtype=dtype, std=std)[:, heads:] for i in (1, 2))
        want = dref.Cache(cache)
        want.append((K, V), table, sp)
        assert nv.kv_append(cache, K, V, table, lens, starts_of(sp)) is cache
        got = dref.Cache(cache)
        for a, b in zip(got.codes + got.byte, want.codes + want.byte):
            assert torch.equal(a, b)
        before = [t.clone() for t in cache]
        nv.kv_append(cache, K, V, table, lens, starts_of(sp))  # the same tokens again: nothing moves
        assert all(torch.equal(u8(a), u8(b)) for a, b in zip(before, cache))
        if all(n == 1 for n in new):
            fill(cache, trial)
            nv.kv_append(cache, K[2:-3], V[2:-3], table, lens)
            assert all(torch.equal(u8(a), u8(b)) for a, b in zip(before, cache))


def test_append_token_by_token():
    """A sequence written one token at a time, scales growing on the way, against the reference's same steps."""
    heads, dim = 2, 64
    table, pages = layout(1, [150])
    cache = nv.kv_cache(pages, heads, dim)
    fill(cache, 3)
    want = dref.Cache(cache)
    for t in range(150):
        std = 2.0 ** ((t * 7) % 13 - 4)
        K, V = rand(t, 1, heads, dim, std=std), rand(t + 999, 1, heads, dim, std=1 / std)
        nv.kv_append(cache, K, V, table, ints([t + 1]))
        want.append((K, V), table, [(0, 1, t + 1)])
    got = dref.Cache(cache)
    for a, b in zip(got.codes + got.byte, want.codes + want.byte):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_append_of_values_that_are_not_finite(bad):
    heads, dim = 2, 32
    table, pages = layout(1, [130])
    cache = nv.kv_cache(pages, heads, dim)
    fill(cache, 3)
    want = dref.Cache(cache)
    K, V = rand(1, 130, heads, dim), rand(2, 130, heads, dim)
    K[70, 1, 5] = bad
    for lo, hi in ((0, 100), (100, 130)):  # the second call adds to the block that is NaN by then
        nv.kv_append(cache, K[lo:hi], V[lo:hi], table, ints([hi]), ints([0, hi - lo]))
        want.append((K[lo:hi], V[lo:hi]), table, [(0, hi - lo, hi)])
    got = dref.Cache(cache)
    for a, b in zip(got.codes, want.codes):
        assert torch.equal(torch.nan_to_num(a, 1e9), torch.nan_to_num(b, 1e9))
    assert all(torch.equal(a, b) for a, b in zip(got.byte, want.byte))
    page = int(table[0, 1])
    assert u8(cache.k_scales)[page].tolist()[1] == 255 and (u8(cache.k)[page, 1] == 0x7F).all()
    # a new sequence that begins in the block
    nv.kv_append(cache, K[:1], V[:1], table[:, 1:], ints([1]))
    assert u8(cache.k_scales)[page].tolist()[1] != 255


def test_append_leaves_out_what_has_no_place():
    heads, dim = 1, 16
    cache = nv.kv_cache(4, heads, dim)
    fill(cache, 1)
    before = [t.clone() for t in cache]
    K = rand(1, 200, heads, dim)
    for page in (-1, 4, 1 << 30, -(1 << 31)):
        nv.kv_append(cache, K, K, torch.full((1, 4), page, dtype=torch.int32, device="cuda"), ints([200]), ints([0, 200]))
    nv.kv_append(cache, K, K, ints([[0, 1]]), ints([0]), ints([0, 0]))
    nv.kv_append(cache, K, K, ints([[0, 1]]), ints([-5]), ints([0, 100]))
    assert all(torch.equal(u8(a), u8(b)) for a, b in zip(before, cache))
    # more tokens than the table's row holds, and more than the sequence has: the last ones, and only where there is room
    want = dref.Cache(cache)
    want.append((K, K), ints([[2]]), [(0, 200, 64)])
    nv.kv_append(cache, K, K, ints([[2]]), ints([64]), ints([0, 200]))
    got = dref.Cache(cache)
    assert torch.equal(got.codes[0], want.codes[0]) and torch.equal(got.codes[1], want.codes[1])


# ---------------------------------------------------------------------------------------- attention

SPLIT = 70  # blocks of a table that few rows take over several work-groups


def ready(seed, lengths, heads, dim, extra=2, width=None):
    table, pages = layout(seed, lengths, extra, width)
    cache = nv.kv_cache(pages, heads, dim)
    fill(cache, seed)
    return cache, table


ATTENTION = [
    # lengths, new tokens, heads, kv heads, dim
    ([1], [1], 1, 1, 16),
    ([64], [1], 4, 1, 64),
    ([5, 63, 64, 65, 128, 1000], [1] * 6, 8, 2, 128),
    ([0, 1, 4000], [1] * 3, 5, 1, 96),
    ([700, 2], [1, 1], 40, 2, 80),
    ([300], [1], 68, 1, 128),
    ([513, 90], [1, 1], 6, 3, 256),
    ([200, 31], [1, 1], 3, 3, 192),
    ([70, 500, 9, 0, 33, 129], [3, 6, 9, 0, 1, 4], 14, 2, 64),
    ([100, 3], [20, 5], 8, 1, 48),
    ([400, 40, 64], [100, 40, 64], 4, 2, 128),
    ([333], [333], 2, 1, 144),
    ([257, 600], [257, 77], 3, 1, 256),
]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim", ATTENTION)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_matches_binary64(lengths, new, heads, kv_heads, dim, causal, width):
    say(f"attention {lengths} {new} {heads} {kv_heads} {dim} {causal} {width}")
    cache, table = ready(11, lengths, kv_heads, dim, width=width)
    sp = spans(lengths, new, first=1)
    rows = sum(new) + 3
    for std in (0.05, 2.0):  # even weights, and a few tokens that take all
        q = rand(3, rows, heads + 3, dim, std=std)[:, 1:heads + 1]
        out = torch.full((rows, heads, dim), 7.0, dtype=BF16, device="cuda")
        args = (q, cache, table, ints(lengths), starts_of(sp))
        assert nv.attention(*args, causal=causal, out=out) is out
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, causal)
        want[0], want[-2:] = 7.0, 7.0  # rows of no sequence
        check(out, want, err)
        if all(n == 1 for n in new):
            alone = nv.attention(q[1:-2], cache, table, ints(lengths), causal=causal)
            check(alone, want[1:-2], err[1:-2])
    o = nv.attention(*args, scale=-0.3, causal=causal)
    want, err = dref.attention(q, cache, table, sp, -0.3, causal)
    check(o[1:-2], want[1:-2], err[1:-2])


# rows over the waves of a work-group (many rows), for each head size compiled for; and a mixture of prompts and tokens
LONG = [([2300, 190], [2300, 190], 16, 8, 64), ([4200], [2100], 32, 8, 128), ([1100, 5, 900], [1000, 1, 900], 24, 12, 192),
        ([1500, 64, 3], [1500, 1, 1], 16, 16, 256), ([3000] + [100] * 20, [2000] + [1] * 20, 16, 8, 112)]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim", LONG)
def test_attention_of_prompts(lengths, new, heads, kv_heads, dim):
    say(f"prompts {lengths} {new} {heads} {kv_heads} {dim}")
    cache, table = ready(5, lengths, kv_heads, dim)
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    for causal in (True, False):
        o = nv.attention(q, cache, table, ints(lengths), starts_of(sp), causal=causal)
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, causal)
        check(o, want, err)


# Prompts and single tokens in a call: pieces of few rows among those of many, whole and, where the prompts are few, in parts
MIXED = [([2500, 800, 900, 0, 700, 1], [2200, 1, 3, 1, 600, 1], 16, 4, 128), ([1800, 640, 130], [700, 4, 1], 8, 1, 64),
         ([500, 3000, 64], [300, 1, 1], 4, 2, 80), ([400, 1000], [300, 2], 3, 1, 256), ([700, 800, 900], [129, 65, 1], 2, 2, 192)]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim", MIXED)
@pytest.mark.parametrize("width", [None, 200])
def test_attention_of_prompts_and_single_tokens(lengths, new, heads, kv_heads, dim, width):
    say(f"mixed {lengths} {new} {heads} {kv_heads} {dim} {width}")
    table, pages = layout(6, lengths, width=width)
    cache = nv.kv_cache(pages, kv_heads, dim)
    fill(cache, 6)
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    args = (q, cache, table, ints(lengths), starts_of(sp))
    for causal in (True, False):
        o = nv.attention(*args, causal=causal)
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, causal)
        check(o, want, err)
        assert torch.equal(nv.attention(*args, causal=causal), o)
    u8(cache.v_scales)[int(table[1, 3 % (-(-lengths[1] // 64))]), 0] = 255
    table[1, 0] = -1
    want, err = dref.attention(q, cache, table, sp, dim ** -0.5, True)
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    check(nv.attention(*args), want, err)


# Some tens to hundreds of rows: rows over the waves with the blocks in parts, for each head size compiled for, 64 and 128
# rows a work-group, tables far wider than the sequences
PARTS = [([3000], [40], 4, 1, 128), ([2100, 65, 5000], [12, 9, 20], 8, 2, 64), ([1999], [300], 6, 3, 80), ([4444, 10], [33, 10], 3, 1, 256),
         ([2500, 0, 700], [50, 0, 50], 5, 1, 176), ([6000], [70], 17, 1, 48)]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim", PARTS)
def test_attention_in_parts(lengths, new, heads, kv_heads, dim):
    say(f"parts {lengths} {new} {heads} {kv_heads} {dim}")
    table, pages = layout(6, lengths, width=160)
    cache = nv.kv_cache(pages, kv_heads, dim)
    fill(cache, 6)
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    args = (q, cache, table, ints(lengths), starts_of(sp))
    ws = torch.full((nv.attention_workspace_bytes(sum(new), len(new), table.shape[1], heads, kv_heads, dim),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    for causal in (True, False):
        o = nv.attention(*args, causal=causal, workspace=ws)
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, causal)
        check(o, want, err)
        assert torch.equal(nv.attention(*args, causal=causal), o)
    u8(cache.v_scales)[int(table[0, 20]), 0] = 255
    u8(cache.v)[int(table[0, 20]), 0] = 0x7F
    table[0, 5] = -1
    o = nv.attention(*args)
    want, err = dref.attention(q, cache, table, sp, dim ** -0.5, True)
    assert torch.isnan(want).any()
    check(o, want, err)


# Tiles that end inside a work-group's share, and shares of several tiles: few and many sequences
@pytest.mark.parametrize("seqs", [2, 5, 16, 33, 64, 65, 300])
def test_attention_shares(seqs):
    """Few rows of sequences of very different lengths, over tables that take them so."""
    lengths = [1 + (i * 977) % 2900 for i in range(seqs)]
    new = [1 + (i * 5) % 4 for i in range(seqs)]
    lengths = [max(a, b) for a, b in zip(lengths, new)]
    cache, table = ready(8, lengths, 1, 64, width=SPLIT)
    sp = spans(lengths, new)
    q = rand(3, sum(new), 7, 64)
    o = nv.attention(q, cache, table, ints(lengths), starts_of(sp))
    want, err = dref.attention(q, cache, table, sp, 64 ** -0.5, True)
    check(o, want, err)


# Tiles of 32 rows, which a table wide enough takes, for each head size compiled for: full tiles and parts of one, blocks of NaN
WIDE = [([900, 64, 2001, 7], [5, 7, 8, 1], 16, 4, 64), ([1300, 129], [8, 9], 24, 8, 128), ([700, 1900, 63], [3, 3, 2], 8, 1, 80),
        ([2500, 11, 0, 640], [4, 11, 0, 5], 10, 2, 192), ([513, 300], [17, 30], 1, 1, 48), ([800, 1000], [20, 31], 2, 2, 160)]


@pytest.mark.parametrize("lengths,new,heads,kv_heads,dim", WIDE)
def test_attention_of_wide_tables(lengths, new, heads, kv_heads, dim):
    say(f"wide {lengths} {new} {heads} {kv_heads} {dim}")
    table, pages = layout(6, lengths, width=40 * 512 // kv_heads // len(lengths) + 1)
    cache = nv.kv_cache(pages, kv_heads, dim)
    fill(cache, 6)
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    args = (q, cache, table, ints(lengths), starts_of(sp))
    for causal in (True, False):
        o = nv.attention(*args, causal=causal)
        want, err = dref.attention(q, cache, table, sp, dim ** -0.5, causal)
        check(o, want, err)
        assert torch.equal(nv.attention(*args, causal=causal), o)
    u8(cache.k_scales)[int(table[0, 5]), 0] = 255
    table[0, 2] = -1
    want, err = dref.attention(q, cache, table, sp, dim ** -0.5, True)
    assert torch.isnan(want).any()
    check(nv.attention(*args), want, err)


@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_of_many_sequences(width):
    """More sequences than a wave has lanes, of very different lengths."""
    lengths = [(i * 37) % 150 for i in range(200)] + [3000]
    cache, table = ready(9, lengths, 2, 32, width=width)
    q = rand(1, len(lengths), 4, 32)
    o = nv.attention(q, cache, table, ints(lengths))
    want, err = dref.attention(q, cache, table, spans(lengths, [1] * len(lengths)), 32 ** -0.5, True)
    check(o, want, err)
    new = [(i * 11) % 4 for i in range(201)]
    lengths = [max(a, b) for a, b in zip(lengths, new)]
    sp = spans(lengths, new)
    q = rand(2, sum(new), 4, 32)
    cache, table = ready(10, lengths, 2, 32, width=width)
    o = nv.attention(q, cache, table, ints(lengths), starts_of(sp))
    want, err = dref.attention(q, cache, table, sp, 32 ** -0.5, True)
    check(o, want, err)


@pytest.mark.parametrize("new", [1, 30, 900])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_does_not_look_behind_the_end(new, width):
    """Bytes behind a sequence's end, and pages of no sequence, may be NaN."""
    lengths, heads, dim = [1000 - 11], 8, 128
    cache, table = ready(2, lengths, 8, dim, width=width)
    sp = spans(lengths, [new])
    q = rand(3, new, 16, dim)
    args = (q, cache, table, ints(lengths), starts_of(sp))
    o = nv.attention(*args)
    page = int(table[0, 15])
    u8(cache.k)[page, :, lengths[0] % 64:] = 0x7F
    u8(cache.v)[page, :, :, lengths[0] % 64:] = 0xFF
    mine = set(table[0, :16].tolist())
    for other in set(range(cache.k.shape[0])) - mine:
        u8(cache.k)[other] = 0x7F
        u8(cache.k_scales)[other] = 255
    assert torch.equal(nv.attention(*args), o)


@pytest.mark.parametrize("heads,new", [(8, [1, 1]), (8, [20, 9]), (16, [700, 700])])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_of_blocks_of_nan(heads, new, width):
    """Rows that see a block of NaN are NaN, the others are what they are without it."""
    lengths, dim = [777, 700], 128
    cache, table = ready(2, lengths, 8, dim, width=width)
    u8(cache.k_scales)[int(table[0, 11]), 1] = 255
    u8(cache.k)[int(table[0, 11]), 1] = 0x7F
    u8(cache.v_scales)[int(table[1, 10]), 0] = 255  # its last block
    u8(cache.v)[int(table[1, 10]), 0] = 0x7F
    sp = spans(lengths, new)
    q = rand(3, sum(new), heads, dim)
    o = nv.attention(q, cache, table, ints(lengths), starts_of(sp))
    want, err = dref.attention(q, cache, table, sp, dim ** -0.5, True)
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    check(o, want, err)


@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_of_queries_that_are_not_finite(width):
    cache, table = ready(2, [200, 200], 1, 64, width=width)
    q = rand(3, 2, 4, 64)
    clean = nv.attention(q, cache, table, ints([200, 200]))
    q[1, 2, 5] = float("nan")
    o = nv.attention(q, cache, table, ints([200, 200]))
    assert torch.isnan(o[1, 2]).all()
    o[1, 2] = clean[1, 2]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("new", [1, 5, 600])
@pytest.mark.parametrize("width", [None, SPLIT])
def test_attention_of_sequences_without_tokens(new, width):
    """Lengths of zero, more new tokens than tokens, pages outside the cache, tables of nothing: zeros, or what is there."""
    cache, table = ready(2, [640, 640], 8, 128, width=width)
    q = rand(3, 2 * new, 16, 128)
    starts = ints([0, new, 2 * new])
    assert (nv.attention(q, cache, table, ints([0, -3]), starts) == 0).all()
    none = torch.full_like(table, -1)
    assert (nv.attention(q, cache, none, ints([640, 640]), starts) == 0).all()
    for hole in (0, 5, 9):
        t = table.clone()
        t[0, hole] = 1 << 29
        sp = spans([640, 3], [new, new])
        o = nv.attention(q, cache, t, ints([640, 3]), starts)
        want, err = dref.attention(q, cache, t, sp, 128 ** -0.5, True)
        check(o, want, err)
    # counts as what the table holds, pages outside the cache left out
    long = nv.attention(q, cache, table, ints([1 << 30, 640]), starts, causal=False)
    whole = nv.attention(q, cache, table, ints([640, 640]), starts, causal=False)
    if width is None:
        assert torch.equal(long, whole)
    else:  # (other shares, another order of its sums: twice what one order's bound allows, and roundings of the same value)
        _, err = dref.attention(q, cache, table, spans([640, 640], [new, new]), 128 ** -0.5, False)
        assert ((long.double() - whole.double()).abs() <= 2 * err + 2 * whole.double().abs() * 2.0 ** -8).all()


def test_attention_is_reproducible_and_takes_a_workspace():
    lengths = [3000, 10, 777, 64]
    cache, table = ready(4, lengths, 2, 128)
    q = rand(1, 4, 8, 128)
    lens = ints(lengths)
    o = nv.attention(q, cache, table, lens)
    need = nv.attention_workspace_bytes(4, 4, table.shape[1], 8, 2, 128)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere
    for _ in range(3):
        assert torch.equal(nv.attention(q, cache, table, lens, workspace=ws), o)
    with pytest.raises(nv.NVFP4Error):
        nv.attention(q, cache, table, lens, workspace=ws[:-1].clone())


def test_attention_with_large_offsets():
    """A cache of more than 2^32 bytes of keys."""
    heads, dim = 8, 256
    pages = (1 << 32) // (heads * 64 * dim) + 40
    cache = nv.kv_cache(pages, heads, dim)
    lengths = [300, 90]
    table = ints([[pages - 1, 3, pages - 7, pages // 2, pages - 2], [pages - 5, pages - 3, 0, 0, 0]])
    K, V = rand(1, 390, heads, dim), rand(2, 390, heads, dim)
    nv.kv_append(cache, K, V, table, ints(lengths), ints([0, 300, 390]))
    q = rand(3, 2, 16, dim)
    o = nv.attention(q, cache, table, ints(lengths))
    want, err = [], []
    small = nv.kv_cache(8, heads, dim)
    for a, b in zip(small, cache):  # the same pages in a small cache
        for i, page in enumerate([pages - 1, 3, pages - 7, pages // 2, pages - 2, pages - 5, pages - 3]):
            u8(a)[i] = u8(b)[page]
    t = ints([[0, 1, 2, 3, 4], [5, 6, 7, 7, 7]])
    want, err = dref.attention(q, small, t, spans(lengths, [1, 1]), dim ** -0.5, True)
    check(o, want, err)


# -------------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("width", [None, SPLIT])
def test_stream_and_graph(width):
    """The three calls on a stream of their own, and captured and replayed as a decoding step with growing lengths."""
    heads, kv_heads, dim, seqs = 8, 2, 64, 3
    lengths = [60, 126, 0]
    table, pages = layout(1, [400] * seqs, width=width)
    caches = [nv.kv_cache(pages, kv_heads, dim) for _ in range(2)]
    for c in caches:
        fill(c, 5)
    qkv = rand(1, seqs, heads + 2 * kv_heads, dim)
    lens = ints(lengths)
    pos = torch.zeros(seqs, dtype=torch.int64, device="cuda")
    ws = torch.empty(nv.attention_workspace_bytes(seqs, seqs, table.shape[1], heads, kv_heads, dim), dtype=torch.uint8, device="cuda")
    out = torch.empty(seqs, heads, dim, dtype=BF16, device="cuda")

    def step(x, cache, stream=None):
        nv.rotary(x[:, :heads + kv_heads], pos, out=x[:, :heads + kv_heads], stream=stream)
        nv.kv_append(cache, x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], table, lens, stream=stream)
        return nv.attention(x[:, :heads], cache, table, lens, workspace=ws, out=out, stream=stream)

    work = qkv.clone()
    side = torch.cuda.Stream()
    lens += 1
    side.wait_stream(torch.cuda.current_stream())  # for the lengths too
    step(work, caches[0], side)
    torch.cuda.current_stream().wait_stream(side)
    work.copy_(qkv)
    expect = step(work, caches[1]).clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(work, caches[0])
    for i in range(5):
        x = rand(20 + i, *qkv.shape)
        lens += 1
        pos += 3
        work.copy_(x)
        expect = step(work, caches[1]).clone()
        work.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect)
        assert all(torch.equal(u8(a), u8(b)) for a, b in zip(*caches))
        torch.randn(1000, device="cuda").sum().item()


def test_refusals():
    x = rand(1, 4, 2, 64)
    pos = torch.arange(4, device="cuda")
    E = nv.NVFP4Error
    for kw in (dict(sections=(33,)), dict(sections=(0,)), dict(sections=(-1,)), dict(sections=(8, 8)), dict(base=0.0),
               dict(base=float("inf")), dict(out=x[:, :1]), dict(out=x.float()), dict(out=x.transpose(0, 1)),
               dict(out=torch.empty(4, 2, 128, dtype=BF16, device="cuda")[..., :64])):
        with pytest.raises(E):
            nv.rotary(x, pos, **kw)
    for a in ((x[0], pos), (x.half(), pos), (x, pos[:3]), (x, pos.float()), (x, pos.cpu()), (x[..., ::2], pos),
              (x, torch.zeros(5, 4, dtype=torch.int64, device="cuda")), (x.expand(4, 2, 64)[:, :1].expand(4, 2, 64), pos)):
        with pytest.raises(E):
            nv.rotary(*a)
    cache, table = ready(1, [100, 70], 2, 64)
    lens, K = ints([100, 70]), rand(2, 2, 2, 64)
    good = (cache, K, K, table, lens)
    for at, bad in ((0, cache[:3]), (0, (cache[2],) + tuple(cache[1:])), (0, tuple(t.cpu() for t in cache)),
                    (0, nv.kv_cache(3, 2, 32)), (0, nv.kv_cache(3, 1, 64)), (1, K.half()), (1, K[:1]), (2, K.float()),
                    (2, K[:, :1]), (3, table.long()), (3, table[0]), (3, table[:1]), (3, table[:, :0]), (4, lens.long()),
                    (4, lens[:1]), (4, lens.cpu())):
        args = list(good)
        args[at] = bad
        with pytest.raises(E):
            nv.kv_append(*args)
    q = rand(3, 2, 4, 64)
    for bad in (q[:, :3], q.float(), q[..., :32], q[:1], q[..., ::2], q[:, :0]):
        with pytest.raises(E):
            nv.attention(bad, cache, table, lens)
    for kw in (dict(starts=ints([0, 1])), dict(starts=torch.tensor([0, 1, 2], device="cuda")), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(out=q.float()), dict(out=q[:1])):
        with pytest.raises(E):
            nv.attention(q, cache, table, lens, **kw)
    with torch.enable_grad():
        with pytest.raises(E):
            nv.attention(q.clone().requires_grad_(), cache, table, lens)
        with pytest.raises(E):
            nv.rotary(x.clone().requires_grad_(), pos)
        with pytest.raises(E):
            nv.kv_append(cache, K.clone().requires_grad_(), K, table, lens)
    for bad in (dict(dim=24), dict(dim=272), dict(kv_heads=0), dict(pages=-1)):
        with pytest.raises(E):
            nv.kv_cache(**{**dict(pages=1, kv_heads=1, dim=64), **bad})
    assert nv.attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 4, 64)
