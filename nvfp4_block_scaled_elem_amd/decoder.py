"""A decoder layer's operators beside its products: rotary positions, a paged cache of keys and values in 8 bits and
attention over it, and a layer of experts (C ABI: ``include/nvfp4.h``). Marshalling only, like the rest of the binding.

    rotary(qk, positions, out=qk)                                # qk: the query and key heads of a product, in place
    cache = kv_cache(pages, kv_heads, dim)                       # codes and scales, all zeros
    kv_append(cache, K, V, table, lengths)                       # a token of each sequence, or, with starts, several
    O = attention(Q, cache, table, lengths)                      # of the same tokens' queries
    Y = moe(X, logits, up, down, top_k)                          # up, down: stacked (codes, scales, alphas) of the experts

Streams, scratch and autograd are as for the layer operators (``layer.py``): outputs are allocated on the call's stream, and
where grad mode is on an operand that requires a gradient is refused. ``rotary``'s gradient is ``rotary`` with
``inverse=True``; the cache is for serving, and its attention has no gradient, nor has the experts' layer for few tokens.

Sequences: ``table`` [seqs, width] int32 holds the pages of each, 64 tokens a page; ``lengths`` [seqs] int32 their tokens, those
of the call among them; with ``starts`` [seqs + 1] int32 the rows starts[s] .. starts[s + 1] - 1 of the operands are the last
tokens of sequence s, without it row s is the one new token of sequence s. They are device data and not looked at by
the host: pages outside the cache are left out, rows of no sequence are neither read nor written. The pages that ``kv_append``
writes to must belong to one sequence each; pages that are only read may be shared.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import struct

import torch

from . import DTYPES, NVFP4Error, _check, lib
from .layer import ACTIVATIONS, _no_graph, _output, _ptr, _rows, _run, _space

PAGE = 64  # tokens of a page
KVCache = collections.namedtuple("KVCache", "k v k_scales v_scales")
_CODES = (torch.float8_e4m3fn, torch.uint8)
_SCALES = (torch.float8_e8m0fnu, torch.uint8)
_AXES = 4
_Sections = ctypes.c_int * _AXES
_FORMATS = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_double: "d", ctypes.c_size_t: "N",
            _Sections: f"{_AXES}i"}


def _packer(args):
    """A function that lays out the values of a structure's fields (null: 0) as C does, in bytes: a third of the time that
    making the structure takes, which for single tokens is a good part of a call."""
    form = struct.Struct("@" + "".join(_FORMATS[t] for _, t in args._fields_) + "0q")

    def pack(*values):
        try:
            return form.pack(*values)
        except struct.error as e:
            raise NVFP4Error(f"an argument is out of range: {e}") from None

    return pack


class _RotaryArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("xs", ctypes.c_int64), ("xh", ctypes.c_int64), ("y", ctypes.c_void_p),
        ("ys", ctypes.c_int64), ("yh", ctypes.c_int64), ("dtype", ctypes.c_int), ("tokens", ctypes.c_int64),
        ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("positions", ctypes.c_void_p), ("positions64", ctypes.c_int),
        ("axes", ctypes.c_int), ("sections", _Sections), ("base", ctypes.c_double), ("inverse", ctypes.c_int),
        ("stream", ctypes.c_void_p),
    ]


_rotary_args = _packer(_RotaryArgs)


class _Cache(ctypes.Structure):
    _fields_ = [
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int), ("dim", ctypes.c_int),
    ]


class _Sequences(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p), ("ldt", ctypes.c_int64), ("lengths", ctypes.c_void_p), ("starts", ctypes.c_void_p),
        ("seqs", ctypes.c_int), ("width", ctypes.c_int),
    ]


_cache_args, _sequences_args = _packer(_Cache), _packer(_Sequences)


def _heads(t, name, dtypes, dev=None, shape=None):
    """Checks a [tokens, heads, dim] operand with unit column stride; returns its token and head strides."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3 or not t.is_cuda or t.dtype not in dtypes:
        raise NVFP4Error(f"{name} must be a [tokens, heads, dim] CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if dev is not None and t.device != dev:
        raise NVFP4Error(f"{name} must be on {dev}")
    tokens, heads, dim = t.shape
    if shape is not None and t.shape != shape:
        raise NVFP4Error(f"{name} must be {list(shape)}, got {[tokens, heads, dim]}")
    st, sh, sc = t.stride()
    if (sc != 1 and dim > 1) or (heads > 1 and sh < dim) or (tokens > 1 and st < dim):
        raise NVFP4Error(f"{name} must have unit column stride and rows that do not overlap")
    return st, sh


def _apart(out, t, name):
    """Refuses a contiguous output that shares memory with an operand of its shape and is not the operand itself: rows would be
    read after others were written over them."""
    a, b, size = t.data_ptr(), out.data_ptr(), t.element_size()
    span = 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    if a >= b + out.numel() * size or b >= a + span * size or not out.numel() or (a == b and t.is_contiguous()):
        return
    begin = torch.zeros((), dtype=torch.int64, device="cpu")  # of each row, from the operand's first
    for n, s in zip(t.shape[:-1], t.stride()[:-1]):
        begin = begin[..., None] + s * torch.arange(n, device="cpu")
    begin = a + begin * size
    if ((begin < b + out.numel() * size) & (begin + t.shape[-1] * size > b)).any():
        raise NVFP4Error(f"out may be {name} itself (contiguous), but may not share memory with it otherwise")


def rotary(x: torch.Tensor, positions: torch.Tensor, *, sections=None, base: float = 10000.0, inverse: bool = False,
           out=None, stream=None) -> torch.Tensor:
    """Rotary positions of ``x`` ([tokens, heads, dim] bf16 or fp32): with R = 2 * sum(sections) <= dim, columns j and j +
    R/2 are turned by the angle positions[axis(j)] * base^(-2j/R), columns from R on pass. ``positions`` is [tokens] or
    [axes, tokens] (up to four axes) int32 or int64, contiguous; ``sections`` the number of consecutive pairs of each axis
    (None: one axis, all dim // 2 pairs). Angles are binary64, off by some 2^-51 of themselves: below what binary32
    holds of a turn for positions to 2^27. ``inverse`` turns back: the gradient. Returns y, in ``out`` if given: x itself (in
    place), or a contiguous tensor apart from it."""
    xs, xh = _heads(x, "x", DTYPES)
    tokens, heads, dim = x.shape
    dev = x.device
    if (not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64) or positions.device != dev
            or positions.dim() not in (1, 2) or positions.shape[-1] != tokens or not positions.is_contiguous()):
        raise NVFP4Error(f"positions must be a contiguous [{tokens}] or [axes, {tokens}] int32 or int64 tensor on {dev}")
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    if sections is None:
        sections = (dim // 2,)
        if dim % 2:
            raise NVFP4Error("an odd dim needs sections")
    if not 1 <= axes <= _AXES or len(sections) != axes:
        raise NVFP4Error(f"sections must give the pairs of each of {axes} axes (at most {_AXES})")
    if min(sections) < 0 or not 0 < 2 * sum(sections) <= dim:
        raise NVFP4Error(f"the sections must be of one to {dim // 2} pairs together")
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.shape != x.shape or out.dtype != x.dtype or out.device != dev:
            raise NVFP4Error(f"out must be a {[tokens, heads, dim]} {x.dtype} tensor on {dev}")
        if out.data_ptr() == x.data_ptr():
            if out.stride() != x.stride():
                raise NVFP4Error("out may be x itself, not another view of its memory")
            if tokens > 1 and heads > 1 and xs < (heads - 1) * xh + dim and xh < (tokens - 1) * xs + dim:
                raise NVFP4Error("in place, the rows of x may not overlap")
        elif not out.is_contiguous():
            raise NVFP4Error("out must be contiguous or x itself")
        else:
            _apart(out, x, "x")
    _no_graph(x, out)

    def call(st):
        y = torch.empty_like(x, memory_format=torch.contiguous_format) if out is None else out
        ys, yh, _ = y.stride()
        a = _rotary_args(x.data_ptr(), xs, xh, y.data_ptr(), ys, yh, DTYPES[x.dtype], tokens, heads, dim, positions.data_ptr(),
                         int(positions.dtype == torch.int64), axes, *sections, *(0,) * (_AXES - axes), base, int(inverse), st)
        _check(lib().nvfp4_rotary(a))
        return y

    return _run(dev, stream, call)


def kv_cache(pages: int, kv_heads: int, dim: int, device="cuda") -> KVCache:
    """An empty cache: k [pages, kv_heads, 64, dim] and v [pages, kv_heads, dim, 64] E4M3 codes (zeros), k_scales and
    v_scales [pages, kv_heads] E8M0, one power of two per page and head. dim % 16 == 0, dim <= 256."""
    if pages < 0 or kv_heads <= 0 or dim <= 0 or dim % 16 or dim > 256:
        raise NVFP4Error("a cache has at least one head, and a dim that is a multiple of 16 up to 256")
    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=device)
    return KVCache(zeros(pages, kv_heads, PAGE, dim).view(_CODES[0]), zeros(pages, kv_heads, dim, PAGE).view(_CODES[0]),
                   zeros(pages, kv_heads).view(_SCALES[0]), zeros(pages, kv_heads).view(_SCALES[0]))


def _cache(cache, dev):
    """Checks a cache; returns its C form, heads and dim."""
    if not isinstance(cache, (tuple, list)) or len(cache) != 4:
        raise NVFP4Error("the cache must be (k, v, k_scales, v_scales), as kv_cache makes it")
    k, v, ks, vs = cache
    at = dev.index
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and isinstance(ks, torch.Tensor) and isinstance(vs, torch.Tensor)
            and k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == at and k.dtype in _CODES and v.dtype in _CODES
            and ks.dtype in _SCALES and vs.dtype in _SCALES and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous()):
        raise NVFP4Error(f"the cache's codes must be contiguous E4M3 and its scales contiguous E8M0 tensors on {dev}")
    if k.dim() != 4 or k.shape[2] != PAGE or not k.shape[1]:
        raise NVFP4Error(f"the cache's k must be [pages, kv_heads, {PAGE}, dim] of at least one head")
    pages, heads, _, dim = k.shape
    if v.shape != (pages, heads, dim, PAGE) or ks.shape != (pages, heads) or vs.shape != (pages, heads):
        raise NVFP4Error(f"the cache's v must be {[pages, heads, dim, PAGE]} and its scales {[pages, heads]}")
    return _cache_args(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, heads, dim), heads, dim


def _ints(t, name, n, dev):
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.get_device() != dev.index or t.shape != (n,)
            or not t.is_contiguous()):
        raise NVFP4Error(f"{name} must be a contiguous [{n}] int32 tensor on {dev}")


def _sequences(table, lengths, starts, tokens, dev):
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.dtype != torch.int32 or table.get_device() != dev.index:
        raise NVFP4Error(f"table must be a [seqs, width] int32 tensor on {dev}")
    seqs, width = table.shape
    ldt, unit = table.stride()
    if (width > 1 and unit != 1) or (seqs > 1 and ldt < width):
        raise NVFP4Error("table must have unit column stride and rows that do not overlap")
    _ints(lengths, "lengths", seqs, dev)
    if starts is not None:
        _ints(starts, "starts", seqs + 1, dev)
    elif tokens != seqs:
        raise NVFP4Error(f"without starts there is one token for each of the {seqs} sequences, got {tokens}")
    if tokens and seqs and not width:
        raise NVFP4Error("the table has no columns")
    return _sequences_args(table.data_ptr(), ldt, lengths.data_ptr(), _ptr(starts) or 0, seqs, width), seqs, width


def kv_append(cache, K: torch.Tensor, V: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, starts=None, *,
              stream=None):
    """Writes the keys and values ``K`` and ``V`` ([tokens, kv_heads, dim], bf16 or fp32) of the sequences' last tokens
    into the cache, and returns it. Per block of 64 tokens and head the scale is the smallest power of two under which
    nothing saturates; where a block already holds tokens of the sequence it does not fall, and their codes are
    rounded to the new one if it grows. A NaN, an infinity or a magnitude of 248 * 2^120 and more makes its block one of
    NaNs."""
    kt, kh = _heads(K, "K", DTYPES)
    dev = K.device
    vt, vh = _heads(V, "V", (K.dtype,), dev, K.shape)
    c, heads, dim = _cache(cache, dev)
    tokens = K.shape[0]
    if K.shape[1:] != (heads, dim):
        raise NVFP4Error(f"K must be [tokens, {heads}, {dim}], as the cache")
    q, _, _ = _sequences(table, lengths, starts, tokens, dev)
    _no_graph(K, V)

    def call(st):
        _check(lib().nvfp4_kv_append(c, q, K.data_ptr(), kt, kh, V.data_ptr(), vt, vh,
                                     DTYPES[K.dtype], tokens, st))
        return cache

    return _run(dev, stream, call)


@functools.lru_cache(maxsize=1024)  # (a function of the sizes alone; asked for by every call)
def attention_workspace_bytes(tokens: int, seqs: int, width: int, heads: int, kv_heads: int, dim: int) -> int:
    return int(lib().nvfp4_attention_workspace_bytes(tokens, seqs, width, heads, kv_heads, dim))


def attention(Q: torch.Tensor, cache, table: torch.Tensor, lengths: torch.Tensor, starts=None, *, scale=None,
              causal: bool = True, out=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of ``Q`` ([tokens, heads, dim] bf16; heads a multiple of the cache's) over the cache: softmax(scale * Q
    K^T) V over the tokens that a row sees, [tokens, heads, dim] bf16, in ``out`` if given (contiguous; it may be Q).
    ``causal``: row i of a sequence's n sees its first length - n + i + 1 tokens; else all of them (the cached states of an
    encoder). ``scale`` None: dim^-0.5. A row that sees no token gives zeros; one that sees a block written with a NaN or an infinity, or
    any token where its query holds one, gives NaN. Prompts and single tokens may come in one call."""
    qt, qh = _heads(Q, "Q", (torch.bfloat16,))
    dev = Q.device
    c, kv_heads, dim = _cache(cache, dev)
    tokens, heads, qdim = Q.shape
    if qdim != dim or heads % kv_heads or not heads:
        raise NVFP4Error(f"Q must be [tokens, heads, {dim}] with a multiple of {kv_heads} heads")
    q, seqs, width = _sequences(table, lengths, starts, tokens, dev)
    if out is not None and (not isinstance(out, torch.Tensor) or out.shape != Q.shape or out.dtype != torch.bfloat16
                            or out.device != dev or not out.is_contiguous()):
        raise NVFP4Error(f"out must be a contiguous {list(Q.shape)} bf16 tensor on {dev}")
    if out is not None:
        _apart(out, Q, "Q")
    _no_graph(Q, out)

    def call(st):
        O = torch.empty_like(Q, memory_format=torch.contiguous_format) if out is None else out
        ws, nbytes = _space(workspace, attention_workspace_bytes(tokens, seqs, width, heads, kv_heads, dim), dev)
        _check(lib().nvfp4_attention(c, q, Q.data_ptr(), qt, qh, heads, tokens,
                                     dim ** -0.5 if scale is None else scale, int(causal), O.data_ptr(), _ptr(ws), nbytes, st))
        return O

    return _run(dev, stream, call)


class _MoeArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("logits", ctypes.c_void_p), ("ldl", ctypes.c_int64),
        ("logits_dtype", ctypes.c_int), ("tokens", ctypes.c_int64), ("width", ctypes.c_int64), ("inner", ctypes.c_int64),
        ("experts", ctypes.c_int), ("top_k", ctypes.c_int), ("up_codes", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
        ("up_alpha", ctypes.c_void_p), ("down_codes", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
        ("down_alpha", ctypes.c_void_p), ("activation", ctypes.c_int), ("gated", ctypes.c_int), ("scoring", ctypes.c_int),
        ("normalize", ctypes.c_int), ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("y", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
    ]


_moe_args = _packer(_MoeArgs)


SCORING = {"softmax": 0, "sigmoid": 1}  # enum nvfp4_scoring


def _experts(W, name, experts, dev, rows=None, cols=None):
    """Checks stacked NVFP4 weights (codes [experts, rows, cols/2], scales [experts, rows, cols/16], alphas [experts]);
    returns (rows, cols)."""
    if not isinstance(W, (tuple, list)) or len(W) != 3 or not all(isinstance(t, torch.Tensor) for t in W):
        raise NVFP4Error(f"{name} must be (codes, scales, alphas)")
    codes, scales, alphas = W
    if codes.dim() != 3 or codes.shape[0] != experts or codes.shape[2] % 8:
        raise NVFP4Error(f"{name}'s codes must be [{experts}, rows, cols/2] with cols % 16 == 0")
    n, k = codes.shape[1], 2 * codes.shape[2]
    if (rows is not None and n != rows) or (cols is not None and k != cols):
        raise NVFP4Error(f"{name} must be {experts} matrices of {[rows, cols]}, got {[n, k]}")
    if scales.shape != (experts, n, k // 16) or alphas.shape != (experts,):
        raise NVFP4Error(f"{name}'s scales must be {[experts, n, k // 16]} and its alphas [{experts}]")
    if (codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or alphas.dtype != torch.float32 or codes.device != dev
            or scales.device != dev or alphas.device != dev or not codes.is_contiguous() or not scales.is_contiguous()
            or not alphas.is_contiguous()):
        raise NVFP4Error(f"{name} must be contiguous uint8 codes and scales and float32 alphas on {dev}")
    return n, k


@functools.lru_cache(maxsize=1024)  # (a function of the sizes alone; asked for by every call)
def moe_workspace_bytes(tokens: int, width: int, inner: int, experts: int, top_k: int) -> int:
    return int(lib().nvfp4_moe_workspace_bytes(tokens, width, inner, experts, top_k))


def moe(X: torch.Tensor, logits: torch.Tensor, up, down, top_k: int, *, activation="silu", gated: bool = True,
        scoring: str = "softmax", normalize: bool = True, residual=None, out=None, workspace=None, stream=None):
    """A layer of experts for a few tokens (tokens * top_k <= 8192): each token's ``top_k`` largest ``logits`` ([tokens,
    experts] bf16 or fp32; equal ones by the lower index, -inf never) choose its experts, weighted by their ``softmax`` over
    all experts or the ``sigmoid``, with ``normalize`` divided by their sum; Y = residual + sum of weight * W2 act(W1 x),
    gated act(gate) * up, [tokens, width] bf16, in ``out`` if given (contiguous; it may be the residual). ``X`` is [tokens,
    width] bf16; ``up`` and ``down`` are the experts' NVFP4 weights stacked, as ``quantize`` returns them for each: codes
    [experts, N, K/2], scales [experts, N, K/16], alphas [experts], with (N, K) = (inner, or gated 2 * inner with the
    gate's rows first, width) and (width, inner). The activations between the products are rounded to bf16. A token of
    no experts (all logits -inf) gives its residual, or zeros."""
    ldx = _rows(X, "X", (torch.bfloat16,))
    tokens, width = X.shape
    dev = X.device
    ldl = _rows(logits, "logits", DTYPES, dev)
    if logits.shape[0] != tokens:
        raise NVFP4Error(f"logits must be [{tokens}, experts]")
    experts = logits.shape[1]
    if activation not in ACTIVATIONS or (gated and activation is None):
        raise NVFP4Error('activation must be None (not gated), "silu" or "gelu"')
    if scoring not in SCORING:
        raise NVFP4Error('scoring must be "softmax" or "sigmoid"')
    n, _ = _experts(up, "up", experts, dev, None, width)
    if gated and n % 2:
        raise NVFP4Error("gated experts have an even number of rows")
    inner = n // 2 if gated else n
    _experts(down, "down", experts, dev, width, inner)
    ldr = 0 if residual is None else _rows(residual, "residual", (torch.bfloat16,), dev, (tokens, width))
    _output(out, "out", (tokens, width), torch.bfloat16, dev)
    if out is not None and residual is not None:
        _apart(out, residual, "the residual")
    _no_graph(X, logits, up[2], down[2], residual, out)

    def call(st):
        Y = torch.empty_like(X, memory_format=torch.contiguous_format) if out is None else out
        ws, nbytes = _space(workspace, moe_workspace_bytes(tokens, width, inner, experts, top_k), dev)
        a = _moe_args(X.data_ptr(), ldx, logits.data_ptr(), ldl, DTYPES[logits.dtype], tokens, width, inner, experts, top_k,
                      up[0].data_ptr(), up[1].data_ptr(), up[2].data_ptr(), down[0].data_ptr(), down[1].data_ptr(),
                      down[2].data_ptr(), ACTIVATIONS[activation], int(gated), SCORING[scoring], int(normalize),
                      _ptr(residual) or 0, ldr, Y.data_ptr(), _ptr(ws) or 0, nbytes, st)
        _check(lib().nvfp4_moe(a))
        return Y

    return _run(dev, stream, call)
