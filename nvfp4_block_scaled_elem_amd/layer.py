"""Layer operators: what a layer computes around its NVFP4 products, forward and backward (C ABI: the layer
operators of ``include/nvfp4.h``). Marshalling only, like the rest of the binding.

    h8, s = rms_norm(X, w, residual=R, out_dtype="mxfp8")       # s = X + R, h8 = (codes, scales)
    dX, dw = rms_norm_grad(dY, s, w, dS=dS)
    Y, Z = linear(h8, *W, activation="silu", gated=True, keep="mxfp8")   # W = quantize(...)'s codes, scales, alpha
    dX, dZ, _ = linear_grad(dY, *W, Z=Z, activation="silu", gated=True)
    kept = quantize_mxfp8(A)                                    # an activation kept in 8 bits ...
    A_hat = dequantize_mxfp8(*kept)                             # ... and read back

An MXFP8 tensor is a pair (codes, scales): codes [rows, cols] ``torch.float8_e4m3fn`` and scales
[rows, ceil(cols / 32)] ``torch.float8_e8m0fnu``, a power of two per 32 consecutive columns (uint8 tensors
of the same bits are accepted too). Operands may have any row stride >= their columns; outputs are
contiguous and are allocated on the call's stream: ``stream``, or the current stream of the operands' device.

No call records an autograd graph: the gradients are calls of their own, for a program's own backward pass or
inside a ``torch.autograd.Function``. Where grad mode is on, an operand or a given output that requires a gradient is
refused, since its gradient would be lost without a word; ``torch.no_grad()`` or ``detach()`` says that none is wanted.
"""
from __future__ import annotations

import ctypes

import torch

from . import DTYPES, NVFP4Error, _check, _check_buffer, lib

MXFP8 = "mxfp8"
_MX = 2  # NVFP4_DTYPE_MXFP8
_CODES = (torch.float8_e4m3fn, torch.uint8)
_SCALES = (torch.float8_e8m0fnu, torch.uint8)


def _raw_stream(index: int) -> int:
    """The device's current stream. torch's own accessor of the raw pointer: a Stream object costs 3 us, more than
    half of what a one-token call spends on the host."""
    return torch._C._cuda_getCurrentRawStream(index)


ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2}  # enum nvfp4_activation


class _LinearArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_scales", ctypes.c_void_p), ("x_dtype", ctypes.c_int),
        ("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p), ("alpha", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("bias_dtype", ctypes.c_int), ("activation", ctypes.c_int), ("gated", ctypes.c_int),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("residual_dtype", ctypes.c_int),
        ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int), ("z", ctypes.c_void_p), ("z_scales", ctypes.c_void_p),
        ("z_dtype", ctypes.c_int), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
    ]


class _LinearGradArgs(ctypes.Structure):
    _fields_ = [
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
        ("z_scales", ctypes.c_void_p), ("z_dtype", ctypes.c_int), ("M", ctypes.c_int64), ("K", ctypes.c_int64),
        ("N", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
        ("activation", ctypes.c_int), ("gated", ctypes.c_int), ("dx", ctypes.c_void_p), ("dz", ctypes.c_void_p),
        ("dbias", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
    ]


def _run(dev, stream, call):
    """``call(raw stream)`` with the operands' device current, and the call's stream current where one is given
    (so that outputs and scratch are allocated on it)."""
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            return call(_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return call(_raw_stream(dev.index))
    if stream.device != dev:
        raise NVFP4Error(f"the stream is on {stream.device}, the operands on {dev}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _rows(t, name, dtypes, dev=None, shape=None):
    """Checks a 2-D operand with unit column stride; returns the elements between its rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda or t.dtype not in dtypes:
        raise NVFP4Error(f"{name} must be a 2-D CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if dev is not None and t.device != dev:
        raise NVFP4Error(f"{name} must be on {dev}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise NVFP4Error(f"{name} must be {list(shape)}, got {[rows, cols]}")
    if rows < 2:
        if cols > 1 and rows and t.stride(1) != 1:
            raise NVFP4Error(f"{name} must have unit column stride")
        return cols
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or s0 < cols:
        raise NVFP4Error(f"{name} must have unit column stride and rows that do not overlap")
    return s0


def _mx_pair(t, name, dev=None, shape=None):
    """Checks an MXFP8 pair; returns (codes, scales, elements between the codes' rows)."""
    if not isinstance(t, (tuple, list)) or len(t) != 2:
        raise NVFP4Error(f"{name} must be a pair (codes, scales)")
    codes, scales = t
    ld = _rows(codes, f"{name}'s codes", _CODES, dev, shape)
    rows, cols = codes.shape
    nb = -(-cols // 32)
    if (not isinstance(scales, torch.Tensor) or scales.dtype not in _SCALES or scales.device != codes.device
            or tuple(scales.shape) != (rows, nb) or not scales.is_contiguous()):
        raise NVFP4Error(f"{name}'s scales must be a contiguous [{rows}, {nb}] E8M0 tensor beside its codes")
    return codes, scales, ld


def _vector(t, name, n, dev, dtypes=DTYPES):
    if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.device != dev or tuple(t.shape) != (n,)
            or not t.is_contiguous()):
        raise NVFP4Error(f"{name} must be a contiguous [{n}] bf16 or fp32 tensor on {dev}")


def _output(t, name, shape, dtype, dev):
    if t is not None and (not isinstance(t, torch.Tensor) or tuple(t.shape) != shape or t.dtype != dtype
                          or t.device != dev or not t.is_contiguous()):
        raise NVFP4Error(f"{name} must be a contiguous {list(shape)} {dtype} tensor on {dev}")


def _new_mx(rows, cols, dev):
    return (torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=dev),
            torch.empty((rows, -(-cols // 32)), dtype=torch.float8_e8m0fnu, device=dev))


def _no_graph(*operands):
    if torch.is_grad_enabled():
        for t in operands:
            if t is not None and t.requires_grad:
                raise NVFP4Error("the layer and decoder operators record no autograd graph: call them under torch.no_grad() or "
                                 "in a torch.autograd.Function, with detached operands. The gradients that there are, are "
                                 "calls of their own: rms_norm_grad, linear_grad, and rotary with inverse=True; attention, "
                                 "kv_append and moe have none")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _space(workspace, need, dev):
    """(the scratch tensor or None, its bytes): the caller's, checked, or one allocated on the call's stream."""
    if workspace is not None:
        _check_buffer(workspace, "workspace", need, dev)
        return workspace, workspace.numel() * workspace.element_size()
    return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need else (None, 0)


def quantize_mxfp8(X: torch.Tensor, *, stream=None):
    """MXFP8 (codes, scales) of ``X`` ([rows, cols] bf16 or fp32 CUDA tensor): per 32 consecutive columns the
    smallest power-of-two scale under which nothing saturates, and the nearest E4M3 codes (ties to even)."""
    ld = _rows(X, "X", DTYPES)
    _no_graph(X)
    rows, cols = X.shape
    dev = X.device

    def call(st):
        codes, scales = _new_mx(rows, cols, dev)
        _check(lib().nvfp4_mxfp8_quantize(X.data_ptr(), ld, DTYPES[X.dtype], rows, cols, codes.data_ptr(),
                                          scales.data_ptr(), st))
        return codes, scales

    return _run(dev, stream, call)


def dequantize_mxfp8(codes: torch.Tensor, scales: torch.Tensor, dtype=torch.bfloat16, *, stream=None) -> torch.Tensor:
    """The values of an MXFP8 tensor as bf16 or fp32."""
    codes, scales, ld = _mx_pair((codes, scales), "the tensor")
    _no_graph(codes)
    if dtype not in DTYPES:
        raise NVFP4Error("dtype must be bf16 or fp32")
    rows, cols = codes.shape
    dev = codes.device

    def call(st):
        out = torch.empty((rows, cols), dtype=dtype, device=dev)
        _check(lib().nvfp4_mxfp8_dequantize(codes.data_ptr(), ld, scales.data_ptr(), rows, cols, out.data_ptr(),
                                            DTYPES[dtype], st))
        return out

    return _run(dev, stream, call)


def rms_norm(X: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, *, residual=None, out_dtype=None,
             sum_out=None, stream=None):
    """Root-mean-square norm of ``X`` ([rows, cols] bf16 or fp32) over its rows: Y = h / sqrt(mean(h^2) + eps) *
    weight with h = X, or X + residual. Y is of X's dtype, of ``out_dtype`` (bf16 or fp32), or an MXFP8 pair
    (``out_dtype="mxfp8"``). Returns Y, or (Y, h) where a ``residual`` (X's shape and dtype) is given: h rounded to
    X's dtype, in ``sum_out`` if given (which may be a contiguous ``residual``)."""
    ldx = _rows(X, "X", DTYPES)
    rows, cols = X.shape
    dev = X.device
    _vector(weight, "weight", cols, dev)
    out_dtype = X.dtype if out_dtype is None else out_dtype
    if out_dtype != MXFP8 and out_dtype not in DTYPES:
        raise NVFP4Error('out_dtype must be bf16, fp32 or "mxfp8"')
    if residual is None and sum_out is not None:
        raise NVFP4Error("sum_out needs a residual")
    ldr = 0 if residual is None else _rows(residual, "residual", (X.dtype,), dev, (rows, cols))
    _output(sum_out, "sum_out", (rows, cols), X.dtype, dev)
    _no_graph(X, weight, residual, sum_out)

    def call(st):
        if out_dtype == MXFP8:
            Y = _new_mx(rows, cols, dev)
            y, ys, yt = Y[0].data_ptr(), Y[1].data_ptr(), _MX
        else:
            Y = torch.empty_like(X, dtype=out_dtype, memory_format=torch.contiguous_format)
            y, ys, yt = Y.data_ptr(), None, DTYPES[out_dtype]
        h = sum_out
        if residual is not None and h is None:
            h = torch.empty_like(X, memory_format=torch.contiguous_format)
        _check(lib().nvfp4_rms_norm(X.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), DTYPES[X.dtype],
                                    DTYPES[weight.dtype], rows, cols, eps, _ptr(h), y, ys, yt, st))
        return Y if residual is None else (Y, h)

    return _run(dev, stream, call)


def rms_norm_grad_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_rms_norm_grad_workspace_bytes(rows, cols))


def rms_norm_grad(dY: torch.Tensor, S, weight: torch.Tensor, eps: float = 1e-6, *, dS=None, workspace=None,
                  stream=None):
    """Gradients of ``rms_norm``: ``dY`` at its output, ``S`` the h it normed (of dY's dtype, or an MXFP8 pair: a
    checkpoint of it), ``dS`` (nullable, dY's dtype) the gradient at h from its other uses. Returns (dX,
    dweight): dX of dY's dtype, the gradient at X and at the residual alike, and dweight [cols] fp32."""
    lddy = _rows(dY, "dY", DTYPES)
    rows, cols = dY.shape
    dev = dY.device
    if isinstance(S, (tuple, list)):
        h, hs, ldh = _mx_pair(S, "S", dev, (rows, cols))
        ht = _MX
    else:
        ldh = _rows(S, "S", (dY.dtype,), dev, (rows, cols))
        h, hs, ht = S, None, DTYPES[dY.dtype]
    _vector(weight, "weight", cols, dev)
    ldds = 0 if dS is None else _rows(dS, "dS", (dY.dtype,), dev, (rows, cols))
    _no_graph(dY, h, weight, dS)

    def call(st):
        dX = torch.empty_like(dY, memory_format=torch.contiguous_format)
        dw = torch.empty(cols, dtype=torch.float32, device=dev)
        ws, nbytes = _space(workspace, rms_norm_grad_workspace_bytes(rows, cols), dev)
        _check(lib().nvfp4_rms_norm_grad(dY.data_ptr(), lddy, h.data_ptr(), ldh, _ptr(hs), ht, weight.data_ptr(),
                                         _ptr(dS), ldds, DTYPES[dY.dtype], DTYPES[weight.dtype], rows, cols, eps,
                                         dX.data_ptr(), dw.data_ptr(), _ptr(ws), nbytes, st))
        return dX, dw

    return _run(dev, stream, call)


def _weights(codes, scales, alpha, dev, K=None):
    """Checks NVFP4 weights as ``quantize`` returns them; returns (N, K)."""
    if codes.dim() != 2 or (K is not None and 2 * codes.shape[1] != K) or codes.shape[1] % 8:
        raise NVFP4Error("codes must be [N, K/2] with K % 16 == 0")
    N, half = codes.shape
    K = 2 * half
    if (codes.device == scales.device == alpha.device == dev and codes.dtype == scales.dtype == torch.uint8
            and alpha.dtype == torch.float32 and scales.numel() >= N * half // 8 and alpha.numel() >= 1
            and codes.is_contiguous() and scales.is_contiguous() and alpha.is_contiguous()):
        return N, K
    _check_buffer(codes, "codes", N * K // 2, dev, torch.uint8)
    _check_buffer(scales, "scales", N * K // 16, dev, torch.uint8)
    _check_buffer(alpha, "alpha", 4, dev, torch.float32)
    return N, K


def _activation(activation, gated, N):
    if activation not in ACTIVATIONS:
        raise NVFP4Error('activation must be None, "silu" or "gelu"')
    if gated and (activation is None or N % 2):
        raise NVFP4Error("a gated product needs an activation and an even number of weight rows")
    return N // 2 if gated else N


def linear_workspace_bytes(M: int, K: int, N: int, gated: bool = False, keep=None, x_mxfp8: bool = False) -> int:
    return int(lib().nvfp4_linear_workspace_bytes(M, K, N, _MX if x_mxfp8 else 0, int(gated), _MX if keep == MXFP8 else 0))


def linear(X, codes: torch.Tensor, scales: torch.Tensor, alpha: torch.Tensor, *, bias=None, activation=None,
           gated: bool = False, residual=None, out_dtype=torch.bfloat16, keep=None, out=None, workspace=None,
           stream=None):
    """Product with NVFP4 weights (codes [N, K/2], scales [N, K/16], alpha [1], as ``quantize`` returns them) and
    the rest of a projection in its epilogue: Z = alpha * (X @ Wq.T) + bias and Y = act(Z) + residual, or, gated
    with F = N // 2, Y = act(Z[:, :F]) * Z[:, F:] + residual. ``X`` is [M, K] bf16 or an MXFP8 pair; ``activation`` None,
    "silu" or "gelu" (tanh form); ``bias`` [N] and ``residual`` (Y's shape) bf16 or fp32; Y is of ``out_dtype``, in
    ``out`` if given (contiguous; it may be the residual itself). ``keep`` (None, torch.bfloat16 or "mxfp8") asks
    for Z too, [M, N] in that form, for ``linear_grad`` (gated and "mxfp8": F % 32 == 0). Returns Y, or (Y, Z). Without
    any of these it is ``matmul``'s product by other kernels: faster for 2 to 64 rows and for thousands, slower for most
    one-row products and some of a few hundred rows."""
    if isinstance(X, (tuple, list)):
        x, xs, ldx = _mx_pair(X, "X")
        xt = _MX
    else:
        ldx = _rows(X, "X", (torch.bfloat16,))
        x, xs, xt = X, None, 0
    M, K = x.shape
    dev = x.device
    N, K = _weights(codes, scales, alpha, dev, K)
    F = _activation(activation, gated, N)
    if out_dtype not in DTYPES:
        raise NVFP4Error("out_dtype must be bf16 or fp32")
    if keep not in (None, torch.bfloat16, MXFP8):
        raise NVFP4Error('keep must be None, torch.bfloat16 or "mxfp8"')
    if bias is not None:
        _vector(bias, "bias", N, dev)
    ldr = 0 if residual is None else _rows(residual, "residual", DTYPES, dev, (M, F))
    _output(out, "out", (M, F), out_dtype, dev)
    _no_graph(x, alpha, bias, residual, out)

    def call(st):
        Y = torch.empty((M, F), dtype=out_dtype, device=dev) if out is None else out
        Z, z, zs = None, None, None
        if keep == MXFP8:
            Z = _new_mx(M, N, dev)
            z, zs = Z[0].data_ptr(), Z[1].data_ptr()
        elif keep is not None:
            Z = torch.empty((M, N), dtype=keep, device=dev)
            z = Z.data_ptr()
        ws, nbytes = _space(workspace, linear_workspace_bytes(M, K, N, gated, keep, xt == _MX), dev)
        a = _LinearArgs(x.data_ptr(), ldx, _ptr(xs), xt, M, K, N, codes.data_ptr(), scales.data_ptr(), alpha.data_ptr(),
                        _ptr(bias), 0 if bias is None else DTYPES[bias.dtype], ACTIVATIONS[activation], int(gated),
                        _ptr(residual), ldr, 0 if residual is None else DTYPES[residual.dtype], Y.data_ptr(),
                        DTYPES[out_dtype], z, zs, _MX if keep == MXFP8 else 0, _ptr(ws), nbytes, st)
        _check(lib().nvfp4_linear(ctypes.byref(a)))
        return Y if keep is None else (Y, Z)

    return _run(dev, stream, call)


def linear_grad_workspace_bytes(M: int, K: int, N: int, gated: bool = False, bias: bool = False) -> int:
    return int(lib().nvfp4_linear_grad_workspace_bytes(M, K, N, int(gated), int(bias)))


def linear_grad(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, alpha: torch.Tensor, *, Z=None,
                activation=None, gated: bool = False, bias: bool = False, workspace=None, stream=None):
    """Gradients of ``linear`` for ``dY`` (bf16, Y's shape) at its output, with ``Z`` as it kept it (bf16 or an MXFP8
    pair; None without an activation). Returns (dX, dZ, dbias): dZ [M, N] bf16, the gradient at Z (None without an
    activation, where it is dY); dX [M, K] bf16, the product of dZ as rounded; dbias [N] fp32 where ``bias`` is true,
    else None, of dZ unrounded. The residual's gradient is dY; the weights are frozen."""
    lddy = _rows(dY, "dY", (torch.bfloat16,))
    dev = dY.device
    N, K = _weights(codes, scales, alpha, dev)
    F = _activation(activation, gated, N)
    M = dY.shape[0]
    if dY.shape[1] != F:
        raise NVFP4Error(f"dY must be [M, {F}]")
    if (Z is None) != (activation is None):
        raise NVFP4Error("Z is needed with an activation, and only there")
    z, zs, ldz, zt = None, None, 0, 0
    if isinstance(Z, (tuple, list)):
        z, zs, ldz = _mx_pair(Z, "Z", dev, (M, N))
        zt = _MX
    elif Z is not None:
        ldz = _rows(Z, "Z", (torch.bfloat16,), dev, (M, N))
        z = Z
    _no_graph(dY, alpha, z)

    def call(st):
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        dZ = None if activation is None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        db = torch.empty(N, dtype=torch.float32, device=dev) if bias else None
        ws, nbytes = _space(workspace, linear_grad_workspace_bytes(M, K, N, gated, bias), dev)
        a = _LinearGradArgs(dY.data_ptr(), lddy, _ptr(z), ldz, _ptr(zs), zt, M, K, N, codes.data_ptr(),
                            scales.data_ptr(), alpha.data_ptr(), ACTIVATIONS[activation], int(gated), dX.data_ptr(),
                            _ptr(dZ), _ptr(db), _ptr(ws), nbytes, st)
        _check(lib().nvfp4_linear_grad(ctypes.byref(a)))
        return dX, dZ, db

    return _run(dev, stream, call)
