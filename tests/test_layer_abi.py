"""The layer operators' C entry points refuse bad arguments on the host, before anything touches a device, and
the binding's structs have the C compiler's layout (CPU only: no call here enqueues anything)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from nvfp4_block_scaled_elem_amd import build as nvbuild
from nvfp4_block_scaled_elem_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -3
FAKE = 0x100000  # never dereferenced: every call below fails validation first, or has no rows


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        nvbuild.build()
    return nv.lib()


def test_rms_norm_rejects(L):
    def call(x=FAKE, ldx=64, r=None, ldr=0, w=FAKE, dt=0, wt=0, rows=4, cols=64, eps=1e-6, h=None, y=FAKE, ys=None, yt=0):
        return L.nvfp4_rms_norm(x, ldx, r, ldr, w, dt, wt, rows, cols, eps, h, y, ys, yt, None)

    assert call(x=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID
    assert call(dt=2) == INVALID and call(dt=3) == INVALID and call(wt=2) == INVALID and call(yt=3) == INVALID
    assert call(rows=-1) == INVALID and call(cols=0) == INVALID and call(cols=-8) == INVALID
    assert call(eps=-1e-6) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(ldx=63) == INVALID and call(r=FAKE, h=FAKE, ldr=63) == INVALID
    assert call(r=FAKE, ldr=64) == INVALID and call(h=FAKE) == INVALID  # one without the other
    assert call(yt=2) == INVALID and call(ys=FAKE) == INVALID  # MXFP8 and its scales go together
    assert call(x=FAKE + 1) == INVALID and call(dt=1, x=FAKE + 2) == INVALID and call(y=FAKE + 1) == INVALID
    assert call(wt=1, w=FAKE + 2) == INVALID and call(yt=1, y=FAKE + 2) == INVALID
    assert call(rows=(1 << 23) + 1) == SHAPE and call(rows=1 << 20, cols=1 << 15) == SHAPE
    assert call(rows=1, cols=1 << 35) == SHAPE and call(cols=(1 << 63) - 1) == SHAPE
    assert call(rows=0) == OK and call(rows=0, x=None, y=None) == OK


def test_rms_norm_grad_rejects(L):
    def call(dy=FAKE, lddy=64, h=FAKE, ldh=64, hs=None, ht=0, w=FAKE, dh=None, lddh=0, dt=0, wt=0, rows=4, cols=64,
             eps=1e-6, dx=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
        return L.nvfp4_rms_norm_grad(dy, lddy, h, ldh, hs, ht, w, dh, lddh, dt, wt, rows, cols, eps, dx, dw, ws, n, None)

    for kw in (dict(dy=None), dict(h=None), dict(w=None), dict(dx=None), dict(dw=None), dict(dt=2, ht=2), dict(ht=1),
               dict(wt=2), dict(ht=2), dict(hs=FAKE), dict(lddy=63), dict(ldh=63), dict(dh=FAKE, lddh=63),
               dict(eps=-1.0), dict(dy=FAKE + 1), dict(dw=FAKE + 2), dict(ws=FAKE + 16), dict(rows=-1), dict(cols=0)):
        assert call(**kw) == INVALID, kw
    assert call(rows=(1 << 23) + 1) == SHAPE
    need = L.nvfp4_rms_norm_grad_workspace_bytes(4, 64)
    assert need == 4 * 4 * 64 and call(n=need - 1) == WORKSPACE
    assert L.nvfp4_rms_norm_grad_workspace_bytes(0, 64) == 0 and L.nvfp4_rms_norm_grad_workspace_bytes(-1, 64) == 0
    assert L.nvfp4_rms_norm_grad_workspace_bytes(100, 20000) == 4 * (2 * 20000 + 100)


def test_mxfp8_rejects(L):
    q, d = L.nvfp4_mxfp8_quantize, L.nvfp4_mxfp8_dequantize
    assert q(None, 64, 0, 4, 64, FAKE, FAKE, None) == INVALID and q(FAKE, 63, 0, 4, 64, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 64, 2, 4, 64, FAKE, FAKE, None) == INVALID and q(FAKE + 1, 64, 0, 4, 64, FAKE, FAKE, None) == INVALID
    assert q(FAKE, 64, 0, 4, 64, None, FAKE, None) == INVALID and q(FAKE, 64, 0, 4, 64, FAKE, None, None) == INVALID
    assert q(FAKE, 1, 0, 1 << 24, 1, FAKE, FAKE, None) == SHAPE and q(None, 64, 0, 0, 64, None, None, None) == OK
    assert d(None, 64, FAKE, 4, 64, FAKE, 0, None) == INVALID and d(FAKE, 63, FAKE, 4, 64, FAKE, 0, None) == INVALID
    assert d(FAKE, 64, FAKE, 4, 64, FAKE, 2, None) == INVALID and d(FAKE, 64, FAKE, 4, 64, FAKE + 2, 1, None) == INVALID
    assert d(FAKE, 64, FAKE, -1, 64, FAKE, 0, None) == INVALID and d(None, 64, None, 0, 64, None, 0, None) == OK


def linear_args(**kw):
    a = layer._LinearArgs(x=FAKE, ldx=96, M=4, K=96, N=64, codes=FAKE, scales=FAKE, alpha=FAKE, y=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(x=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(alpha=None), INVALID),
    (dict(y=None), INVALID), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(K=104), SHAPE),
    (dict(x_dtype=1), INVALID), (dict(x_dtype=2), INVALID), (dict(x_scales=FAKE), INVALID), (dict(y_dtype=2), INVALID),
    (dict(activation=3), INVALID), (dict(activation=-1), INVALID), (dict(gated=1), INVALID),
    (dict(gated=2, activation=1), INVALID), (dict(gated=1, activation=1, N=63), SHAPE), (dict(ldx=95), INVALID),
    (dict(bias=FAKE, bias_dtype=2), INVALID), (dict(bias=FAKE + 1), INVALID), (dict(bias=FAKE + 2, bias_dtype=1), INVALID),
    (dict(residual=FAKE, ldr=63), INVALID), (dict(residual=FAKE, ldr=64, residual_dtype=2), INVALID),
    (dict(z=FAKE, z_dtype=1), INVALID), (dict(z=FAKE, z_dtype=2), INVALID), (dict(z=FAKE, z_scales=FAKE), INVALID),
    (dict(z_scales=FAKE), INVALID), (dict(gated=1, activation=1, N=96, z=FAKE, z_scales=FAKE, z_dtype=2), SHAPE),
    (dict(codes=FAKE + 4), INVALID), (dict(alpha=FAKE + 2), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(workspace=FAKE + 16), INVALID), (dict(K=(1 << 21) + 16), SHAPE),
    (dict(N=(1 << 21) + 1), SHAPE), (dict(ldx=1 << 23), SHAPE), (dict(M=1 << 20, K=1 << 16, ldx=1 << 16), SHAPE), (dict(M=0), OK),
    (dict(M=100, K=4096, ldx=4096, workspace=FAKE, workspace_bytes=256), WORKSPACE),
])
def test_linear_rejects(L, kw, err):
    assert L.nvfp4_linear(ctypes.byref(linear_args(**kw))) == err


def grad_args(**kw):
    a = layer._LinearGradArgs(dy=FAKE, lddy=64, M=4, K=96, N=64, codes=FAKE, scales=FAKE, alpha=FAKE, dx=FAKE,
                              workspace=FAKE, workspace_bytes=256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


WITH_Z = dict(activation=1, z=FAKE, ldz=64, dz=FAKE)


@pytest.mark.parametrize("kw,err", [
    (dict(dy=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(alpha=None), INVALID),
    (dict(dx=None), INVALID), (dict(lddy=63), INVALID), (dict(M=-1), INVALID), (dict(K=104), SHAPE),
    (dict(z=FAKE), INVALID), (dict(dz=FAKE), INVALID), (dict(z_scales=FAKE), INVALID), (dict(activation=1), INVALID),
    (dict(WITH_Z, dz=None), INVALID), (dict(WITH_Z, ldz=63), INVALID), (dict(WITH_Z, z_dtype=1), INVALID),
    (dict(WITH_Z, z_dtype=2), INVALID), (dict(WITH_Z, z=FAKE + 1), INVALID), (dict(gated=1), INVALID),
    (dict(WITH_Z, gated=1, N=96, z_dtype=2, z_scales=FAKE), SHAPE), (dict(WITH_Z, gated=1, N=63), SHAPE),
    (dict(dbias=FAKE + 2), INVALID), (dict(workspace=FAKE + 16), INVALID), (dict(dy=FAKE + 1), INVALID),
    (dict(lddy=1 << 23), SHAPE), (dict(codes=FAKE + 4), INVALID), (dict(K=48), WORKSPACE), (dict(WITH_Z, K=48), WORKSPACE), (dict(M=0), OK),
])
def test_linear_grad_rejects(L, kw, err):
    assert L.nvfp4_linear_grad(ctypes.byref(grad_args(**kw))) == err


def test_null_arguments(L):
    assert L.nvfp4_linear(None) == INVALID and L.nvfp4_linear_grad(None) == INVALID


def test_workspace_sizes(L):
    assert L.nvfp4_linear_workspace_bytes(1, 4096, 4096, 0, 0, 0) == 0
    assert L.nvfp4_linear_workspace_bytes(0, 4096, 4096, 0, 0, 0) == 0
    assert L.nvfp4_linear_workspace_bytes(4, 100, 64, 0, 0, 0) == 0  # no such product
    assert L.nvfp4_linear_workspace_bytes(100, 4096, 64, 0, 0, 0) > 0
    assert L.nvfp4_linear_workspace_bytes(100, 96, 64, 2, 0, 0) >= 2 * 100 * 96  # an MXFP8 X, decoded
    # the decoded weights, and a partial sum of the bias per chunk of rows
    assert L.nvfp4_linear_grad_workspace_bytes(4096, 4096, 4096, 0, 0) >= 2 * 4096 * 4096
    assert (L.nvfp4_linear_grad_workspace_bytes(64, 96, 64, 0, 1) > L.nvfp4_linear_grad_workspace_bytes(64, 96, 64, 0, 0))


@pytest.mark.parametrize("name,struct", [("nvfp4_linear_args_t", layer._LinearArgs),
                                         ("nvfp4_linear_grad_args_t", layer._LinearGradArgs)])
def test_struct_layouts(tmp_path, name, struct):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "nvfp4.h"\nint main(void) {\n'
                   + f'printf("%zu\\n", sizeof({name}));\n'
                   + "".join(f'printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert out == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: nv.quantize_mxfp8(x), lambda: nv.rms_norm(x, x[0]), lambda: nv.rms_norm_grad(x, x, x[0]),
                 lambda: nv.linear(x, x, x, x), lambda: nv.linear_grad(x, x, x, x),
                 lambda: nv.dequantize_mxfp8(x.to(torch.float8_e4m3fn), x[:, :2])):
        with pytest.raises(nv.NVFP4Error):
            call()


def test_weights_are_bounded(L):
    """2^35 weights: refused by the products, like any operand of that size."""
    lin = layer._LinearArgs(x=FAKE, M=1, K=1 << 20, N=1 << 15, codes=FAKE, scales=FAKE, alpha=FAKE, y=FAKE)
    grad = layer._LinearGradArgs(dy=FAKE, M=1, K=1 << 20, N=1 << 15, codes=FAKE, scales=FAKE, alpha=FAKE, dx=FAKE)
    assert L.nvfp4_linear(ctypes.byref(lin)) == SHAPE and L.nvfp4_linear_grad(ctypes.byref(grad)) == SHAPE
    assert L.nvfp4_linear_workspace_bytes(100, 1 << 20, 1 << 15, 0, 0, 0) == 0
    assert L.nvfp4_linear_workspace_bytes(100, 1 << 20, (1 << 15) - 16, 0, 0, 0) > 0
    assert L.nvfp4_linear_grad_workspace_bytes(100, 1 << 20, 1 << 15, 0, 0) == 0
