"""The layer operators and autograd: no call drops a gradient silently, and they make a torch.autograd.Function."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def test_operands_that_require_gradients_are_refused():
    W = nv.quantize(rand(1, 64, 96, std=0.05), "4o6")
    x, w, b, r, dy, z = rand(2, 4, 96), rand(3, 96), rand(4, 64), rand(5, 4, 64), rand(6, 4, 64), rand(7, 4, 64)
    alpha = W[2].clone().requires_grad_()
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    calls = [
        lambda: nv.quantize_mxfp8(leaf(x)), lambda: nv.rms_norm(leaf(x), w), lambda: nv.rms_norm(x, leaf(w)),
        lambda: nv.rms_norm(x, w, residual=leaf(x)), lambda: nv.rms_norm_grad(leaf(x), x, w),
        lambda: nv.rms_norm_grad(x, leaf(x), w), lambda: nv.rms_norm_grad(x, x, leaf(w)),
        lambda: nv.rms_norm_grad(x, x, w, dS=leaf(x)), lambda: nv.linear(leaf(x), *W),
        lambda: nv.linear(x, *W[:2], alpha), lambda: nv.linear(x, *W, bias=leaf(b)),
        lambda: nv.linear(x, *W, residual=leaf(r)), lambda: nv.linear_grad(leaf(dy), *W),
        lambda: nv.linear_grad(dy, *W, Z=leaf(z), activation="silu"), lambda: nv.linear_grad(dy, *W[:2], alpha),
        lambda: nv.linear(x * leaf(x), *W),  # not a leaf
    ]
    for i, call in enumerate(calls):
        print(f"call {i}", flush=True)
        with pytest.raises(nv.NVFP4Error, match="autograd"):
            call()
        with torch.no_grad():
            call()


def test_outputs_that_require_gradients_are_refused():
    W = nv.quantize(rand(21, 64, 96, std=0.05), "4o6")
    x, w = rand(22, 4, 96), rand(23, 96)
    for call in (lambda: nv.linear(x, *W, out=rand(24, 4, 64).requires_grad_()),
                 lambda: nv.rms_norm(x, w, residual=x, sum_out=rand(25, 4, 96).requires_grad_())):
        with pytest.raises(nv.NVFP4Error, match="autograd"):
            call()
        with torch.no_grad():
            call()


class Projection(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wn, codes, scales, alpha):
        h = nv.rms_norm(x, wn)
        y, Z = nv.linear(h, codes, scales, alpha, activation="silu", gated=True, keep="mxfp8")
        ctx.save_for_backward(x, wn, codes, scales, alpha, *Z)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, wn, codes, scales, alpha, *Z = ctx.saved_tensors
        dh, _, _ = nv.linear_grad(dy, codes, scales, alpha, Z=tuple(Z), activation="silu", gated=True)
        dx, dw = nv.rms_norm_grad(dh, x, wn)
        return dx, dw.to(wn.dtype), None, None, None


def test_operators_in_an_autograd_function():
    W = nv.quantize(rand(11, 128, 96, std=0.05), "4o6")
    x, wn, dy = rand(12, 20, 96), rand(13, 96) + 1, rand(14, 20, 64)
    xg, wg = x.clone().requires_grad_(), wn.clone().requires_grad_()
    y = Projection.apply(xg, wg, *W)
    y.backward(dy)
    h = nv.rms_norm(x, wn)
    want, Z = nv.linear(h, *W, activation="silu", gated=True, keep="mxfp8")
    dh, _, _ = nv.linear_grad(dy, *W, Z=Z, activation="silu", gated=True)
    dx, dw = nv.rms_norm_grad(dh, x, wn)
    assert torch.equal(y, want) and torch.equal(xg.grad, dx) and torch.equal(wg.grad, dw.to(BF16))
