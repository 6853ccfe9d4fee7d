"""The layer operators where their inputs are extreme, on the GPU against binary64 (tests/layer_ref.py)."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print(msg, flush=True)


def rand(seed, *shape, dtype=BF16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def make_weights(n, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(n * 31 + k + seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(0x10, 0x60, (n, k // 16), generator=g, device="cuda").to(torch.uint8)
    return codes, scales, torch.full((1,), 0.0123, device="cuda")


ACTS = [("silu", False), ("gelu", False), ("silu", True), ("gelu", True)]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("m,k", [(8, 208), (300, 208), (300, 48)])
@pytest.mark.parametrize("act,gated", ACTS)
def test_gradient_of_values_that_are_not_finite(act, gated, m, k, mx):
    """A NaN or an infinity in z or dy makes dZ what the formula makes of it (in MXFP8, throughout its block), dX NaN
    in its row and dbias in its columns; every other value is the one of the call without them, bit for bit."""
    F = 96
    n = 2 * F if gated else F
    W = make_weights(n, k)
    say(f"not finite: {act} gated={gated} M={m} K={k} mx={mx}")
    z, dy = rand(1, m, n, std=2.0), rand(2, m, F)
    bad_z, bad_dy = z.clone(), dy.clone()
    bad_z[2, 5], bad_z[3, 40], bad_z[4, 70] = float("nan"), float("inf"), -float("inf")
    bad_z[5, n - 9] = float("nan")  # the up part where gated
    bad_dy[6, 11], bad_dy[7, 12] = float("nan"), float("inf")
    kind = nv.quantize_mxfp8 if mx else (lambda t: t)
    kw = dict(activation=act, gated=gated, bias=True)
    clean = nv.linear_grad(dy, *W, Z=kind(z), **kw)
    Z = kind(bad_z)
    dX, dZ, db = nv.linear_grad(bad_dy, *W, Z=Z, **kw)
    want, _ = ref.linear_dz(bad_dy.double(), ref.value(Z), act, gated)
    assert torch.equal(dZ.isnan(), want.isnan())
    assert want[2:6].isnan().any(1).all() and want[6].isnan().any() and not want[7].isfinite().all()
    assert torch.equal(dZ.isinf(), want.isinf()) and torch.equal(dZ[dZ.isinf()].double(), want[want.isinf()])
    ok = want.isfinite()
    assert torch.equal(dZ[ok], clean[1][ok])
    rows = ok.all(1)
    assert rows.sum() == m - 6
    assert torch.equal(dX[rows], clean[0][rows]) and not dX[~rows].isfinite().any()
    cols = ok.all(0)
    assert torch.equal(db[cols], clean[2][cols]) and not db[~cols].isfinite().any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_far_from_zero(act):
    """|z| to 1e19: the slope is 0 or 1 to binary32 (the logistic function's error is at most 2^-22 of it, and 2^-126
    times the terms' factors where it vanishes)."""
    F, k = 96, 64
    W = make_weights(F, k)
    at = torch.tensor([29.0, 30.0, 31.0, 100.0, 1e4, 1e19], device="cuda")
    z = torch.cat((at, -at)).repeat(8).repeat(12, 1).to(BF16)
    dy = rand(3, 12, F)
    _, dZ, _ = nv.linear_grad(dy, *W, Z=z, activation=act)
    slope = ref.act_slope(z.double(), act)
    # |z| = 29 to 31 under silu: e^-|z| off by |z| 2^-24 and a few units of itself, times 1 + |z|
    small = 64 * ref.U * torch.exp(-z.double().abs()) * (1 + z.double().abs()) * (act == "silu")
    err = dy.double().abs() * (2.0 ** -22 * slope.abs() + small + ref.TINY * (1 + z.double().abs()))
    want = dy.double() * slope
    assert ((dZ.double() - want).abs() <= err + want.abs() * ref.HALF[BF16]).all()


def test_weight_gradient_of_very_long_rows():
    """More than 2^27 columns: dweight's last columns too. The sum of a row's squares has paths of cols / 1024 additions
    (layer_ref.norm_depth), each off by 2^-24 of it."""
    cols = (1 << 27) + 40
    say(f"rms_norm_grad 1 x {cols}")
    dy, h, w = rand(5, 1, cols), rand(6, 1, cols), rand(7, cols) + 1
    dx, dw = nv.rms_norm_grad(dy, h, w, 1e-6)
    rx, rw, ex, ew = ref.rms_norm_grad(dy, h, w, 1e-6)
    assert ((dw.double() - rw).abs() <= ew + rw.abs() * ref.U).all()
    assert ((dx.double() - rx).abs() <= ex + rx.abs() * ref.HALF[BF16]).all()
    del rx, rw, ex, ew, dx, dw
    _, none = nv.rms_norm_grad(dy[:0], h[:0], w, 1e-6)
    assert none.shape == (cols,) and (none == 0).all()
