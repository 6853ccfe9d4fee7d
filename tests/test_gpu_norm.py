"""The root-mean-square norm, its gradient and the MXFP8 form on the GPU, against binary64 (tests/layer_ref.py).

Tolerances: the kernels work in binary32 and round each output once. A row's sum of squares adds at most
`norm_depth` terms on a path, each addition off by 2^-24 of the (non-negative) sum, which the square root
halves; the remaining steps (h, mean, root, reciprocal, two products) are eight roundings at most. An output
adds half a step of its type. The gradient's bounds are in layer_ref.rms_norm_grad. MXFP8 of given values is
exact: the scale is a power of two and each code one rounding, so codes and scales must be equal."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def say(msg):
    print(msg, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(seed, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * std).to(dtype)


def u8(t):
    return t.view(torch.uint8)


COLS = [1, 2, 7, 8, 9, 31, 32, 33, 63, 100, 512, 513, 1000, 1024, 1030, 2047, 2048, 2056, 4096, 4104, 8192, 8200,
        16384, 16392, 20001, 40000]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 5])
def test_mxfp8_is_exact(rows, cols, dtype):
    say(f"mxfp8 {rows}x{cols} {dtype}")
    x = rand(rows + cols, rows, cols, dtype=F32)
    x = (x * 2.0 ** torch.randint(-20, 20, (rows, cols), generator=gen(1), device="cuda").float()).to(dtype)
    x[0, : cols // 2] = 0
    codes, scales = nv.quantize_mxfp8(x)
    q, b = ref.mx_quantize(x.double())
    assert torch.equal(u8(scales), b)
    assert torch.equal(codes.double(), q)
    for out in (BF16, F32):
        y = nv.dequantize_mxfp8(codes, scales, out)
        assert y.dtype == out and torch.equal(y.double(), ref.mx_values(codes, scales))
    assert torch.equal(nv.dequantize_mxfp8(u8(codes), u8(scales)), nv.dequantize_mxfp8(codes, scales))


def test_mxfp8_borders():
    """Block maxima at and next to 448 * 2^e, the ends of the scale's range, and the smallest codes."""
    up, down = torch.tensor(448.0).view(torch.int32) + 1, torch.tensor(448.0).view(torch.int32) - 1
    tops = [448.0, up.view(F32).item(), down.view(F32).item(), 256.0, 255.9, 1.0, 0.0, 2.0 ** -126, 1.75 * 2.0 ** -119,
            1.76 * 2.0 ** -119, 2.0 ** -130, 3.3e38, 1.75 * 2.0 ** 127, 2.0 ** -149]
    x = torch.zeros(len(tops), 64, device="cuda")
    for i, t in enumerate(tops):
        x[i, 3] = t
        x[i, 4:20] = t * 2.0 ** -torch.arange(3, 19, device="cuda").float() * 1.5
        x[i, 40] = -t
    codes, scales = nv.quantize_mxfp8(x)
    q, b = ref.mx_quantize(x.double())
    assert torch.equal(u8(scales), b)
    assert torch.equal(codes.double(), q)


def test_mxfp8_not_finite():
    """A block with a NaN or an infinity reads back as NaN; its neighbours are untouched."""
    x = rand(3, 4, 96, dtype=F32)
    x[0, 40], x[1, 5], x[2, 95] = float("nan"), float("inf"), -float("inf")
    codes, scales = nv.quantize_mxfp8(x)
    bad = torch.zeros(4, 3, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 0] = bad[2, 2] = True
    assert torch.equal(u8(scales) == 255, bad)
    y = nv.dequantize_mxfp8(codes, scales, F32)
    assert torch.equal(y.isnan(), bad.repeat_interleave(32, 1))
    q, b = ref.mx_quantize(torch.where(bad.repeat_interleave(32, 1), 0.0, x).double())
    good = ~bad.repeat_interleave(32, 1)
    assert torch.equal(codes.double()[good], q[good])


def check_y(y, want, cols, extra=0.0):
    """y (a tensor or an MXFP8 pair) against binary64 values that binary32 has to a relative `tol`."""
    tol = (ref.norm_depth(cols) / 2 + 8) * ref.U
    if isinstance(y, tuple):
        b = ref.mx_blocks(want).abs().amax(-1)
        byte = u8(y[1]).to(torch.int64)
        lo, hi = (ref.mx_scale_exp(b * (1 + s * tol)) + 127 for s in (-1, 1))
        assert ((byte == lo) | (byte == hi)).all()
        scale = ref.pow2(byte - 127).repeat_interleave(32, 1)[:, :cols]
        err = (ref.mx_values(*y) - want).abs()
        assert (err <= want.abs() * (2.0 ** -4 + 2 * tol) + 2.0 ** -10 * scale).all()
    else:
        err = (y.double() - want).abs()
        bound = want.abs() * (tol + ref.HALF[y.dtype]) + 1e-38
        assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 3, 515])
def test_rms_norm(rows, cols, dtype):
    if rows * cols > 5_000_000:
        rows = 6
    say(f"rms_norm {rows}x{cols} {dtype}")
    x, w = rand(1, rows, cols, dtype=dtype), rand(2, cols, dtype=dtype) + 1
    r = rand(3, rows, cols, dtype=dtype, std=3.0)
    for res in (None, r):
        want, h = ref.rms_norm(x, w, EPS, res)
        for out in (None, BF16, F32, "mxfp8"):
            got = nv.rms_norm(x, w, EPS, residual=res, out_dtype=out)
            if res is not None:
                got, s = got
                assert s.dtype == dtype
                # h in binary32, then rounded to the type
                assert ((s.double() - h).abs() <= h.abs() * (ref.U + ref.HALF[dtype] * (dtype == BF16))).all()
            assert isinstance(got, tuple) == (out == "mxfp8")
            check_y(got, want, cols)


def test_rms_norm_weight_types_strides_and_sum_in_place():
    big = rand(5, 40, 700)
    x, r = big[3:30, 8:520], big[5:32, 100:612]
    w = rand(6, 512, dtype=F32)
    want, h = ref.rms_norm(x, w, 1e-3, r)
    y, s = nv.rms_norm(x, w, 1e-3, residual=r)
    check_y(y, want, 512)
    odd = big[:, 1:514]  # rows at odd addresses
    y = nv.rms_norm(odd, rand(7, 513), 1e-3, out_dtype="mxfp8")
    check_y(y, ref.rms_norm(odd, rand(7, 513), 1e-3)[0], 513)
    for cols in (512, 20000):  # the long form reads its rows twice
        x, r = rand(8, 9, cols), rand(9, 9, cols)
        want, h = ref.rms_norm(x, torch.ones(cols, device="cuda"), 1e-3, r)
        apart, s = nv.rms_norm(x, torch.ones(cols, device="cuda"), 1e-3, residual=r)
        same, s2 = nv.rms_norm(x, torch.ones(cols, device="cuda"), 1e-3, residual=r, sum_out=r)
        assert s2.data_ptr() == r.data_ptr() and torch.equal(s, s2) and torch.equal(apart, same)


def test_rms_norm_special_rows():
    x = rand(11, 6, 1000, dtype=F32)
    x[0] = 0
    x[1, 7], x[2, 9] = float("nan"), float("inf")
    x[3] = 1e-30
    w = torch.ones(1000, device="cuda")
    y = nv.rms_norm(x, w, EPS)
    assert (y[0] == 0).all() and y[1].isnan().all()
    assert y[2, 9].isnan() and (y[2, :9] == 0).all()
    check_y(y[3:], ref.rms_norm(x[3:], w, EPS)[0], 1000)
    codes, scales = nv.rms_norm(x, w, EPS, out_dtype="mxfp8")
    assert (u8(scales)[0] == 0).all() and (codes[0].float() == 0).all()
    assert (u8(scales)[1] == 255).all()
    zero = nv.rms_norm(x[:1], w, 0.0)  # 0 / 0: the formula's NaN
    assert zero.isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 7, 1100])
def test_rms_norm_grad(rows, cols, dtype):
    if rows * cols > 5_000_000:
        rows = 70
    say(f"rms_norm_grad {rows}x{cols} {dtype}")
    dy, h, w = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype), rand(3, cols, dtype=dtype) + 1
    dh = rand(4, rows, cols, dtype=dtype)
    for S in (h, nv.quantize_mxfp8(h)):
        for d in (None, dh):
            dx, dw = nv.rms_norm_grad(dy, S, w, EPS, dS=d)
            rx, rw, ex, ew = ref.rms_norm_grad(dy, ref.value(S), w, EPS, d)
            assert dx.dtype == dtype and dw.dtype == F32
            assert ((dx.double() - rx).abs() <= ex + rx.abs() * ref.HALF[dtype] + 1e-38).all()
            assert ((dw.double() - rw).abs() <= ew + rw.abs() * ref.U).all()


def test_rms_norm_grad_by_differences():
    """Central differences of the forward kernel's loss sum(y dy) + sum(h dh), in fp32: a step t along a random
    direction moves the loss by t <gradient, direction> up to t^3; the forward's rounding (2^-20 of each
    term, adding like a random walk over 12000 terms) over 2 t bounds the rest."""
    rows, cols = 12, 1000
    x, r, dy, dh = (rand(20 + i, rows, cols, dtype=F32) for i in range(4))
    w = rand(25, cols, dtype=F32) + 1

    def loss(x, r, w):
        y, h = nv.rms_norm(x, w, EPS, residual=r)
        return ((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum()).item()

    _, h = nv.rms_norm(x, w, EPS, residual=r)
    dx, dw = nv.rms_norm_grad(dy, h, w, EPS, dS=dh)
    t = 2.0 ** -7
    for i, g in enumerate((dx, dx, dw)):
        v = rand(30 + i, *g.shape, dtype=F32)
        args = [[x, r, w], [x, r, w]]
        args[0][i], args[1][i] = args[0][i] + t * v, args[1][i] - t * v
        slope = (loss(*args[0]) - loss(*args[1])) / (2 * t)
        want = (g.double() * v.double()).sum().item()
        assert abs(slope - want) <= 2.0 ** -20 * 4 * (rows * cols) ** 0.5 / t + 1e-3 * abs(want) + 0.05


def test_rms_norm_grad_strides_and_types():
    big = rand(40, 60, 900)
    dy, h, d = big[1:50, 3:803], big[2:51, 50:850], big[5:54, 90:890]
    w = rand(41, 800, dtype=F32)
    dx, dw = nv.rms_norm_grad(dy, h, w, EPS, dS=d)
    rx, rw, ex, ew = ref.rms_norm_grad(dy, h, w, EPS, d)
    assert ((dx.double() - rx).abs() <= ex + rx.abs() * ref.HALF[BF16]).all()
    assert ((dw.double() - rw).abs() <= ew + rw.abs() * ref.U).all()


def test_no_rows():
    e = torch.empty(0, 96, dtype=BF16, device="cuda")
    w = torch.ones(96, dtype=BF16, device="cuda")
    codes, scales = nv.quantize_mxfp8(e)
    assert codes.shape == (0, 96) and scales.shape == (0, 3)
    assert nv.dequantize_mxfp8(codes, scales).shape == (0, 96)
    y, s = nv.rms_norm(e, w, residual=e)
    assert y.shape == s.shape == (0, 96)
    dx, dw = nv.rms_norm_grad(e, e, w)
    assert dx.shape == (0, 96) and (dw == 0).all()


def test_streams_and_graph_replays():
    rows, cols = 300, 1000
    x, r, dy = rand(50, rows, cols), rand(51, rows, cols), rand(52, rows, cols)
    w = rand(53, cols)

    def work(stream=None):
        y, s = nv.rms_norm(x, w, residual=r, out_dtype="mxfp8", stream=stream)
        k = nv.quantize_mxfp8(s, stream=stream)
        dx, dw = nv.rms_norm_grad(dy, k, w, dS=dy, stream=stream)
        return [u8(y[0]), u8(y[1]), s, u8(k[0]), nv.dequantize_mxfp8(*k, stream=stream), dx, dw]

    eager = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = work(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = work()
    for _ in range(4):
        for t in held:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
        work()  # eager work between replays
    torch.cuda.synchronize()


def test_refusals():
    x, w = rand(60, 4, 64), rand(61, 64)
    codes, scales = nv.quantize_mxfp8(x)
    bad = [
        lambda: nv.quantize_mxfp8(x.half()), lambda: nv.quantize_mxfp8(x.cpu()), lambda: nv.quantize_mxfp8(x[0]),
        lambda: nv.quantize_mxfp8(x.T), lambda: nv.quantize_mxfp8(x[:1].expand(4, 64)),
        lambda: nv.quantize_mxfp8(x[:, :0]),
        lambda: nv.dequantize_mxfp8(codes, scales[:3]), lambda: nv.dequantize_mxfp8(codes, scales.float()),
        lambda: nv.dequantize_mxfp8(codes, scales, torch.float16), lambda: nv.dequantize_mxfp8(x, scales),
        lambda: nv.rms_norm(x, w[:63]), lambda: nv.rms_norm(x, w.double()), lambda: nv.rms_norm(x, w, -1.0),
        lambda: nv.rms_norm(x, w, float("nan")), lambda: nv.rms_norm(x, w, residual=x.float()),
        lambda: nv.rms_norm(x, w, residual=x[:3]), lambda: nv.rms_norm(x, w, out_dtype=torch.float16),
        lambda: nv.rms_norm(x, w, sum_out=x), lambda: nv.rms_norm(x, w, residual=x, sum_out=x.T),
        lambda: nv.rms_norm_grad(x, x.float(), w), lambda: nv.rms_norm_grad(x, x[:3], w),
        lambda: nv.rms_norm_grad(x, (codes, scales[:, :1]), w), lambda: nv.rms_norm_grad(x, codes, w),
        lambda: nv.rms_norm_grad(x, x, w, dS=x.float()),
        lambda: nv.rms_norm_grad(x, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(nv.NVFP4Error):
            call()
            say(f"call {i} was not refused")


def test_rms_norm_squares_past_binary32():
    """The sum of a row's squares overflows: its y is 0, and the rows beside it are what they are alone."""
    x = rand(12, 3, 1000)
    x[1] = torch.finfo(BF16).min
    w, dy = torch.ones(1000, device="cuda"), rand(13, 3, 1000)
    y = nv.rms_norm(x, w, EPS)
    assert (y[1] == 0).all()
    check_y(y[::2], ref.rms_norm(x[::2], w, EPS)[0], 1000)
    dx, dw = nv.rms_norm_grad(dy, x, w, EPS)
    alone = nv.rms_norm_grad(dy[:1], x[:1], w, EPS)[0], nv.rms_norm_grad(dy[2:], x[2:], w, EPS)[0]
    assert torch.equal(dx[:1], alone[0]) and torch.equal(dx[2:], alone[1])
