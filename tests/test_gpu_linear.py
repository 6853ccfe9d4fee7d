"""Products with NVFP4 weights and an epilogue, their gradients, and a layer's operators run together, on the GPU
against binary64 (tests/layer_ref.py).

Tolerances: products are exact and summed in fp32, so a sum of L terms is off by at most L 2^-23 of the sum of
their magnitudes; the epilogue's own roundings are counted in layer_ref; an output adds half a step of its
type. One-hot inputs leave one product per output: those cases are exact, and show every value at its
place. dX is held to the product of the dZ that came with it."""
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
    """Every code and a wide range of scales, not the quantiser's alone."""
    g = torch.Generator(device="cuda").manual_seed(n * 31 + k + seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(0x10, 0x60, (n, k // 16), generator=g, device="cuda").to(torch.uint8)
    return codes, scales, torch.full((1,), 0.0123, device="cuda")


def kinds(x):
    return x, nv.quantize_mxfp8(x)


def u8(t):
    return t.view(torch.uint8)


def check(y, want, err):
    bound = err + want.abs() * ref.HALF[y.dtype] + 1e-38
    bad = (y.double() - want).abs() - bound
    assert (bad <= 0).all(), float(bad.max())


def check_kept(Z, want, err):
    if not isinstance(Z, tuple):
        check(Z, want, err)
        return
    cols = want.shape[1]
    top = ref.mx_blocks(want).abs().amax(-1)
    slack = ref.mx_blocks(err).amax(-1)
    byte = u8(Z[1]).to(torch.int64)
    lo, hi = (ref.mx_scale_exp((top + s * slack).clamp_min(0)) + 127 for s in (-1, 1))
    assert ((byte >= lo) & (byte <= hi)).all()
    scale = ref.pow2(byte - 127).repeat_interleave(32, 1)[:, :cols]
    off = (ref.mx_values(*Z) - want).abs()
    assert (off <= want.abs() * 2.0 ** -4 + 2.0 ** -10 * scale + 2 * err).all()


# (M, N, K): the skinny kernel (M <= 64) with each count of its row tiles; the tile kernel at each height (the last
# four: 256-row, 128-row and 256-row tiles, and wide outputs), K split and not; odd N, K of 16 mod 32 and mod 64
SHAPES = [(1, 256, 1024), (1, 16, 16), (2, 7, 48), (5, 96, 272), (16, 130, 4112), (17, 33, 512), (33, 64, 2064),
          (48, 17, 160), (64, 100, 8208), (65, 40, 320), (100, 256, 1024), (130, 260, 528), (300, 520, 96),
          (257, 1000, 4176), (32800, 256, 80), (51300, 200, 48), (300, 25601, 112), (2100, 6400, 64)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_matches_binary64(m, n, k):
    W = make_weights(n, k)
    X = rand(m + n, m, k)
    say(f"linear M={m} N={n} K={k}")
    for x in kinds(X):
        v = ref.value(x)
        for out, bias, act, res, keep in (
                (F32, None, None, None, None),
                (BF16, rand(1, n, dtype=F32), "silu", None, BF16),
                (BF16, rand(2, n), "gelu", rand(3, m, n), "mxfp8"),
                (F32, None, "gelu", rand(4, m, n, dtype=F32), None)):
            y, z, ey, ez = ref.linear(v, *W, bias=bias, act=act, res=res)
            got = nv.linear(x, *W, bias=bias, activation=act, residual=res, out_dtype=out, keep=keep)
            if keep is not None:
                got, Z = got
                check_kept(Z, z, ez)
            assert got.dtype == out
            check(got, y, ey)


GATED = [(1, 64, 1024), (3, 34, 48), (20, 512, 272), (40, 96, 528), (64, 1030, 2064), (70, 258, 320), (300, 512, 1040),
         (32800, 128, 80), (51300, 192, 48), (300, 25602, 112)]


@pytest.mark.parametrize("m,n,k", GATED)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_linear_matches_binary64(m, n, k, act):
    W = make_weights(n, k)
    X = rand(m + n, m, k)
    say(f"gated M={m} N={n} K={k} {act}")
    for x in kinds(X):
        v = ref.value(x)
        for out, bias, res, keep in ((F32, None, None, None), (BF16, rand(1, n), rand(2, m, n // 2), BF16),
                                     (BF16, None, None, "mxfp8")):
            if keep == "mxfp8" and n % 64:
                with pytest.raises(nv.NVFP4Error):
                    nv.linear(x, *W, activation=act, gated=True, keep=keep)
                continue
            y, z, ey, ez = ref.linear(v, *W, bias=bias, act=act, gated=True, res=res)
            got = nv.linear(x, *W, bias=bias, activation=act, gated=True, residual=res, out_dtype=out, keep=keep)
            if keep is not None:
                got, Z = got
                check_kept(Z, z, ez)
            check(got, y, ey)


MANY = [(9000, 4352, 2064), (12300, 4352, 1040)]  # weights decoded first; more than a round of tall tiles


@pytest.mark.parametrize("m,n,k", MANY)
def test_many_rows(m, n, k):
    """The forms for many rows of X (the weights decoded before the product, the last columns of tiles at half the
    height), forward plain, with every extra and gated, and the gradient; each output against binary64."""
    W = make_weights(n, k)
    Wv, alpha = ref.weights(*W[:2]), float(W[2])
    X = rand(1, m, k)
    assert nv.linear_workspace_bytes(m, k, n) >= 2 * n * k  # decoded weights
    say(f"many M={m} N={n} K={k}")
    y, z, ey, ez = ref.linear(X.double(), *W)
    check(nv.linear(X, *W), y, ey)
    bias, res = rand(2, n), rand(3, m, n)
    y, z, ey, ez = ref.linear(X.double(), *W, bias=bias, act="gelu", res=res)
    got, Z = nv.linear(X, *W, bias=bias, activation="gelu", residual=res, keep="mxfp8")
    check(got, y, ey)
    check_kept(Z, z, ez)
    del y, z, ey, ez, got, Z
    x8 = nv.quantize_mxfp8(X)
    y, z, ey, ez = ref.linear(ref.value(x8), *W, act="silu", gated=True)
    got, Z = nv.linear(x8, *W, activation="silu", gated=True, keep=BF16)
    check(got, y, ey)
    check(Z, z, ez)
    del y, z, ey, ez, got, Z
    dy = rand(4, m, n)
    dX, _, db = nv.linear_grad(dy, *W, bias=True)
    check(dX, alpha * (dy.double() @ Wv), ref.product_error(dy.double(), Wv.T, alpha, n))
    assert ((db.double() - dy.double().sum(0)).abs() <= (m + 8) * ref.U * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("n,k", [(96, 64), (200, 176), (256, 512), (300, 1040)])
def test_one_hot_rows_are_exact(n, k):
    """X = I, repeated: each output is one weight times alpha, rounded once."""
    W = make_weights(n, k)
    want = ((ref.weights(*W[:2]).float() * W[2]).T).contiguous()
    eye = torch.eye(k, device="cuda").to(BF16)
    each = torch.arange(k, device="cuda")
    for at in (each[:9], each[k // 2:k // 2 + 40], each, each.repeat(3)):
        for x in kinds(eye[at].contiguous()):
            assert torch.equal(nv.linear(x, *W, out_dtype=F32), want[at])
    wide = torch.zeros(34000, k, dtype=BF16, device="cuda")  # the taller tiles
    at = torch.arange(34000, device="cuda") % k
    wide[torch.arange(34000, device="cuda"), at] = 1
    assert torch.equal(nv.linear(wide, *W, out_dtype=F32), want[at])


@pytest.mark.parametrize("n,k", [(96, 64), (77, 176), (256, 512), (1030, 304)])
def test_one_hot_gradients_are_exact(n, k):
    W = make_weights(n, k)
    want = (ref.weights(*W[:2]).float() * W[2]).to(BF16)
    at = torch.arange(700, device="cuda") % n
    for m in (1, 30, 700):
        dy = torch.zeros(m, n, dtype=BF16, device="cuda")
        dy[torch.arange(m, device="cuda"), at[:m]] = 1
        assert torch.equal(nv.linear_grad(dy, *W)[0], want[at[:m]])


# One more column of tiles than whole rounds of work-groups take: it runs by itself, with K split. Columns that end
# inside a tile and inside eight, gated or not; weights as stored and decoded first.
REST = [(1500, 10843, 1040, False), (1500, 10944, 1040, False), (1500, 10944, 1040, True), (1500, 10946, 1040, True),
        (2050, 3984, 2064, False)]


@pytest.mark.parametrize("m,n,k,gated", REST)
def test_last_columns_alone(m, n, k, gated):
    F = n // 2 if gated else n
    W = make_weights(n, k)
    say(f"rest M={m} N={n} K={k} {gated}")
    X, bias, res = rand(1, m, k), rand(2, n), rand(3, m, F)
    act = "silu" if gated else None
    y, z, ey, ez = ref.linear(X.double(), *W, act=act, gated=gated)
    check(nv.linear(X, *W, activation=act, gated=gated), y, ey)
    y, z, ey, ez = ref.linear(X.double(), *W, bias=bias, act="gelu", gated=gated, res=res)
    for keep in (BF16, "mxfp8"):
        if keep == "mxfp8" and gated and F % 32:
            continue
        got, Z = nv.linear(X, *W, bias=bias, activation="gelu", gated=gated, residual=res, keep=keep)
        check(got, y, ey)
        check_kept(Z, z, ez) if keep == "mxfp8" else check(Z, z, ez)
    need = nv.linear_workspace_bytes(m, k, n, gated)
    assert need > 0
    space = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")  # a call stays inside its workspace
    off = -space.data_ptr() % 256
    again = nv.linear(X, *W, bias=bias, activation="gelu", gated=gated, residual=res, workspace=space[off:off + need])
    assert torch.equal(again, got) and (space[off + need:] == 0x5A).all()


@pytest.mark.parametrize("m,n,k", [(1500, 2064, 10992), (4100, 272, 4128)])
def test_last_columns_alone_gradient(m, n, k):
    W = make_weights(n, k)
    Wv, alpha = ref.weights(*W[:2]), float(W[2])
    dy = rand(4, m, n)
    say(f"rest gradient M={m} N={n} K={k}")
    dX, _, db = nv.linear_grad(dy, *W, bias=True)
    check(dX, alpha * (dy.double() @ Wv), ref.product_error(dy.double(), Wv.T, alpha, n))
    assert ((db.double() - dy.double().sum(0)).abs() <= (m + 8) * ref.U * dy.double().abs().sum(0)).all()
    x, held = rand(5, m, k), None
    work = lambda: (nv.linear(x, *W), nv.linear_grad(dy, *W)[0])  # noqa: E731
    eager = work()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = work()
    for _ in range(3):
        for t in held:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager))
        work()


GRADS = [(1, 256, 1024), (1, 1, 16), (5, 7, 48), (33, 130, 272), (64, 64, 2064), (100, 1001, 176), (300, 520, 96),
         (130, 4100, 528), (32800, 80, 256), (51300, 48, 208), (300, 112, 25600), (2100, 64, 6400)]


@pytest.mark.parametrize("m,n,k", GRADS)
@pytest.mark.parametrize("act,gated", [(None, False), ("silu", False), ("gelu", False), ("silu", True), ("gelu", True)])
def test_linear_grad_matches_binary64(m, n, k, act, gated):
    n = (n + 31) // 32 * 64 if gated else n
    F = n // 2 if gated else n
    W = make_weights(n, k)
    Wv, alpha = ref.weights(*W[:2]), float(W[2])
    dy, z = rand(m, m, F), rand(m + 1, m, n, std=2.0)
    say(f"linear_grad M={m} N={n} K={k} {act} {gated}")
    for Z in (kinds(z) if act else (None,)):
        for bias in (False, True):
            dX, dZ, db = nv.linear_grad(dy, *W, Z=Z, activation=act, gated=gated, bias=bias)
            dz, edz = ref.linear_dz(dy.double(), ref.value(Z) if act else None, act, gated)
            if act:
                check(dZ, dz, edz)
            else:
                assert dZ is None
            used = (dZ if act else dy).double()
            check(dX, alpha * (used @ Wv), ref.product_error(used, Wv.T, alpha, n))
            assert (db is not None) == bias
            if bias:
                off = (db.double() - dz.sum(0)).abs()
                assert (off <= edz.sum(0) + (m + 8) * ref.U * dz.abs().sum(0)).all()


def test_linear_grad_by_differences():
    """Central differences of the forward kernel (fp32 output), inputs moved by 2^-5 along signs, all of them exact in
    bf16. z moves by about 0.01, so the cubic term is below 1e-4 of the slope; the forward's rounding, 2^-18 of
    a term, is divided by the 2^-4 between the two points; dX and dZ are rounded to bf16."""
    m, F, k = 20, 96, 256
    g = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randint(-48, 49, (m, k), generator=g, device="cuda") / 16).to(BF16)
    codes, scales, alpha = nv.quantize(rand(6, 2 * F, k, std=0.05), "4o6")
    dy = rand(7, m, F)
    v = torch.randint(0, 2, (m, k), generator=g, device="cuda") * 2.0 - 1
    t = 2.0 ** -5
    for act, gated in ((None, False), ("silu", False), ("gelu", True)):
        W = (codes, scales, alpha) if gated else (codes[:F].contiguous(), scales[:F].contiguous(), alpha)
        kw = dict(activation=act, gated=gated)
        _, Z = nv.linear(x, *W, keep=BF16, **kw)
        dX, _, _ = nv.linear_grad(dy, *W, Z=Z if act else None, **kw)
        up, down = ((x.float() + s * t * v).to(BF16) for s in (1, -1))
        assert torch.equal(up.float(), x.float() + t * v)
        y1, y0 = (nv.linear(p, *W, out_dtype=F32, **kw).double() for p in (up, down))
        slope = ((y1 - y0) * dy.double()).sum(1) / (2 * t)
        want = (dX.double() * v.double()).sum(1)
        scale = (dX.double().abs()).sum(1)
        assert ((slope - want).abs() <= 2.0 ** -7 * scale).all()


def test_strides_in_place_residual_and_workspaces():
    W = make_weights(200, 272)
    big = rand(8, 90, 900)
    for m in (20, 80):
        x = big[:m, 5:277]
        assert torch.equal(nv.linear(x, *W), nv.linear(x.contiguous(), *W))
        r = big[2:m + 2, 301:501]
        y = nv.linear(x, *W, residual=r)
        same = r.contiguous()
        assert nv.linear(x, *W, residual=same, out=same) is same and torch.equal(same, y)
        codes, scales = nv.quantize_mxfp8(x)
        wide = torch.zeros(m, 400, dtype=torch.uint8, device="cuda")
        wide[:, 3:275] = u8(codes)
        assert torch.equal(nv.linear((wide[:, 3:275], u8(scales)), *W), nv.linear((codes, scales), *W))
        dy, z = big[:m, 7:207], big[:m, 401:601]
        a = nv.linear_grad(dy, *W, Z=z, activation="gelu", bias=True)
        b = nv.linear_grad(dy.contiguous(), *W, Z=z.contiguous(), activation="gelu", bias=True)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        assert torch.equal(nv.linear_grad(dy, *W)[0], nv.linear_grad(dy.contiguous(), *W)[0])
    # a guarded workspace: exactly its bytes are used
    x = rand(9, 100, 1024)
    W = make_weights(256, 1024)
    for need, call in ((nv.linear_workspace_bytes(100, 1024, 256), lambda w: nv.linear(x, *W, workspace=w)),
                       (nv.linear_grad_workspace_bytes(100, 1024, 256, bias=True),
                        lambda w: nv.linear_grad(x[:, :256], *W, bias=True, workspace=w)[0])):
        assert need > 0
        buf = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(buf[:need]), call(None))
        assert (buf[need:] == 0xAB).all()


def test_rows_behind_the_last_are_left():
    """Outputs stay inside their rows: guards after the last row of every output of a ragged call."""
    W = make_weights(100, 160)
    for m in (3, 70):
        x = rand(m, m, 160)
        buf = torch.full((m + 1, 100), 7.0, dtype=BF16, device="cuda")
        nv.linear(x, *W, out=buf[:m])
        assert (buf[m] == 7.0).all()


def test_not_finite_inputs_stay_in_their_rows():
    W = make_weights(300, 208)
    for m in (8, 90):
        x = rand(m, m, 208)
        clean = nv.linear(x, *W)
        bad = x.clone()
        bad[2, 100], bad[5, 207] = float("nan"), float("inf")
        y = nv.linear(bad, *W)
        keep = torch.ones(m, dtype=torch.bool, device="cuda")
        keep[2] = keep[5] = False
        assert torch.equal(y[keep], clean[keep])
        assert y[2].isnan().all() and not y[5].isfinite().any()
        codes, scales = nv.quantize_mxfp8(bad)
        y8 = nv.linear((codes, scales), *W)
        assert y8[2].isnan().all() and y8[5].isnan().all() and y8[keep].isfinite().all()
        y, Z = nv.linear(bad, *W, activation="silu", keep="mxfp8")
        assert (u8(Z[1])[2] == 255).all() and (u8(Z[1])[keep] != 255).all()


def test_no_rows():
    W = make_weights(64, 96)
    e = torch.empty(0, 96, dtype=BF16, device="cuda")
    y, Z = nv.linear(e, *W, activation="silu", gated=True, keep="mxfp8")
    assert y.shape == (0, 32) and Z[0].shape == (0, 64) and Z[1].shape == (0, 2)
    dX, dZ, db = nv.linear_grad(y, *W, Z=Z, activation="silu", gated=True, bias=True)
    assert dX.shape == (0, 96) and dZ.shape == (0, 64) and (db == 0).all() and db.shape == (64,)


def layer(x, r, wn, W1, W2, dy, stream=None):
    """A feed-forward layer as it is used: residual and norm to 8 bits, gated product with its z kept in 8 bits,
    product with the residual; and all of it backward, from the 8-bit copies."""
    h8, s = nv.rms_norm(x, wn, residual=r, out_dtype="mxfp8", stream=stream)
    a, Z = nv.linear(h8, *W1, activation="silu", gated=True, keep="mxfp8", stream=stream)
    y = nv.linear(a, *W2, residual=s, stream=stream)
    s8 = nv.quantize_mxfp8(s, stream=stream)
    da, _, _ = nv.linear_grad(dy, *W2, stream=stream)
    dh, dz, db = nv.linear_grad(da, *W1, Z=Z, activation="silu", gated=True, bias=True, stream=stream)
    dx, dw = nv.rms_norm_grad(dh, s8, wn, dS=dy, stream=stream)
    return h8, s, a, Z, y, s8, da, dh, dz, db, dx, dw


@pytest.mark.parametrize("m", [1, 9, 300])
def test_layer_together(m):
    """Each step against its formula on what the step before gave; and the gradient of the whole against binary64
    with the same 8-bit values, where every product rounds to bf16 once (dh, dz, da: three steps of 2^-8)."""
    d, F = 256, 320
    x, r, dy = rand(1, m, d), rand(2, m, d, std=2.0), rand(3, m, d)
    wn = rand(4, d) + 1
    W1, W2 = (nv.quantize(rand(5 + i, n, k, std=0.05), "4o6") for i, (n, k) in enumerate(((2 * F, d), (d, F))))
    h8, s, a, Z, y, s8, da, dh, dz, db, dx, dw = layer(x, r, wn, W1, W2, dy)
    h, hs = ref.rms_norm(x, wn, 1e-6, r)
    assert ((ref.value(h8) - h).abs() <= h.abs() * 0.0626 + 2.0 ** -10 * ref.mx_blocks(h).abs().amax() / 224).all()
    ya, z, ea, ez = ref.linear(ref.value(h8), *W1, act="silu", gated=True)
    check(a, ya, ea)
    check_kept(Z, z, ez)
    yy, _, ey, _ = ref.linear(a.double(), *W2, res=s)
    check(y, yy, ey)
    da64 = dy.double() @ (ref.weights(*W2[:2]) * float(W2[2]))
    dz64, _ = ref.linear_dz(da64, ref.value(Z), "silu", True)
    dh64 = dz64 @ (ref.weights(*W1[:2]) * float(W1[2]))
    dx64, dw64, _, _ = ref.rms_norm_grad(dh64, ref.value(s8), wn, 1e-6, dy)
    for got, want in ((da, da64), (dz, dz64), (dh, dh64), (dx, dx64), (dw, dw64), (db, dz64.sum(0))):
        assert (got.double() - want).norm() <= 4 * 2.0 ** -8 * want.norm() + 1e-30


def test_layer_on_streams_and_in_graphs():
    d, F = 512, 704
    W1, W2 = (nv.quantize(rand(15 + i, n, k, std=0.05), "4o6") for i, (n, k) in enumerate(((2 * F, d), (d, F))))
    wn = rand(14, d) + 1
    flat = lambda out: [q.view(torch.uint8) if q.element_size() == 1 else q  # noqa: E731
                        for t in out for q in (t if isinstance(t, tuple) else (t,))]
    for m in (3, 200):
        x, r, dy = rand(11, m, d), rand(12, m, d), rand(13, m, d)
        eager = flat(layer(x, r, wn, W1, W2, dy))
        torch.cuda.synchronize()
        sides = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for side in sides:  # two at once
            side.wait_stream(torch.cuda.current_stream())
            got.append(flat(layer(x, r, wn, W1, W2, dy, stream=side)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, eager))
        graphs, held = [], []
        for _ in range(2):  # two graphs with scratch of their own
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                held.append(flat(layer(x, r, wn, W1, W2, dy)))
            graphs.append(g)
        for _ in range(3):
            for g, h in zip(graphs, held):
                for t in h:
                    t.zero_()
                g.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(h, eager))
                layer(x, r, wn, W1, W2, dy)  # eager work between replays
        torch.cuda.synchronize()


def test_many_rows_in_graphs():
    """Captured calls of the tall tiles, the decoding before them and the split sums give the eager results on every
    replay."""
    for m, n, k in ((2600, 4352, 1040), (12300, 4352, 1040), (700, 512, 2048)):
        W = make_weights(n, k)
        x, dy = rand(1, m, k), rand(2, m, n)
        work = lambda: (nv.linear(x, *W), nv.linear_grad(dy, *W)[0])  # noqa: E731
        eager = work()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = work()
        for _ in range(3):
            for t in held:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, eager))
            work()
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """X, Y, dY and dX of more than 2^31 values: the last rows equal those of a call of their own."""
    m, k, n = 525_000, 4112, 48
    W = make_weights(n, k)
    x = torch.zeros(m, k, dtype=BF16, device="cuda")
    x[-300:] = rand(1, 300, k)
    assert x.numel() > 2 ** 31
    y = nv.linear(x, *W)
    want, _, ey, _ = ref.linear(x[-300:].double(), *W)
    check(y[-300:], want, ey)
    assert (y[:-300] == 0).all()
    dy = torch.zeros(m, n, dtype=BF16, device="cuda")
    dy[-300:] = rand(2, 300, n)
    dX, _, _ = nv.linear_grad(dy, *W)
    Wv, alpha = ref.weights(*W[:2]), float(W[2])
    d = dy[-300:].double()
    check(dX[-300:], alpha * (d @ Wv), ref.product_error(d, Wv.T, alpha, n))
    del dX, y, dy
    s8 = nv.quantize_mxfp8(x)
    q, b = ref.mx_quantize(x[-300:].double())
    assert torch.equal(s8[0][-300:].double(), q) and torch.equal(u8(s8[1])[-300:], b)
    h, s = nv.rms_norm(x, torch.ones(k, device="cuda"), 1e-3, residual=x, out_dtype="mxfp8")
    h1, s1 = nv.rms_norm(x[-300:], torch.ones(k, device="cuda"), 1e-3, residual=x[-300:], out_dtype="mxfp8")
    assert torch.equal(s[-300:], s1) and torch.equal(u8(h[0])[-300:], u8(h1[0])) and torch.equal(u8(h[1])[-300:], u8(h1[1]))
    del h, s
    dx, dw = nv.rms_norm_grad(x, s8, torch.ones(k, device="cuda"), 1e-3)
    dx1, dw1 = nv.rms_norm_grad(x[-300:], (s8[0][-300:], s8[1][-300:]), torch.ones(k, device="cuda"), 1e-3)
    assert torch.equal(dx[-300:], dx1) and torch.allclose(dw, dw1, rtol=1e-4, atol=1e-4)


def test_refusals():
    W = make_weights(64, 96)
    x, dy = rand(1, 4, 96), rand(2, 4, 64)
    c, s, a = W
    x8 = nv.quantize_mxfp8(x)
    z = rand(3, 4, 64)
    bad = [
        lambda: nv.linear(x.float(), *W), lambda: nv.linear(x[:, :80], *W), lambda: nv.linear(x.cpu(), *W),
        lambda: nv.linear(x8[0], *W), lambda: nv.linear((x8[0], x8[1][:, :2]), *W), lambda: nv.linear((x, x8[1]), *W),
        lambda: nv.linear(x, c[:, :4], s, a), lambda: nv.linear(x, c, s[:60], a), lambda: nv.linear(x, c, s, a.double()),
        lambda: nv.linear(x, c.cpu(), s, a), lambda: nv.linear(x, *W, bias=rand(1, 63)),
        lambda: nv.linear(x, *W, bias=rand(1, 64).half()), lambda: nv.linear(x, *W, activation="relu"),
        lambda: nv.linear(x, *W, gated=True), lambda: nv.linear(x, c[:63], s[:63], a, activation="silu", gated=True),
        lambda: nv.linear(x, *W, residual=rand(1, 4, 63)), lambda: nv.linear(x, *W, residual=rand(1, 3, 64)),
        lambda: nv.linear(x, *W, activation="silu", gated=True, residual=rand(1, 4, 64)),
        lambda: nv.linear(x, *W, out_dtype=torch.float16), lambda: nv.linear(x, *W, keep=F32),
        lambda: nv.linear(x, *W, out=rand(1, 4, 63)), lambda: nv.linear(x, *W, out=rand(1, 4, 64, dtype=F32)),
        lambda: nv.linear_grad(dy.float(), *W), lambda: nv.linear_grad(dy[:, :32], *W),
        lambda: nv.linear_grad(dy, *W, Z=z), lambda: nv.linear_grad(dy, *W, activation="silu"),
        lambda: nv.linear_grad(dy, *W, Z=z[:3], activation="silu"),
        lambda: nv.linear_grad(dy, *W, Z=z, activation="silu", gated=True),
        lambda: nv.linear_grad(dy, *W, Z=z.float(), activation="silu"),
        lambda: nv.linear_grad(dy, *W, bias=True, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: nv.linear(rand(1, 100, 96), *make_weights(64, 96), keep="mxfp8", activation="silu",
                          workspace=torch.empty(0, dtype=torch.uint8)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(nv.NVFP4Error):
            call()
            say(f"call {i} was not refused")


def test_graphs_that_share_a_workspace():
    """Calls captured into two graphs with one workspace, replayed in turn: each writes what it reads of it."""
    m, n, k = 700, 512, 2048  # K split forward and backward
    W = make_weights(n, k)
    x, dy, w = rand(1, m, k), rand(2, m, n), torch.ones(k, device="cuda")
    need = max(nv.linear_workspace_bytes(m, k, n), nv.linear_grad_workspace_bytes(m, k, n, bias=True),
               nv.rms_norm_grad_workspace_bytes(m, k))
    assert nv.linear_workspace_bytes(m, k, n) > 0
    space = torch.empty(need, dtype=torch.uint8, device="cuda")

    def work(scale):
        a, b = x * scale, dy * scale
        return (nv.linear(a, *W, workspace=space), *nv.linear_grad(b, *W, bias=True, workspace=space)[::2],
                *nv.rms_norm_grad(a, x, w, workspace=space))

    graphs = []
    for scale in (1.0, -3.0):
        eager = work(scale)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = work(scale)
        graphs.append((g, held, eager))
    for _ in range(3):
        for g, held, eager in graphs:
            for t in held:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(held, eager))
        work(2.0)
    torch.cuda.synchronize()
