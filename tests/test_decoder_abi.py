"""The C entry points of rotary positions, the cache and its attention refuse bad arguments on the host, before
anything touches a device, and the binding's structs have the C compiler's layout (CPU only: no call here enqueues
anything)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from nvfp4_block_scaled_elem_amd import build as nvbuild
from nvfp4_block_scaled_elem_amd import decoder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -3
FAKE = 0x100000  # never dereferenced: every call below fails validation first, or has no rows


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        nvbuild.build()
    return nv.lib()


@pytest.mark.parametrize("kw,err", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(positions=None), INVALID), (dict(dtype=2), INVALID),
    (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID), (dict(axes=0), INVALID),
    (dict(axes=5), INVALID), (dict(inverse=2), INVALID), (dict(positions64=2), INVALID), (dict(base=0.0), INVALID),
    (dict(base=-1.0), INVALID), (dict(base=float("nan")), INVALID), (dict(base=float("inf")), INVALID),
    (dict(sections=(0, 0, 0, 0)), INVALID), (dict(sections=(-1, 0, 0, 0)), INVALID), (dict(sections=(33, 0, 0, 0)), SHAPE),
    (dict(axes=2, sections=(20, 13, 0, 0)), SHAPE), (dict(axes=2, sections=(1 << 30, 1 << 30, 0, 0)), INVALID),
    (dict(tokens=(1 << 23) + 1), SHAPE), (dict(heads=65536), SHAPE), (dict(dim=257, xs=600, ys=600, xh=257, yh=257), SHAPE),
    (dict(xs=63), INVALID), (dict(ys=63), INVALID), (dict(xh=63), INVALID), (dict(yh=63), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(y=FAKE + 1), INVALID), (dict(positions=FAKE + 2), INVALID),
    (dict(positions=FAKE + 4, positions64=1), INVALID), (dict(dtype=1, x=FAKE + 2), INVALID),
    (dict(x=2 * FAKE, ys=192), INVALID), (dict(tokens=0), OK), (dict(tokens=0, x=None), OK),
])
def test_rotary_rejects(L, kw, err):
    a = decoder._RotaryArgs(x=FAKE, xs=128, xh=64, y=2 * FAKE, ys=128, yh=64, tokens=4, heads=2, dim=64, positions=FAKE,
                            axes=1, sections=(32, 0, 0, 0), base=10000.0)
    for k, v in kw.items():
        setattr(a, k, (ctypes.c_int * 4)(*v) if k == "sections" else v)
    assert L.nvfp4_rotary(ctypes.byref(a)) == err


def cache_args(**kw):
    c = decoder._Cache(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, pages=10, kv_heads=2, dim=64)
    s = decoder._Sequences(table=FAKE, ldt=8, lengths=FAKE, starts=FAKE, seqs=4, width=8)
    for k, v in kw.items():
        setattr(c if hasattr(c, k) else s, k, v)
    return ctypes.byref(c), ctypes.byref(s)


CACHE = [
    (dict(k_codes=None), INVALID), (dict(v_codes=None), INVALID), (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID),
    (dict(pages=0), INVALID), (dict(pages=-1), INVALID), (dict(pages=1 << 31), SHAPE), (dict(kv_heads=0), INVALID),
    (dict(kv_heads=65536), SHAPE), (dict(dim=0), INVALID), (dict(dim=24), SHAPE), (dict(dim=272), SHAPE),
    (dict(table=None), INVALID), (dict(lengths=None), INVALID), (dict(ldt=7), INVALID), (dict(width=0), INVALID),
    (dict(width=-1), INVALID), (dict(width=(1 << 24) + 1, ldt=1 << 25), SHAPE), (dict(seqs=-1), INVALID),
    (dict(starts=None), INVALID), (dict(starts=FAKE + 2), INVALID), (dict(table=FAKE + 2), INVALID),
    (dict(lengths=FAKE + 2), INVALID), (dict(k_codes=FAKE + 8), INVALID), (dict(v_codes=FAKE + 8), INVALID),
    (dict(seqs=(1 << 23) + 1), SHAPE), (dict(seqs=0), OK),
]


@pytest.mark.parametrize("kw,err", CACHE)
def test_cache_is_checked(L, kw, err):
    cache, seqs = cache_args(**kw)
    c = cache._obj
    st = max(c.dim, 1)
    append = L.nvfp4_kv_append(cache, seqs, FAKE, st * c.kv_heads, st, FAKE, st * c.kv_heads, st, 0, 9, None)
    assert append == err
    heads = max(c.kv_heads, 1)
    assert L.nvfp4_attention(cache, seqs, FAKE, st * heads, st, heads, 9, 1.0, 1, FAKE, FAKE, 1 << 40, None) == err


def test_append_rejects(L):
    cache, seqs = cache_args()

    def call(k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, dtype=0, tokens=9):
        return L.nvfp4_kv_append(cache, seqs, k, kt, kh, v, vt, vh, dtype, tokens, None)

    for kw in (dict(k=None), dict(v=None), dict(kt=63), dict(kh=63), dict(vt=63), dict(vh=63), dict(dtype=2),
               dict(tokens=-1), dict(k=FAKE + 1), dict(v=FAKE + 1), dict(dtype=1, k=FAKE + 2)):
        assert call(**kw) == INVALID, kw
    assert call(tokens=(1 << 23) + 1) == SHAPE and call(tokens=0) == OK and call(tokens=0, k=None) == OK
    assert L.nvfp4_kv_append(None, seqs, FAKE, 128, 64, FAKE, 128, 64, 0, 9, None) == INVALID
    assert L.nvfp4_kv_append(cache, None, FAKE, 128, 64, FAKE, 128, 64, 0, 9, None) == INVALID


def test_attention_rejects(L):
    cache, seqs = cache_args()

    def call(q=FAKE, qt=256, qh=64, heads=4, tokens=9, scale=1.0, causal=1, out=FAKE, ws=FAKE, n=1 << 40):
        return L.nvfp4_attention(cache, seqs, q, qt, qh, heads, tokens, scale, causal, out, ws, n, None)

    for kw in (dict(q=None), dict(out=None), dict(qt=63), dict(qh=63), dict(heads=3), dict(heads=0), dict(heads=-2),
               dict(tokens=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(q=FAKE + 1),
               dict(out=FAKE + 8), dict(ws=FAKE + 16)):
        assert call(**kw) == INVALID, kw
    assert call(tokens=(1 << 23) + 1) == SHAPE and call(heads=65536) == SHAPE and call(tokens=0) == OK
    need = L.nvfp4_attention_workspace_bytes(9, 4, 80, 4, 2, 64)
    long = decoder._Sequences(table=FAKE, ldt=80, lengths=FAKE, starts=FAKE, seqs=4, width=80)
    assert need > 0
    assert L.nvfp4_attention(cache, ctypes.byref(long), FAKE, 256, 64, 4, 9, 1.0, 1, FAKE, FAKE, need - 1, None) == WORKSPACE
    assert L.nvfp4_attention_workspace_bytes(9, 4, 8, 4, 2, 64) == 0  # a short table: no parts
    assert L.nvfp4_attention_workspace_bytes(0, 4, 8, 4, 2, 64) == 0
    assert L.nvfp4_attention_workspace_bytes(9, 4, 8, 3, 2, 64) == 0  # no such call
    assert L.nvfp4_attention_workspace_bytes(9, 4, 8, 4, 2, 24) == 0
    # more pieces than a grid takes, and lists of blocks longer than their 32-bit numbers
    wide = decoder._Sequences(table=FAKE, ldt=1 << 24, lengths=FAKE, starts=FAKE, seqs=1 << 20, width=1 << 24)
    assert L.nvfp4_attention(cache, ctypes.byref(wide), FAKE, 256, 64, 4, 9, 1.0, 1, FAKE, FAKE, 1 << 40, None) == SHAPE


@pytest.mark.parametrize("name,struct", [("nvfp4_rotary_args_t", decoder._RotaryArgs), ("nvfp4_kv_cache_t", decoder._Cache),
                                         ("nvfp4_sequences_t", decoder._Sequences),
                                         ("nvfp4_moe_args_t", decoder._MoeArgs)])
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


@pytest.mark.parametrize("args,pack", [(decoder._RotaryArgs, decoder._rotary_args), (decoder._Cache, decoder._cache_args),
                                       (decoder._Sequences, decoder._sequences_args), (decoder._MoeArgs, decoder._moe_args)])
def test_packed_arguments(args, pack):
    """The bytes that the binding passes are those of the structure."""
    values, fields = [], {}
    for i, (name, kind) in enumerate(args._fields_):
        v = [-2.5 * i] if kind is ctypes.c_double else [3 * i + k + 1 for k in range(4)] if kind is decoder._Sections else [1 << 20 | i]
        values += v
        fields[name] = kind(*v) if kind is decoder._Sections else v[0]
    a, b = args.from_buffer_copy(pack(*values)), args(**fields)
    for name, kind in args._fields_:
        x, y = getattr(a, name), getattr(b, name)
        assert list(x) == list(y) if kind is decoder._Sections else x == y, name
    with pytest.raises(decoder.NVFP4Error):
        pack(*(1 << 70 for _ in values))


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: nv.rotary(x, i), lambda: nv.kv_append((x, x, x, x), x, x, i.view(4, 1), i),
                 lambda: nv.attention(x, (x, x, x, x), i.view(4, 1), i)):
        with pytest.raises(nv.NVFP4Error):
            call()


@pytest.mark.parametrize("kw,err", [
    (dict(x=None), INVALID), (dict(logits=None), INVALID), (dict(up_codes=None), INVALID), (dict(up_scales=None), INVALID),
    (dict(up_alpha=None), INVALID), (dict(down_codes=None), INVALID), (dict(down_scales=None), INVALID),
    (dict(down_alpha=None), INVALID), (dict(y=None), INVALID), (dict(tokens=-1), INVALID), (dict(width=0), INVALID),
    (dict(inner=0), INVALID), (dict(experts=0), INVALID), (dict(top_k=0), INVALID), (dict(width=72), SHAPE),
    (dict(inner=40), SHAPE), (dict(width=(1 << 21) + 16), SHAPE), (dict(inner=(1 << 21) + 16), SHAPE), (dict(experts=513), SHAPE),
    (dict(top_k=9), SHAPE), (dict(experts=64, top_k=33), SHAPE), (dict(tokens=4097), SHAPE), (dict(tokens=1 << 40), SHAPE),
    (dict(width=1 << 16, inner=1 << 14, ldx=1 << 16), SHAPE), (dict(ldx=63), INVALID), (dict(ldl=7), INVALID),
    (dict(residual=FAKE, ldr=63), INVALID), (dict(ldx=1 << 31), SHAPE), (dict(ldl=1 << 31), SHAPE),
    (dict(residual=FAKE, ldr=1 << 31), SHAPE), (dict(logits_dtype=2), INVALID), (dict(activation=3), INVALID),
    (dict(activation=0), INVALID), (dict(gated=2), INVALID), (dict(normalize=2), INVALID), (dict(scoring=2), INVALID),
    (dict(workspace=FAKE + 16), INVALID), (dict(x=FAKE + 1), INVALID), (dict(logits=FAKE + 1), INVALID),
    (dict(logits=FAKE + 2, logits_dtype=1), INVALID), (dict(up_codes=FAKE + 4), INVALID), (dict(down_codes=FAKE + 4), INVALID),
    (dict(up_alpha=FAKE + 2), INVALID), (dict(down_alpha=FAKE + 2), INVALID), (dict(y=FAKE + 1), INVALID),
    (dict(residual=FAKE + 1, ldr=64), INVALID), (dict(workspace=FAKE, workspace_bytes=256), WORKSPACE), (dict(tokens=0), OK),
    (dict(tokens=0, x=None), OK),
])
def test_moe_rejects(L, kw, err):
    a = decoder._MoeArgs(x=FAKE, ldx=64, logits=FAKE, ldl=8, tokens=4, width=64, inner=32, experts=8, top_k=2, up_codes=FAKE,
                         up_scales=FAKE, up_alpha=FAKE, down_codes=FAKE, down_scales=FAKE, down_alpha=FAKE, activation=1,
                         gated=1, y=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    assert L.nvfp4_moe(ctypes.byref(a)) == err
    assert L.nvfp4_moe(None) == INVALID


def test_moe_workspace(L):
    assert L.nvfp4_moe_workspace_bytes(4, 64, 32, 8, 2) > 0 and L.nvfp4_moe_workspace_bytes(0, 64, 32, 8, 2) == 0
    assert L.nvfp4_moe_workspace_bytes(4, 72, 32, 8, 2) == 0
