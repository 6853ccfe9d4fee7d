"""What a wave's lanes pass to each other through LDS in the attention and expert kernels has a barrier between the stores
and the loads in the optimised IR, where the compiler may reorder accesses that it can tell apart (CPU only: compiles,
runs nothing)."""
import os
import re
import subprocess

import pytest

from nvfp4_block_scaled_elem_amd import build as nvbuild

BARRIER = re.compile(r"call void @llvm\.amdgcn\.(wave|s)\.barrier")
STORE = re.compile(r"^\s*store .*ptr addrspace\(3\)")
LOAD = re.compile(r"= load .*ptr addrspace\(3\)")


def kernels(tmp, source, names):
    out = tmp / "k.ll"
    flags = [f for f in nvbuild.FLAGS if f != "-shared"]
    subprocess.run([nvbuild.HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(nvbuild.CSRC, source),
                    "-o", str(out)], check=True, capture_output=True)
    for name, body in re.findall(r"^define [^\n]*@(\w+)\([^\n]*\{\n(.*?)^\}", out.read_text(), re.S | re.M):
        for n in names:
            if re.search(r"\d" + n + r"(I|E)", name):
                yield name, body.splitlines()


@pytest.mark.parametrize("source,names,count", [("attention_kernels.hip", ("k_attn_split",), 10),
                                                ("moe_kernels.hip", ("k_moe_product", "k_moe_rows", "k_moe_down"), 10)])
def test_hand_overs(tmp_path, source, names, count):
    if not os.path.exists(nvbuild.HIPCC):
        pytest.skip("no hipcc")
    seen = 0
    for name, body in kernels(tmp_path, source, names):
        # 16-byte aligned accesses alone: the codes, operands and sums (lists and counters are scalars, behind work-group barriers)
        last, handed = None, 0
        for line in body:
            if BARRIER.search(line) or re.match(r"^\d+:|^[\w.]+:", line):  # a barrier, or a block's start
                last = None
            if "align 16" not in line:
                continue
            kind = "store" if STORE.search(line) else "load" if LOAD.search(line) else None
            if kind:
                assert last in (None, kind), f"{name}: an LDS {kind} follows a {last} with no barrier between\n{line}"
                handed += last is None and kind == "load"
                last = kind
        assert handed >= 1, name
        seen += 1
    assert seen >= count
