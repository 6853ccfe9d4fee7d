"""What a wave's lanes pass to each other through LDS has a barrier between the stores and the loads in the optimised
IR, where the compiler may reorder accesses that it can tell apart (CPU only: compiles, runs nothing)."""
import os
import re
import subprocess

import pytest

from nvfp4_block_scaled_elem_amd import build as nvbuild

BARRIER = re.compile(r"call void @llvm\.amdgcn\.(wave|s)\.barrier")
STORE = re.compile(r"^\s*store .*ptr addrspace\(3\)")
LOAD = re.compile(r"= load .*ptr addrspace\(3\)")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(nvbuild.HIPCC):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("ir") / "linear.ll"
    flags = [f for f in nvbuild.FLAGS if f != "-shared"]
    subprocess.run([nvbuild.HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm",
                    os.path.join(nvbuild.CSRC, "linear_kernels.hip"), "-o", str(out)], check=True, capture_output=True)
    found = {}
    for name, body in re.findall(r"^define [^\n]*@(\w+)\([^\n]*\{\n(.*?)^\}", out.read_text(), re.S | re.M):
        m = re.search(r"(k_lin_skinny|k_lin_tile)((?:I|L[ib]\d+E)+)E", name)
        if m:
            found[m.group(1), tuple(int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2)))] = body.splitlines()
    return found


def test_few_rows(kernels):
    mine = {k: v for k, v in kernels.items() if k[0] == "k_lin_skinny"}
    assert len(mine) > 10
    for name, body in mine.items():
        last, handed = None, 0
        for line in body:
            if BARRIER.search(line) or re.match(r"^\d+:|^[\w.]+:", line):  # a barrier, or a block's start
                last = None
            kind = "store" if STORE.search(line) else "load" if LOAD.search(line) else None
            if kind:
                assert last in (None, kind), f"{name}: an LDS {kind} follows a {last} with no barrier between\n{line}"
                handed += last is None and kind == "load"
                last = kind
        assert handed >= 2, name


def test_tiles(kernels):
    """Codes: from a pair's stores to the lanes' reads. Turned: the scales, the fragments before the loop and after it,
    and the next step's stores over them."""
    mine = {k[1]: v for k, v in kernels.items() if k[0] == "k_lin_tile"}
    assert {src for _, src, _ in mine} == {0, 1, 2}
    for (mt, src, epi), body in mine.items():
        count = sum("@llvm.amdgcn.wave.barrier" in line for line in body)
        assert count >= {0: 1, 1: 0, 2: 8}[src], (mt, src, epi, count)
