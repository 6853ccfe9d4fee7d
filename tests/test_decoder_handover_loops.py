"""What a wave's lanes pass to each other through LDS in the expert and attention kernels has a barrier between the accesses on every
way through the optimised IR, round the loops too, where the compiler may reorder accesses that it can tell apart (CPU
only: compiles, runs nothing)."""
import os
import re
import subprocess

import pytest

from nvfp4_block_scaled_elem_amd import build as nvbuild

BARRIER = re.compile(r"call void @llvm\.amdgcn\.(wave|s)\.barrier")
ACCESS = re.compile(r"(store|= load) (<[^>]*>|\w+).*?ptr addrspace\(3\) (.*?), align")
NAME = re.compile(r"[%@][\w.$]+")


def kernels(tmp, source, name):
    """(mangled name, instructions by block, successors of a block) of each form of a kernel."""
    out = tmp / "k.ll"
    if not out.exists():
        flags = [f for f in nvbuild.FLAGS if f != "-shared"]
        subprocess.run([nvbuild.HIPCC, *flags, "--cuda-device-only", "-S", "-emit-llvm", os.path.join(nvbuild.CSRC, source),
                        "-o", str(out)], check=True, capture_output=True)
    for mangled, body in re.findall(r"^define [^\n]*@(\w+)\([^\n]*\{\n(.*?)^\}", out.read_text(), re.S | re.M):
        if not re.search(r"\d" + name + r"(I|E)", mangled):
            continue
        blocks, to, at = {"": []}, {"": []}, ""
        for line in body.splitlines():
            label = re.match(r"^([\w.$]+):", line)
            if label:
                at = label.group(1)
                blocks[at], to[at] = [], []
                continue
            blocks[at].append(line)
            to[at] += re.findall(r"label %([\w.$]+)", line)
        yield mangled, blocks, to


def origin(defs, pointer, seen):
    """The LDS variables that a pointer may point into."""
    found = set()
    for name in NAME.findall(pointer):
        if name.startswith("@"):
            found.add(name)
        elif name not in seen and name in defs:
            seen.add(name)
            text = defs[name]
            if re.match(r"(getelementptr|phi|select|addrspacecast|bitcast|freeze)", text):
                found |= origin(defs, text, seen)
    return found


def unordered(blocks, to, take):
    """(accesses, pairs of accesses of different kinds with no barrier on some way between them). take(kind, type, variables): the
    accesses that count."""
    defs = {m.group(1): m.group(2) for lines in blocks.values() for m in (re.match(r"\s*(%[\w.$]+) = (.*)", x) for x in lines) if m}
    steps, count = {}, 0
    for label, lines in blocks.items():
        steps[label] = []
        for line in lines:
            if BARRIER.search(line):
                steps[label].append((None, line))
            m = ACCESS.search(line)
            if m:
                kind = "store" if m.group(1) == "store" else "load"
                if take(kind, m.group(2), origin(defs, m.group(3), set())):
                    steps[label].append((kind, line))
                    count += 1
    # at a block's start: the last accesses, since a barrier, of the ways to it
    before, work, bad = {label: set() for label in blocks}, list(blocks), set()
    while work:
        label = work.pop()
        last = set(before[label])
        for step in steps[label]:
            if step[0] is None:
                last = set()
                continue
            bad |= {(x, step) for x in last if x[0] != step[0]}
            last = {step}
        for t in to[label]:
            if not last <= before[t]:
                before[t] |= last
                work.append(t)
    return count, bad


@pytest.fixture(scope="module")
def tmp(tmp_path_factory):
    if not os.path.exists(nvbuild.HIPCC):
        pytest.skip("no hipcc")
    return {s: tmp_path_factory.mktemp(s) for s in ("moe_kernels.hip", "attention_kernels.hip")}


@pytest.mark.parametrize("name,area,forms", [("k_moe_rows", "5lds_w", 10), ("k_moe_product", "3lds", 5), ("k_moe_down", "3lds", 1)])
def test_codes_and_scales_of_experts(tmp, name, area, forms):
    """A wave's codes and scales: from the stores to the loads, and from the loads to the stores of the next ones."""
    seen = 0
    for mangled, blocks, to in kernels(tmp["moe_kernels.hip"], "moe_kernels.hip", name):
        count, bad = unordered(blocks, to, lambda kind, form, names: any(n.endswith(area) for n in names))
        assert count >= 4, mangled
        assert not bad, (mangled, [(a[1].strip(), b[1].strip()) for a, b in list(bad)[:2]])
        seen += 1
    assert seen >= forms


@pytest.mark.parametrize("name,forms", [("k_attn_split", 10), ("k_attn_rows", 12)])
def test_codes_of_a_wave_in_attention(tmp, name, forms):
    """Codes of a block, 16 bytes at a time: no load is reached from a store without a barrier (the values' codes are stored while
    the keys' lie beside them, so a store may follow a load of the others); three hand-overs a block."""
    seen = 0
    for mangled, blocks, to in kernels(tmp["attention_kernels.hip"], "attention_kernels.hip", name):
        count, bad = unordered(blocks, to, lambda kind, form, names: form == "<4 x i32>")
        bad = {(a, b) for a, b in bad if b[0] == "load"}
        assert count >= 16, mangled
        assert not bad, (mangled, [(a[1].strip(), b[1].strip()) for a, b in list(bad)[:2]])
        assert sum("@llvm.amdgcn.wave.barrier" in x for lines in blocks.values() for x in lines) >= 3, mangled
        seen += 1
    assert seen >= forms
