"""CPU tests of the built library's own machine code (llvm-objdump of its
gfx950 code objects).

The products' main loop refills a stage's LDS buffer behind a barrier, which
every wave must reach with its fragments of that stage in registers.  Source
order alone does not give that: the compiler may move an LDS read past the
barrier, into the block that uses it, where it races with the other waves'
direct loads into the same buffer (results then differ now and then).
"""

import os
import re
import shutil
import subprocess

import pytest

import dimuon_newton_schulz_amd as D

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump") or "") if os.path.exists(p)), "")

pytestmark = [pytest.mark.skipif(not os.path.exists(D.LIB_PATH), reason="library not built"),
              pytest.mark.skipif(not OBJDUMP, reason="llvm-objdump not installed")]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel name: [(address, instruction, branch target or None), ...]} of every kernel of the library."""
    folder = tmp_path_factory.mktemp("code")
    lib = shutil.copy(D.LIB_PATH, folder / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=folder, check=True, stdout=subprocess.DEVNULL)
    out = {}
    for name in sorted(os.listdir(folder)):
        if "gfx950" not in name:
            continue
        text = subprocess.run([OBJDUMP, "-d", str(folder / name)], check=True, stdout=subprocess.PIPE, text=True).stdout
        code = None
        for line in text.splitlines():
            head = re.match(r"^([0-9a-f]+) <(\S+)>:$", line)
            if head:
                start, code = int(head.group(1), 16), out.setdefault(head.group(2), [])
                continue
            ins = re.match(r"^\s+(\S.*?)\s*// ([0-9A-F]+): [0-9A-F ]+(?:<\S+\+0x([0-9a-f]+)>)?$", line)
            if ins and code is not None:
                target = None if ins.group(3) is None else start + int(ins.group(3), 16)
                code.append((int(ins.group(2), 16), ins.group(1), target))
    return out


def stages(code):
    """The pairs (16-byte reads, transposing reads) between two barriers, over
    every path of the control flow between them that multiplies and reads
    fragments."""
    place = {address: i for i, (address, _, _) in enumerate(code)}
    counts, seen, todo = set(), set(), [(0, 0, 0, 0)]
    while todo:
        state = todo.pop()
        at, wide, turned, mfma = state
        while state not in seen and at < len(code):
            seen.add(state)
            assert wide + turned <= 256 and mfma <= 1024, "a loop without a barrier"
            _, text, target = code[at]
            op = text.split()[0]
            at += 1
            if op == "s_endpgm":
                break
            if op == "s_barrier":
                if mfma and (wide or turned):
                    counts.add((wide, turned))
                wide = turned = mfma = 0
            elif op == "ds_read_b64_tr_b16":
                turned += 1
            elif op == "ds_read_b128":
                wide += 1
            elif op.startswith("v_mfma"):
                mfma += 1
            elif op == "s_branch":
                at = place[target]
            elif op.startswith("s_cbranch"):
                todo.append((place[target], wide, turned, mfma))
            state = (at, wide, turned, mfma)
    return counts


def test_fragments_are_read_before_the_barrier_that_frees_their_buffer(kernels):
    """Every stage of a product's main loop reads the same number of
    fragments between its two barriers, on every path: none is read a stage
    later."""
    products = {name: code for name, code in kernels.items()
                if ("k_syrk" in name or "k_combine" in name) and any(i.startswith("v_mfma") for _, i, _ in code)}
    assert len(products) >= 20
    bad = {}
    for name, code in products.items():
        counts = stages(code)
        if len(counts) != 1:
            bad[name] = counts
    assert not bad, bad


def test_no_packed_float32_arithmetic(kernels):
    assert kernels
    for name, code in kernels.items():
        assert not any(re.match(r"v_pk_(add|mul|fma)_f32", i) for _, i, _ in code), name
