"""The compiled code of the bf16 products (no GPU needed).

Their large tiles multiply in inline assembly, whose results and operands the
compiler knows nothing of: it must neither move a sum while a matrix instruction
may still be writing it, nor write an operand with a vector instruction right
before it is read.  Both are looked for in what the compiler makes of the
kernels' sources.
"""
import os
import re
import subprocess

import pytest

from combine_topk_idx_amd import build as B

OPTIONS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I", os.path.join(B.ROOT, "include"), "-I", os.path.join(B.PKG, "csrc")]
FILES = ["moe_train_gemm.hip", "moe_train_weight.hip"]


@pytest.fixture(scope="module", params=FILES)
def kernels(request, tmp_path_factory):
    """(name, {label: instructions} in order) of a file's kernels that multiply in inline assembly
    (in others the compiler, which may use accumulators too, knows of every wait)."""
    out = str(tmp_path_factory.mktemp("s") / "k.s")
    subprocess.run([B.hipcc(), *OPTIONS, "-S", "--cuda-device-only", "-o", out,
                    os.path.join(B.PKG, "csrc", request.param)], check=True, capture_output=True, timeout=600)
    found = []
    for m in re.finditer(r"^(_ZN\S+):\s*;.*?\n(.*?)\.Lfunc_end", open(out).read(), re.S | re.M):
        if not re.search(r"#ASMSTART\s+v_mfma\S+ a\[", m[2]):
            continue
        blocks, label = {"entry": []}, "entry"
        for line in m[2].split("\n"):
            line = line.split(";")[0].strip()
            at = re.match(r"(\.LBB\S+):", line)
            if at:
                label = at[1]
                blocks[label] = []
            elif line and not line.startswith("."):
                blocks[label].append(line)
        found.append((m[1], blocks))
    assert found
    return found


def _registers(text):
    got = set()
    for m in re.finditer(r"\bv\[(\d+):(\d+)\]", text):
        got |= set(range(int(m[1]), int(m[2]) + 1))
    return got | {int(m[1]) for m in re.finditer(r"\bv(\d+)\b", text)}


SUM = r"v_mfma\S+ a\["


def test_sums_stay_where_they_are(kernels):
    """No other use of an accumulator inside a loop of matrix instructions, nor on any way from
    one of them to the wait that ends the loop."""
    for name, blocks in kernels:
        labels = list(blocks)
        ways = {}
        for i, label in enumerate(labels):
            to = [m[1] for m in (re.match(r"s_c?branch\S*\s+(\.LBB\S+)", x) for x in blocks[label]) if m]
            ends = any(re.match(r"s_branch\b|s_endpgm", x) for x in blocks[label])
            ways[label] = to + (labels[i + 1:i + 2] if not ends else [])
        pending = dict.fromkeys(labels, False)
        todo = list(labels)
        while todo:
            label = todo.pop(0)
            flying = pending[label]
            for x in blocks[label]:
                if re.match(SUM, x):
                    flying = True
                elif re.match(r"s_nop 15", x):
                    flying = False
                else:
                    assert not (flying and re.search(r"\ba\[?\d", x)), f"{name} {label}: {x}"
            for to in ways[label]:
                if flying and not pending[to]:
                    pending[to] = True
                    todo.append(to)
        loops = [b for b in blocks.values() if sum(bool(re.match(SUM, x)) for x in b) >= 16]
        assert loops
        for block in loops:
            assert not [x for x in block if re.search(r"\ba\[?\d", x) and not re.match(SUM, x)], name
            assert any(re.match(r"s_nop 15", x) for x in block), name


def test_operands_come_from_lds(kernels):
    """No vector instruction writes an operand in the three instructions before it is read."""
    seen = 0
    for name, blocks in kernels:
        before = []
        for x in (x for block in blocks.values() for x in block):
            m = re.match(SUM + r"\d+:\d+\], (\S+), (\S+),", x)
            if m:
                seen += 1
                operands = _registers(m[1] + " " + m[2])
                for y in before[-3:]:
                    if re.match(r"v_(?!mfma)", y) and len(y.split(None, 1)) > 1:
                        assert not operands & _registers(y.split(None, 1)[1].split(",")[0]), f"{name}: {y} | {x}"
            before.append(x)
    assert seen > 100
