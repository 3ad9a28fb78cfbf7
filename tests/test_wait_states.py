"""Wait states behind matrix operations, counted in the compiled code.

The result of v_mfma_f32_16x16x32_bf16 may be used by another kind of
instruction no sooner than eight wait states later; nothing in the hardware
holds an earlier use back, so the compiler has to fill them.  It does so
within a block, but has left five behind the join of two short branches, and
the result's last element was stale.  Here the sources with such operations
beside branches are compiled, and every path from a matrix operation to the
first use of its result is followed."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from dense_linear_projection_amd import _build

NEEDED, FAR = 8, 12
SOURCES = ["attend.hip", "quant.hip", "stream.hip"]


def registers(text):
    """The vector and accumulation registers of one operand."""
    m = re.match(r"([va])\[(\d+):(\d+)\]$", text)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"([va])(\d+)$", text)
    return {(m.group(1), int(m.group(2)))} if m else set()


def operands(text):
    return [t.strip().split(" ")[0] for t in text.split(None, 1)[1].split(",")] if " " in text or "\t" in text else []


def parse(text):
    """(instructions, label -> index)."""
    code, labels = [], {}
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"^([\w.$]+):", line)
        if m:
            labels[m.group(1)] = len(code)
        elif line and line[0] not in ".#":
            code.append(line)
    return code, labels


def nearest_use(code, labels, at):
    """Fewest wait states from the matrix operation at `at` to a use of its result by another kind of instruction."""
    result, best, seen = registers(operands(code[at])[0]), FAR, {}
    paths = [(at + 1, 0)]
    while paths:
        i, states = paths.pop()
        while i < len(code) and states < best and seen.get(i, FAR) > states:
            seen[i] = states
            words = code[i].split()
            if words[0] == "s_nop":
                states += int(words[1], 0) + 1
            elif words[0] == "s_branch":
                i, states = labels[words[1]], states + 1
                continue
            elif words[0].startswith("s_cbranch"):
                paths.append((labels[words[1]], states + 1))
                states += 1
            elif words[0] == "s_endpgm":
                break
            else:
                used = [registers(o) for o in operands(code[i])]
                if any(u & result for u in used):
                    if not words[0].startswith("v_mfma"):
                        best = min(best, states)
                    break
                states += 1
            i += 1
    return best


def compile_source(src):
    out = subprocess.run([_build.hipcc()] + _build.FLAGS + ["-x", "hip", "-S", "--cuda-device-only",
                                                            os.path.join(_build.CSRC, src), "-o", "-"],
                         check=True, capture_output=True, text=True)
    return out.stdout


@pytest.fixture(scope="module")
def compiled():
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(compile_source, SOURCES)))


@pytest.mark.parametrize("src", SOURCES)
def test_results_are_not_used_early(compiled, src):
    code, labels = parse(compiled[src])
    products = [i for i, t in enumerate(code) if t.startswith("v_mfma_f32_16x16x32_bf16")]
    assert len(products) > 100
    early = [(code[i], n) for i, n in ((i, nearest_use(code, labels, i)) for i in products) if n < NEEDED]
    assert not early, "%d of %d results are used too early: %s" % (len(early), len(products), early[:3])


def test_counting():
    """The count itself, on a join behind two branches and within a block."""
    block = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0\n%s\nv_mul_f32 v5, v3, v6\ns_endpgm"
    for between, states in (("s_nop 7", 8), ("s_nop 3\nv_mov_b32 v20, v21", 5),
                            ("s_cbranch_vccz .L1\ns_nop 9\ns_branch .L2\n.L1:\nv_mov_b32 v20, 0\n.L2:\ns_nop 0", 3)):
        code, labels = parse(block % between)
        assert nearest_use(code, labels, 0) == states
    code, labels = parse("v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[12:15], 0\nv_accvgpr_read_b32 v1, a2\ns_endpgm")
    assert nearest_use(code, labels, 0) == 0
