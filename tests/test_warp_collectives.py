"""Instructions that a whole warp has to reach together (PTX .sync.aligned and
.aligned forms) are undefined for a warp whose lanes are apart.  Branches taken
lane by lane lie in front of them (the column of a row's target, a row that is
outside the matrix), so each helper of the training operators that issues one
joins the lanes itself, whatever its caller did.  Read from the source: no GPU
is needed, and none should run code that fails this."""
import os
import re

import pytest

from collective_all_reduce_rank_gb300 import build

FILES = ["tc_gemm.cuh", "tc_epilogue.cuh", "kernels_gated_ffn.cu", "kernels_tc_store.cu", "kernels_vocab_loss.cu",
         "kernels_skinny.cu", "kernels_norm8.cu"]


def statements(text):
    """(line, asm statement, the source before it in its block) of each warp-collective asm."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    for m in re.finditer(r"asm volatile\(", text):
        end = text.index(";\n", m.start())
        while text[m.start():end].count("(") != text[m.start():end].count(")"):
            end = text.index(";\n", end + 1)
        asm = text[m.start():end]
        if ".aligned" not in asm:
            continue
        depth, i = 0, m.start() - 1
        while i >= 0 and depth >= 0:  # back to the brace that opens this block, nested blocks left out
            depth += {"}": 1, "{": -1}.get(text[i], 0)
            i -= 1
        yield text.count("\n", 0, m.start()) + 1, asm, text[i + 2:m.start()]


@pytest.mark.parametrize("name", FILES)
def test_lanes_are_joined_before_warp_collectives(name):
    text = open(os.path.join(build.CSRC, name)).read()
    bad = []
    for line, asm, before in statements(text):
        # what lies between the join and the instruction is straight-line code
        tail = before.rpartition("__syncwarp();")[2] if "__syncwarp();" in before else None
        if tail is None or re.search(r"\b(if|for|while|switch)\b|\?", tail):
            bad.append((line, asm.split('"')[1]))
    assert not bad, "%s: warp-collective instructions that may be reached by a part of a warp: %s" % (name, bad)


def test_the_reading_finds_them():
    found = sum(len(list(statements(open(os.path.join(build.CSRC, f)).read()))) for f in FILES)
    assert found >= 7
    ok = "{\n  __syncwarp();\n  asm volatile(\"x.sync.aligned;\" ::);\n}\n"
    assert [b for _, _, b in statements(ok)][0].strip() == "__syncwarp();"
