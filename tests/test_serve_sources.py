"""What must hold in the sources of the serving-step operators, as
test_warp_collectives.py reads it of the training step's: lanes are joined
before every instruction that a whole warp has to reach together."""
import os
import re

import pytest

from collective_all_reduce_rank_gb300 import build
from test_warp_collectives import statements

FILES = ["mx4_mma.cuh", "kernels_mx4.cu", "kernels_mx4_product.cu", "kernels_mx4_few.cu", "kernels_vocab_sample.cu"]


@pytest.mark.parametrize("name", FILES)
def test_lanes_are_joined_before_warp_collectives(name):
    bad = []
    for line, asm, before in statements(open(os.path.join(build.CSRC, name)).read()):
        tail = before.rpartition("__syncwarp();")[2] if "__syncwarp();" in before else None
        if tail is None or re.search(r"\b(if|for|while|switch)\b|\?", tail):
            bad.append((line, asm.split('"')[1]))
    assert not bad, "%s: %s" % (name, bad)
