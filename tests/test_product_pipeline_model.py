"""The product kernel's ring of stages as a model: two CTAs, each with a loader
that waits for a stage's release before it fills it, and one issuer whose
commits release a stage in both CTAs, each arrival taking its own time.  No CTA
may leave while an arrival for it is under way (its shared memory is another
block's by then), in any order of arrivals; and the loaders' last waits, one per
stage, are what keeps it.  The parities are those of the kernel's source."""
import os
import random
import re

import pytest

from collective_all_reduce_rank_gb300 import build


class Barrier:
    """One arrival per phase; wait(parity) passes once the phase of that parity is over."""

    def __init__(self):
        self.phase = 0

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(blocks, stages, drain, rng):
    """Random order of events; returns arrivals that met a CTA which had left."""
    empty = [[Barrier() for _ in range(stages)] for _ in range(2)]
    filled = [[0] * stages for _ in range(2)]  # loads of each CTA's stage so far
    loader = [dict(k=0, s=0, parity=1, left=stages if drain else 0, gone=False) for _ in range(2)]
    issued, under_way, late, done_at = 0, [], 0, [False, False]
    while True:
        events = []
        for c in range(2):
            l = loader[c]
            if (l["k"] < blocks or l["left"]) and empty[c][l["s"]].passes(l["parity"]):
                events.append(("load", c))
            elif l["k"] == blocks and not l["left"] and not l["gone"] and issued == blocks:
                events.append(("leave", c))  # the accumulator's commit has been seen: all products are done
        if issued < blocks and all(filled[c][issued % stages] == issued // stages + 1 for c in range(2)):
            events.append(("issue", None))
        events += [("arrive", i) for i in range(len(under_way))]
        if not events:
            assert all(l["gone"] for l in loader), "stuck"
            return late
        what, i = rng.choice(events)
        if what == "load":
            l = loader[i]
            if l["k"] < blocks:
                filled[i][l["s"]] += 1
                l["k"] += 1
            else:
                l["left"] -= 1
            l["s"] += 1
            if l["s"] == stages:
                l["s"], l["parity"] = 0, l["parity"] ^ 1
        elif what == "issue":
            under_way += [(0, issued % stages), (1, issued % stages)]
            issued += 1
        elif what == "arrive":
            c, s = under_way.pop(i)
            late += loader[c]["gone"]
            empty[c][s].phase += 1
        elif loader[0]["k"] == loader[1]["k"] == blocks and not loader[0]["left"] and not loader[1]["left"]:
            loader[i]["gone"] = True  # the cluster barrier lets both go


@pytest.mark.parametrize("blocks", [1, 2, 5, 6, 7, 12, 13, 40])
@pytest.mark.parametrize("stages", [2, 6, 11])
def test_no_arrival_meets_a_cta_that_has_left(blocks, stages):
    for seed in range(40):
        assert run(blocks, stages, True, random.Random(seed)) == 0


def test_the_model_sees_them_without_the_last_waits():
    assert any(run(5, 6, False, random.Random(seed)) for seed in range(40))


def test_the_kernel_makes_the_last_waits():
    text = open(os.path.join(build.CSRC, "tc_gemm.cuh")).read()
    loader = text[text.index("if (warp == 0 || warp == 3) {"):text.index("} else if (warp == 1) {")]
    after = loader[loader.rindex("tc_tma_load"):]
    assert re.search(r"for \(int i = 0; i < nstages && ok && !is_a; \+\+i\) \{\s*ok = tc_wait\(empty0 \+ 8 \* s, parity", after)
