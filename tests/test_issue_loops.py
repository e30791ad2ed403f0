"""Protocol of the loops in which a whole warp runs and one elected lane
issues: a stage is handed back by that lane alone, so every wait of the loop
has to keep the warp in step (mbar_wait_warp).  With a wait that returns to
each lane by itself the elected lane may run ahead until the ring has come
round, and a lane left behind waits for a phase that is past.  Read from the
sources: the fault cannot be provoked without a GPU that waits."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_bf16_mxfp4_gb300", "csrc")


def elected_loops():
    """(file, code) from each election to the wait for the last issued work (the drain barrier: one phase, never
    waited for twice)."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
            for at in re.finditer(r"ptx::elect_one\(\)", code):
                end = re.compile(r"if \(issued\)").search(code, at.end())
                yield name, code[at.end(): end.start()]


LOOPS = list(elected_loops())


def test_the_loops_are_found():
    assert [n for n, _ in LOOPS] == ["lora.cu", "lora.cu", "moe_experts.cu"]


@pytest.mark.parametrize("at", range(3))
def test_every_wait_keeps_the_warp_in_step(at):
    name, code = LOOPS[at]
    waits = re.findall(r"ptx::(mbar_\w*wait\w*)\(", code)
    assert len(waits) == 2 and set(waits) == {"mbar_wait_warp"}, (name, waits)  # the accumulator's and the stage's


def test_the_vote_covers_every_lane():
    code = open(os.path.join(CSRC, "sm100_ptx.cuh")).read()
    body = code[code.index("bool mbar_wait_warp("):]
    body = body[: body.index("\n}")]
    assert re.search(r"return __all_sync\(0xffffffffu, \w+\);", body)
