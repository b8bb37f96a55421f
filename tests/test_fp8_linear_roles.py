"""The order of waits, warp barriers and issues in the loading and the product warps of
fp8_linear.cu, run through a model of two lanes and an mbarrier's phases.

An mbarrier tells a phase by its parity alone. Both lanes wait for phase n in turn n; what the
elected lane issues in turn n lets phase n + 1 end. A lane that first looks when phase n + 1 has
ended too sees the parity of an unfinished phase n, and waits for phase n + 2, which ends only
after turn n + 1: if the warp meets in between, nobody goes on."""
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parents[1] / "diffusion_drafted_lossless_b200" / "csrc" / "fp8_linear.cu"


def _turn(begin, end):
    """What a lane does in one turn of the loop between two marks of the source: W waits, S meets
    the warp, I issues (the elected lane alone)."""
    text = SOURCE.read_text()
    role = text[text.index(begin):text.index(end)]
    marks = re.findall(r"(wait_phase\(&(?:empty|full)\[s\])|(__syncwarp\(\))|(if \(one && ok\))", role)
    order = "".join("WSI"[next(i for i, m in enumerate(found) if m)] for found in marks)
    loop = re.search(r"W[SI]*I[S]*", order)
    assert loop, order
    return loop.group(0)


def _stuck(turn, turns=5):
    """Whether any order of the lanes' steps and the phases' ends leaves both lanes unable to go on."""
    steps = turn * turns
    start, seen = (0, 0, 0, 0), set()  # where lane 0 (elected) and lane 1 are, issues made, phases ended
    todo = [start]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        a, b, issued, ended = state
        nexts = []
        if ended < min(issued + 1, turns):  # the phase of a turn ends once the turn before has issued
            nexts.append((a, b, issued, ended + 1))
        for lane in (0, 1):
            at = (a, b)[lane]
            if at == len(steps):
                continue
            n, what = at // len(turn), steps[at]
            if what == "W" and (ended & 1) == (n & 1):
                continue  # the parity of a phase that has not ended
            if what == "S":  # both at the same meeting
                if a == b:
                    nexts.append((a + 1, b + 1, issued, ended))
                continue
            made = issued + (what == "I" and lane == 0)
            nexts.append((a + 1, b, made, ended) if lane == 0 else (a, b + 1, made, ended))
        if not nexts and (a, b) != (len(steps), len(steps)):
            return True
        todo += nexts
    return False


def test_the_model_tells_the_two_orders_apart():
    assert _stuck("WIS") and _stuck("WI") and not _stuck("WSI") and not _stuck("WSIS")


@pytest.mark.parametrize("role", [("if (warp == 0) {", "} else if (warp <= 2) {"),
                                  ("} else if (warp <= 2) {", "// The scales of the next eight K blocks")])
def test_no_lane_can_miss_its_phase(role):
    turn = _turn(*role)
    assert not _stuck(turn), turn
