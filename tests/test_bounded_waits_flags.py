"""What a lane's own wait may decide, read off the sources as the waits themselves
are (test_bounded_waits.py).  `polls` is zero in a lane whose bounded wait gave up,
and the lanes of a warp may differ in it: a warp's way through its code, and with
it the collective instructions on that way, must not depend on it.  It may guard
what one lane does alone, or go into a vote."""

import os
import re

import pytest

from test_bounded_waits import CSRC

# an arrival of one lane's, or a vote of the whole warp
ALLOWED = (r"\bif \(lane == 0 && polls\)", r"__all_sync\(0xffffffffu, polls != 0\)")


def uses_of_polls(src):
    """(line, text) of every use of a lane's `polls` but its declaration and its
    being handed to the wait."""
    src = re.sub(r"//[^\n]*", "", src)
    out = []
    for n, line in enumerate(src.split("\n"), 1):
        rest = re.sub(r"uint32_t polls = kWaitPolls;|mbar_wait_or_pass\([^;]*\bpolls, p\.err\);", "",
                      line)
        if re.search(r"\bpolls\b", rest):
            out.append((n, rest.strip()))
    return out


@pytest.mark.parametrize("name", ["checkpoint_dw.cu", "mm8.cu"])
def test_a_warps_way_does_not_hang_on_a_lanes_wait(name):
    uses = uses_of_polls(open(os.path.join(CSRC, name)).read())
    assert uses
    bad = [u for u in uses if not any(re.search(a, u[1]) for a in ALLOWED)]
    assert not bad, bad


def test_the_check_sees_a_lane_that_leaves():
    for text in ("if (!polls) continue;", "if (polls && row < rows) x = __shfl_xor_sync(m, x, 1);",
                 "while (polls) {", "const bool on = polls != 0;"):
        assert uses_of_polls(text) == [(1, text)] and not any(re.search(a, text) for a in ALLOWED)


def test_the_weight_gradients_stores_go_by_a_vote():
    """A lane stores its neighbours' values as well as its own: whether a tile is
    stored is the same for the whole warp."""
    src = open(os.path.join(CSRC, "checkpoint_dw.cu")).read()
    tail = src[src.index("float* out = piece"):src.index("} else if (warp >= W_DEC) {")]
    vote = re.search(r"const bool (\w+) = __all_sync\(0xffffffffu, polls != 0\);", src)
    assert vote and re.search(r"if \(!%s\) continue;" % vote.group(1), tail)
    assert tail.index("continue;") < tail.index("__shfl_xor_sync")
