"""Who may wait how: where a warp waits on an mbarrier as a whole, and runs
collective instructions behind the wait, a lane whose bounded wait gave up
has to stay with its warp (it goes on without waiting).  A lane that left would
be waited for without a bound by those that a phase completing around the last
poll let through.  This is read off the sources, since a wait that runs out in
such a moment cannot be brought about."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sequence_latent_norm_gb300", "csrc")


def whole_warp_waits(path):
    """(line, statement up to the wait) of every wait that is not in a block of
    one lane's."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    out, blocks, text = [], [], ""
    for m in re.finditer(r"[{};]|mbar_wait(?:_each|_or_pass|_cluster)?\(|[^{};]", src):
        t = m.group()
        if t == "{":
            blocks.append(text)
        elif t == "}":
            blocks.pop()
        elif t.startswith("mbar_wait"):
            # one lane's, or of a function that one lane calls
            one = r"\b(lane|tl|threadIdx\.x) == 0\b|\bvoid wait_landed\("
            if not any(re.search(one, b) for b in [*blocks, text]):
                out.append((src.count("\n", 0, m.start()) + 1, " ".join((text + t).split())))
        text = "" if t in "{};" else text + t
    return out


@pytest.mark.parametrize("name", ["checkpoint_dw.cu", "residual_ring.cu"])
def test_lanes_that_gave_up_stay_with_their_warp(name):
    waits = whole_warp_waits(os.path.join(CSRC, name))
    assert waits
    stays = r"\bok = ok && mbar_wait_each\($|^(if \([^()]*\) )?mbar_wait_or_pass\($"
    left = [(line, text) for line, text in waits if not re.search(stays, text)]
    assert not left, f"{name}: these waits decide where their lane goes on: {left}"


@pytest.mark.parametrize("name,issue,landed", [
    ("checkpoint_dw.cu", r"tma_load_3d_pair\(", r"wait_landed\(b_full, it, p\.err\);"),
    ("checkpoint_dw.cu", r"tma_load_2d\(", r"wait_landed\(c_full, it, p\.err\);"),
    ("checkpoint_dw.cu", r"mma_ss_pair\(", r"if \(ic > 0\) mbar_wait_each\(&acc_full\[")])
def test_what_is_in_flight_is_waited_for(name, issue, landed):
    """A kernel does not leave its shared memory to copies or products that it
    has in flight, also where a wait gave up: behind the code that issues them
    stands a wait for all of them, with a limit, like the others."""
    src = open(os.path.join(CSRC, name)).read()
    first = re.search(issue, src)
    assert first and re.search(landed, src[first.end():]), name


@pytest.mark.parametrize("name", ["attn_fwd.cu", "attn_bwd_dq.cu", "attn_bwd_kv.cu", "gemm_tc.cu"])
def test_lanes_that_leave_leave_together(name):
    """Kernels whose warps leave a loop on a wait's answer take the wait that
    votes on every poll."""
    waits = whole_warp_waits(os.path.join(CSRC, name))
    assert waits and all(text.endswith("mbar_wait(") for _, text in waits)
    wait = re.search(r"bool mbar_wait\(.*?\n}\n", open(os.path.join(CSRC, "sm100.cuh")).read(),
                     re.S).group()
    loop = re.search(r"for \(uint32_t i = 0; i < kWaitPolls; \+\+i\) \{(.*)\n  \}\n", wait, re.S).group(1)
    assert re.findall(r"if \((.*)\) \{\n[^}]*return true;", loop) == ["__any_sync(together, seen)"]
