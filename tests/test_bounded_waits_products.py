"""Who may wait how in the 8-bit products, read off the source as for the other
kernels (test_bounded_waits.py): a lane whose bounded wait gave up stays with
its warp, and what is in flight is waited for before a CTA leaves."""

import os
import re

from test_bounded_waits import CSRC, whole_warp_waits

SRC = os.path.join(CSRC, "mm8.cu")


def test_lanes_that_gave_up_stay_with_their_warp():
    waits = whole_warp_waits(SRC)
    assert waits
    left = [(line, text) for line, text in waits
            if not re.search(r"^(if \([^()]*\) )?mbar_wait_or_pass\($", text)]
    assert not left, left


def test_what_is_in_flight_is_waited_for():
    src = open(SRC).read()
    for issue, landed in ((r"tma_load_2d_pair\(", r"wait_landed\(full, it, p\.err\);"),
                          (r"mma_mx_pair\(d", r"if \(tile > 0\) mbar_wait_each\(&acc_full\["),
                          (r"tma_store_2d\(ym", r"bulk_wait_read0\(\);\s+__syncwarp\(\);\s+}\s+// neither")):
        first = re.search(issue, src)
        assert first and re.search(landed, src[first.end():]), issue


def test_every_wait_is_bounded():
    """No wait of these files but the bounded ones."""
    for name in ("mm8.cu", "route.cu", "experts.cu", "weight8.cu"):
        src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        assert "mbarrier." not in src and not re.search(r"while \(true\)|for \(;;\)", src), name
