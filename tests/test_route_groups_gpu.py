"""Routing with groups of whole multiples of 32 experts, of which few, half or most
are kept: the choice goes over the kept ones only where they are at most half of
a token's registers.  Checks and bounds are those of the other routing tests."""

import pytest
import torch

from test_experts_gpu import _gen, _route

pytestmark = pytest.mark.gpu

SIZES = [(64, 2, 1, 6), (96, 3, 1, 5), (96, 3, 2, 5), (128, 4, 1, 32), (128, 4, 2, 6), (128, 2, 1, 8),
         (160, 5, 4, 8), (192, 3, 2, 4), (256, 4, 2, 8), (256, 4, 3, 8), (256, 2, 1, 8), (256, 8, 3, 9),
         (384, 3, 2, 8), (512, 16, 8, 8), (512, 16, 3, 12), (512, 4, 2, 31), (512, 2, 1, 8),
         (480, 15, 9, 8), (1024, 32, 8, 8)]


@pytest.mark.parametrize("E,groups,top_groups,k", SIZES)
@pytest.mark.parametrize("score,io", [("sigmoid", "fp32"), ("softmax", "bf16")])
def test_groups_of_whole_registers(E, groups, top_groups, k, score, io):
    _route(67, E, k, groups=groups, top_groups=top_groups, score=score, io=io)
    # equal scores, within a group and across groups
    l = torch.randint(-2, 3, (67, E), generator=_gen(E, k)).float()
    _route(67, E, k, groups=groups, top_groups=top_groups, score=score, io=io, logits=l, bias=None)


def test_fewer_experts_on_than_choices():
    for E, groups, top in ((128, 4, 2), (256, 4, 2), (512, 16, 4)):
        l = torch.randn(40, E, generator=_gen(E))
        l[::2, 3:E // groups] = -float("inf")
        l[::2, E // groups + 2:] = -float("inf")          # three experts, two, and none
        l[1::4] = -float("inf")
        _route(40, E, 8, groups=groups, top_groups=top, logits=l)
