"""Routing of the largest batches: sizes next to 2^31 tokens of one choice."""

import pytest
import torch

DEV = "cuda:0"
MOST = 2 ** 31 - 1 - 128                       # rows that the row order can number


@pytest.fixture(scope="module")
def lib():
    from sequence_latent_norm_gb300.build import build_library
    build_library()
    import sequence_latent_norm_gb300 as pkg
    return pkg._lib


@pytest.mark.parametrize("experts,align", [(1, 1), (3, 1), (600, 1)])
def test_scratch_of_the_largest_batches(lib, experts, align):
    """Counts by expert of 152 blocks at the most, whatever the number of tokens."""
    most = 152 * 4 * ((experts + 3) // 4 * 4) + 255
    for T in (2 ** 20, 2 ** 31 - 2 ** 24, 2 ** 31 - 10 ** 7, MOST - 1000, MOST - 30, MOST):
        d = lib.make_route_dims(T, experts, 1, align=align)
        assert lib.route_rows(d) == T
        assert 0 < lib.route_workspace_bytes(d) <= most, T


def test_larger_batches_are_refused(lib):
    for T in (MOST + 1, 2 ** 31 - 1):
        d = lib.make_route_dims(T, 1, 1, align=1)
        assert lib.route_rows(d) == 0 and lib.route_workspace_bytes(d) == 0


@pytest.mark.gpu
def test_the_largest_batch():
    """Every token's one expert, its weight and gradient, and the row order.  A
    score of a bf16 logit has an error of 8 units of fp32's last place at most."""
    import sequence_latent_norm_gb300 as laga
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    l = torch.empty(MOST, 1, dtype=torch.bfloat16, device=DEV)
    period = torch.linspace(-4, 4, 4093, device=DEV).to(torch.bfloat16)   # prime: no chunk's
    for i in range(0, MOST, 4093 << 14):
        n = min(4093 << 14, MOST - i)
        l[i:i + n, 0] = period.repeat(1 << 14)[:n]
    r = laga.Router(1, 1, renormalise=False, align=1, io_dtype="bf16", device=DEV)
    out = r.forward(l)
    dl = r.backward(l, out, out.weight)
    laga._lib.sync_check()
    assert out.start.tolist() == [0, MOST]
    for i in range(0, MOST, 1 << 28):
        at = slice(i, min(i + (1 << 28), MOST))
        n = torch.arange(at.start, at.stop, dtype=torch.int32, device=DEV)
        assert torch.equal(out.row[at, 0], n) and torch.equal(out.pair[at], n)
        assert not out.expert[at].any()
    for i in (0, 4093 * 300000, MOST - 4093):
        s = torch.sigmoid(l[i:i + 4093, 0].double())
        assert ((out.weight[i:i + 4093, 0].double() - s).abs() <= 8 * 2.0 ** -24 * s).all()
        g = s * s * (1 - s)
        err = (dl[i:i + 4093, 0].double() - g).abs()
        assert (err <= (2.0 ** -8 + 32 * 2.0 ** -24) * g).all()
