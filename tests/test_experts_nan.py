"""Tokens that hold a NaN stay visible all the way through the routed experts: a
token none of whose experts is on because its logits are NaN (one NaN in h makes
every logit of the token one) comes out as NaN, where one that is masked (-inf)
comes out as zeros."""

import numpy as np
import pytest
import torch

from laga_inputs import as_f64
from oracle import experts as oex

DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_oracle_weights_of_a_nan_token(score):
    l = np.zeros((4, 6))
    l[0] = np.nan                              # nothing on
    l[1] = -np.inf                             # masked
    l[2, 2:] = -np.inf
    l[2, 1] = np.nan                           # one on, of three choices
    l[3, 4] = np.nan                           # all choices found
    e, w = oex.choose(l, None, top_k=3, score=score)
    assert e.tolist() == [[-1, -1, -1], [-1, -1, -1], [0, -1, -1], [0, 1, 2]]
    assert np.isnan(w[[0, 2, 3]]).all() and (w[1] == 0).all()
    row, _, _ = oex.order(e, local=6, align=1, rows=4, weight=w)
    assert row.tolist() == [[-2, -2, -2], [-1, -1, -1], [0, -2, -2], [1, 2, 3]]
    out, _ = oex.combine(np.ones((4, 2)), w, row)
    assert np.isnan(out[[0, 2, 3]]).all() and (out[1] == 0).all()
    # the same by the formula: a NaN logit's slope is a NaN
    g = oex.route_bwd(l, e, np.ones((4, 3)), score=score)
    assert np.isnan(g[0]).all() and (g[1] == 0).all() and np.isnan(g[2, 1])


# ------------------------------------------------------------------ routing
def _logits(T, E, score, seed=0):
    """Random logits with tokens of every kind; the kinds by token."""
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(seed + T))
    kind = torch.arange(T) % 6
    l[kind == 1] = NAN                                     # nothing on
    l[kind == 2] = -INF                                    # masked
    l[kind == 3, 1:] = NAN                                 # one on
    if score == "softmax":
        l[kind == 4] = -INF
        l[kind == 4, 2] = INF                              # as good as a NaN, and alone
    else:
        l[kind == 4, ::2] = NAN
    return l, kind.numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,groups,top_groups", [(6, 8, 3, 1, 1), (700, 64, 6, 8, 3),
                                                     (5000, 256, 8, 8, 4), (90, 300, 32, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shard", [None, (2, 5)])
def test_router_marks_nan_tokens(T, E, k, groups, top_groups, score, shard):
    laga = _laga()
    l, kind = _logits(T, E, score)
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1))
    r = laga.Router(E, k, score=score, groups=groups, top_groups=top_groups, shard=shard, device=DEV)
    out = r.forward(l.to(DEV), b.to(DEV))
    laga._lib.sync_check()
    e, w = oex.choose(as_f64(l), as_f64(b), top_k=k, groups=groups, top_groups=top_groups,
                      score=score)
    first, local = shard or (0, E)
    row, pair, start = oex.order(e, first=first, local=local, align=128, rows=out.rows, weight=w)
    assert np.array_equal(out.expert.cpu().numpy(), e)
    got = as_f64(out.weight)
    assert np.array_equal(np.isnan(got), np.isnan(w)) and np.isnan(got[kind == 1]).all()
    assert (got[kind == 2] == 0).all()
    for name, want in (("row", row), ("pair", pair), ("start", start)):
        assert np.array_equal(getattr(out, name).cpu().numpy(), want), name
    assert (row[kind == 1] == -2).all() and (row[kind == 2] == -1).all()
    # the gradient: the formula's NaNs, in the tokens that lack a choice
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2))
    dl = as_f64(r.backward(l.to(DEV), out, dw.to(DEV)))
    want = oex.route_bwd(as_f64(l), e, as_f64(dw), score=score)
    lacks = (e < 0).any(axis=1)
    assert np.array_equal(np.isnan(dl[lacks]), np.isnan(want[lacks]))
    assert np.isnan(dl[kind == 1]).all() and (dl[kind == 2] == 0).all()
    clean = ~np.isnan(as_f64(l)).any(axis=1) & ~np.isposinf(as_f64(l)).any(axis=1)
    assert np.isfinite(dl[clean]).all()


@pytest.mark.gpu
def test_every_bias_a_nan():
    laga = _laga()
    r = laga.Router(16, 2, device=DEV)
    out = r.forward(torch.randn(40, 16, device=DEV), torch.full((16,), NAN, device=DEV))
    assert (out.expert == -1).all() and out.weight.isnan().all() and (out.row == -2).all()
    assert laga.combine(torch.ones(out.rows, 64, device=DEV), out).isnan().all()


# ------------------------------------------------------------------ rows back
@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [256, 129])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_carries_the_nan(d, dt, weighted):
    laga = _laga()
    T, E, k = 66, 8, 3
    l, kind = _logits(T, E, "sigmoid")
    r = laga.Router(E, k, device=DEV).forward(l.to(DEV))
    y = torch.randn(r.rows, d, generator=torch.Generator().manual_seed(3)).to(dt)
    out = laga.combine(y.to(DEV), r, weighted=weighted)
    dout = torch.randn(T, d, generator=torch.Generator().manual_seed(4)).to(dt).to(DEV)
    dy, dw = laga.combine_grad(dout, r, y=y.to(DEV), weighted=weighted)
    laga._lib.sync_check()
    w = as_f64(r.weight) if weighted else np.ones((T, k))
    want, _ = oex.combine(as_f64(y), w, r.row.cpu().numpy())
    assert np.array_equal(np.isnan(as_f64(out)), np.isnan(want))
    assert out[torch.from_numpy(kind == 1)].isnan().all()
    assert (out[torch.from_numpy(kind == 2)] == 0).all()
    # pairs without a row have no gradient
    assert (dw[r.row < 0] == 0).all()


@pytest.mark.gpu
def test_other_ranks_choices_add_nothing():
    """A NaN token whose experts all belong to other ranks: those ranks' outputs
    are NaN, this one's stays zero; a token without any expert is NaN on all."""
    laga = _laga()
    l = torch.zeros(3, 8)
    l[0, 4:] = 2.0
    l[0, 1] = NAN                              # chooses 4 and 5, of another rank
    l[1] = NAN
    for shard, nan in (((0, 4), [False, True, False]), ((4, 4), [True, True, False])):
        r = laga.Router(8, 2, shard=shard, device=DEV).forward(l.to(DEV))
        out = laga.combine(torch.ones(r.rows, 64, device=DEV), r)
        laga._lib.sync_check()
        assert r.weight[0].isnan().all() and out.isnan().all(dim=1).tolist() == nan
        assert out.isnan().any(dim=1).tolist() == nan
        if shard[0] == 0:
            assert (out[0] == 0).all() and (r.row[0] == -1).all()


# ------------------------------------------------------------------ the block
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [40, 700])
def test_block_with_one_nan_in_h(T, score, io):
    laga = _laga()
    d, f, E = 256, 128, 6
    dt = dict(bf16=torch.bfloat16, fp32=torch.float32)[io]
    g = torch.Generator().manual_seed(T)
    h = torch.randn(T, d, generator=g).to(dt).to(DEV)
    w_router = (torch.randn(d, E, generator=g) * d ** -0.5).to(DEV)
    w_in = (torch.randn(E, d, 2 * f, generator=g) * d ** -0.5).to(dt).to(DEV)
    w_out = (torch.randn(E, f, d, generator=g) * f ** -0.5).to(dt).to(DEV)
    dy = torch.randn(T, d, generator=g).to(dt).to(DEV)
    block = laga.RoutedExperts(E, 2, score=score, io_dtype=io, device=DEV)
    y0 = block.forward(h, w_router, w_in, w_out)
    g0 = block.backward(dy)
    h[7, 200] = NAN
    y = block.forward(h, w_router, w_in, w_out)
    g1 = block.backward(dy)
    laga._lib.sync_check()
    rest = torch.arange(T, device=DEV) != 7
    assert y[7].isnan().all() and g1["dh"][7].isnan().all()
    assert torch.equal(y[rest], y0[rest]) and torch.equal(g1["dh"][rest], g0["dh"][rest])
    assert g1["dw_router"].isnan().all()
    # the token has no row: the experts' weights learn nothing from it
    assert torch.isfinite(g1["dw_in"]).all() and torch.isfinite(g1["dw_out"]).all()
