"""The experts' oracle against closed forms, torch and finite differences."""

import numpy as np
import pytest
import torch

from oracle import experts as oex
from oracle import residual as ores


def _rng(seed=0):
    return np.random.default_rng(seed)


def _difference(f, x, g, eps=1e-6):
    """Directional derivative of sum(f(x) g) along a random direction, and that direction."""
    d = _rng(9).standard_normal(x.shape)
    return ((f(x + eps * d) - f(x - eps * d)) * g).sum() / (2 * eps), d


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient(score, renormalise):
    r = _rng(1)
    l, g = r.standard_normal((20, 12)), r.standard_normal((20, 3))
    kw = dict(score=score, renormalise=renormalise, scale=1.7)
    expert, weight = oex.choose(l, None, top_k=3, **kw)

    def weights(x):      # at fixed choice
        s = np.take_along_axis(oex.scores(x, score), expert.astype(int), axis=1)
        return 1.7 * (s / (s.sum(axis=1, keepdims=True) + oex.TINY) if renormalise else s)

    assert np.allclose(weights(l), weight)
    want, d = _difference(weights, l, g)
    assert np.isclose((oex.route_bwd(l, expert, g, **kw) * d).sum(), want, rtol=1e-6)


def test_choice_is_torch_topk_where_nothing_ties():
    r = _rng(2)
    l, b = r.standard_normal((50, 32)), 0.1 * r.standard_normal(32)
    e, _ = oex.choose(l, b, top_k=5, groups=4, top_groups=2)
    c = torch.sigmoid(torch.tensor(l)) + torch.tensor(b)
    best = c.view(50, 4, 8).topk(2, dim=2).values.sum(dim=2).topk(2, dim=1).indices
    keep = torch.zeros(50, 4, dtype=torch.bool).scatter_(1, best, True)
    c = c.masked_fill(~keep.repeat_interleave(8, dim=1), -1.0)
    assert np.array_equal(e, c.topk(5, dim=1).indices.numpy())


def test_choice_of_ties_and_masks():
    l = np.zeros((3, 6))
    l[1, :4] = -np.inf
    l[2] = -np.inf
    e, w = oex.choose(l, None, top_k=3)
    assert e.tolist() == [[0, 1, 2], [4, 5, -1], [-1, -1, -1]]
    assert np.allclose(w, [[1 / 3] * 3, [0.5, 0.5, 0], [0, 0, 0]])


def test_row_order():
    e = np.array([[2, 0], [0, 1], [2, -1]], np.int32)
    row, pair, start = oex.order(e, local=3, align=4, rows=14)
    assert start.tolist() == [0, 4, 8, 12]
    assert row.tolist() == [[8, 0], [1, 4], [9, -1]]
    assert pair.tolist() == [1, 2, -1, -1, 3, -1, -1, -1, 0, 4, -1, -1, -1, -1]
    row, pair, start = oex.order(e, first=1, local=2, align=1, rows=4)
    assert row.tolist() == [[1, -1], [-1, 0], [2, -1]] and start.tolist() == [0, 1, 3]


def test_weight_codes_are_torchs():
    w = _rng(3).standard_normal((2, 130, 200)) * 0.05
    fwd, bwd = oex.pack_weight(w)
    v = ores.unpack(bwd, 200).reshape(2, 130, 200)
    assert np.array_equal(ores.unpack(fwd, 130).reshape(2, 200, 130).transpose(0, 2, 1), v)
    for i, j in ((0, 0), (0, 128), (128, 0), (128, 128)):
        b = w[1, i:i + 128, j:j + 128]
        e = int(np.ceil(np.log2(np.abs(b).max() / 448.0)))
        q = torch.tensor(b / 2.0 ** e).float().to(torch.float8_e4m3fn).double().numpy() * 2.0 ** e
        assert np.array_equal(v[1, i:i + 128, j:j + 128], q)


def test_swiglu_gradient():
    r = _rng(4)
    gu, da = r.standard_normal((5, 14)), r.standard_normal((5, 7))
    assert np.allclose(oex.swiglu(gu), (torch.nn.functional.silu(torch.tensor(gu[:, :7])).numpy()
                                        * gu[:, 7:]))
    want, d = _difference(oex.swiglu, gu, da)
    assert np.isclose((oex.swiglu_bwd(gu, da) * d).sum(), want, rtol=1e-6)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_block_gradients(score):
    """The block without roundings: every gradient against differences."""
    r = _rng(5)
    T, d, f, E, k = 9, 6, 5, 4, 2
    x = dict(h=r.standard_normal((T, d)), w_router=r.standard_normal((d, E)),
             w_in=r.standard_normal((E, d, 2 * f)), w_out=r.standard_normal((E, f, d)))
    kw = dict(top_k=k, score=score, scale=1.3)
    dy = r.standard_normal((T, d))
    _, st = oex.block_fwd(x["h"], x["w_router"], None, x["w_in"], x["w_out"], exact=True, **kw)
    g = oex.block_bwd(st, dy)
    for name, grad in (("h", "dh"), ("w_router", "dw_router"), ("w_in", "dw_in"), ("w_out", "dw_out")):
        def f_of(v):
            y = dict(x, **{name: v})
            return oex.block_fwd(y["h"], y["w_router"], None, y["w_in"], y["w_out"], exact=True,
                                 **kw)[0]
        want, dirn = _difference(f_of, x[name], dy)
        assert np.isclose((g[grad] * dirn).sum(), want, rtol=1e-5), name


def test_bf16_rounding_is_torchs():
    v = _rng(6).standard_normal(1000) * 3.0 ** _rng(7).integers(-20, 20, 1000)
    assert np.array_equal(oex.bf16(v.astype(np.float32).astype(np.float64)),
                          torch.tensor(v.astype(np.float32)).to(torch.bfloat16).double().numpy())
