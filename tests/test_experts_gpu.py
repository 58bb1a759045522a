"""Routing, 8-bit products and the experts' rows on the GPU against the fp64
oracle: every option, odd sizes, experts without rows, tokens without experts.

Tolerances.  A product of 8-bit values is exact in fp32 (4 + 4 significant
bits).  A sum of n terms in fp32 is off by at most n u of the terms' magnitudes,
u = 2^-24 rounded and 2^-23 truncated, as the tensor cores' additions may be;
checks allow (n + 64) 2^-23.  An output's own rounding is half a step: 2^-8
(bf16) or 2^-24 (fp32) of its value."""

import numpy as np
import pytest
import torch

from laga_inputs import as_f64
from oracle import experts as oex
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _sync():
    _laga()._lib.sync_check()


def _gen(*seed):
    return torch.Generator().manual_seed(sum(s * 7919 ** i for i, s in enumerate(seed)))


# ------------------------------------------------------------------ routing
def _route(T, E, k, *, bias=True, io="fp32", logits=None, shard=None, align=128, seed=0, **kw):
    """Both sides of one forward and backward; returns the device Routes."""
    laga = _laga()
    g = _gen(T, E, k, seed)
    if logits is None:
        logits = 1.5 * torch.randn(T, E, generator=g)
    logits = logits.to(DT[io])
    if bias is True:
        bias = 0.1 * torch.randn(E, generator=g)
    r = laga.Router(E, k, io_dtype=io, shard=shard, align=align, device=DEV, **kw)
    d_logits = logits.to(DEV)
    out = r.forward(d_logits, None if bias is None else bias.to(DEV))
    dweight = torch.randn(T, k, generator=g)
    dl = r.backward(d_logits, out, dweight.to(DEV))
    _sync()

    ref = dict(score=kw.get("score", "sigmoid"), renormalise=kw.get("renormalise", True),
               scale=kw.get("scale", 1.0))
    groups = kw.get("groups", 1)
    l64 = as_f64(logits)
    expert, weight = oex.choose(l64, None if bias is None else as_f64(bias), top_k=k, groups=groups,
                                top_groups=kw.get("top_groups", groups), **ref)
    first, local = shard or (0, E)
    row, pair, start = oex.order(expert, first=first, local=local, align=align, rows=out.rows)
    for name, want in (("expert", expert), ("row", row), ("pair", pair), ("start", start)):
        got = getattr(out, name).cpu().numpy()
        assert np.array_equal(got, want), (name, np.argwhere(got != want)[:4].tolist())
    # a score is within 8 units of the last place (and its exponent's rounding,
    # |l - max| of them), a sum of k and a division each within as many
    span = np.where(np.isfinite(l64), np.abs(l64), 0.0).max(initial=0.0)
    tol = (24 + 4 * k + 4 * span) * 2.0 ** -24
    got = as_f64(out.weight)
    assert np.array_equal(np.isnan(got), np.isnan(weight))
    ok = ~np.isnan(weight)
    assert (np.abs(got - weight)[ok] <= tol * np.abs(weight[ok]) + 1e-37).all()
    want = oex.route_bwd(l64, expert, as_f64(dweight), **ref)
    # the differences in it are of terms no larger than |dw| scale / D each; the
    # oracle's largest entry stands for them
    s = oex.scores(l64, ref["score"])
    top = np.zeros(T)
    for t in range(T):
        e = expert[t][expert[t] >= 0]
        if len(e):
            D = s[t, e].sum() + oex.TINY if ref["renormalise"] else 1.0
            top[t] = ref["scale"] * np.abs(as_f64(dweight)[t]).max() / D * s[t, e].max() * k
    err = np.abs(as_f64(dl) - want)
    finite = np.isfinite(want)
    lim = (2 * tol * top[:, None] + HALF[io] * np.abs(want) + 1e-37)
    assert (err <= lim)[finite].all(), float((err / lim)[finite].max())
    return out


@pytest.mark.parametrize("T", [1, 2, 31, 33, 700])
@pytest.mark.parametrize("E,k,groups,top_groups", [(256, 8, 8, 4), (8, 2, 1, 1), (1, 1, 1, 1),
                                                   (40, 6, 4, 2), (65, 7, 5, 3), (33, 32, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route(T, E, k, groups, top_groups, score):
    _route(T, E, k, groups=groups, top_groups=top_groups, score=score, scale=2.5)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("E,k", [(512, 32), (1000, 10), (1024, 8), (300, 4)])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_many_experts(E, k, io, renormalise):
    _route(130, E, k, io=io, renormalise=renormalise, bias=None if E == 512 else True,
           groups=4 if E % 32 == 0 else 1, top_groups=2 if E % 32 == 0 else 1)


def test_route_groups_of_32_and_of_one():
    _route(50, 64, 5, groups=32, top_groups=7)
    _route(50, 32, 3, groups=32, top_groups=3)
    _route(50, 320, 8, groups=10, top_groups=10, score="softmax")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_go_to_the_lowest_index(io, score):
    """Logits on a coarse grid, with and without biases on one: many equal
    scores, and many that differ by less than fp32 shows."""
    g = _gen(5)
    l = torch.randint(-2, 3, (400, 64), generator=g).float()
    _route(400, 64, 6, io=io, score=score, logits=l, bias=None, groups=8, top_groups=3)
    _route(400, 64, 6, io=io, score=score, logits=l,
           bias=torch.randint(-1, 2, (64,), generator=g) / 8.0, groups=8, top_groups=3)
    _route(33, 64, 6, io=io, score=score, logits=torch.zeros(33, 64), bias=None)
    # scores next to one: fp32 shows no difference from a logit of 17 on
    _route(100, 64, 6, io=io, score=score, logits=16.0 + 0.125 * torch.randint(
        0, 60, (100, 64), generator=g).float(), bias=None)


def test_route_close_scores_in_64_bits():
    """Pairs of experts whose sums of score and bias differ by less than one
    unit in the last place of fp32, in either direction."""
    g = _gen(6)
    T, E = 500, 32
    l = torch.randn(T, E, generator=g)
    b = torch.zeros(E)
    b[1::2] = 0.03125
    # logit of the odd neighbour such that s + b is the even one's, up to rounding
    s = torch.sigmoid(l[:, 0::2].double()) - 0.03125
    l[:, 1::2] = torch.where(s > 0.01, torch.log(s.clamp(min=0.01) / (1 - s.clamp(min=0.01))),
                             l[:, 1::2].double()).float()
    _route(T, E, 8, logits=l, bias=b)


def test_route_close_groups_in_64_bits():
    """Groups whose two best sums differ by less than fp32 shows: large biases
    of both signs that cancel within a group, and equal groups."""
    g = _gen(12)
    T, E, G = 600, 64, 8
    l = torch.randn(T, 1, 8, generator=g).repeat(1, G, 1)      # every group the same logits
    l[:, 1::2] += 1e-6 * torch.randn(T, G // 2, 8, generator=g)
    b = torch.zeros(G, 8)
    b[:, 0], b[:, 1] = 100.0, -90.0 + torch.arange(8) * 2.0 ** -17
    for bias in (b.reshape(-1), None):
        for score in ("sigmoid", "softmax"):
            _route(T, E, 4, logits=l.reshape(T, E), bias=bias, groups=G, top_groups=3, score=score)


def test_route_masked_experts_and_tokens():
    g = _gen(7)
    l = torch.randn(300, 48, generator=g)
    l[::5] = -float("inf")                       # padding tokens
    l[1::5, 3:] = -float("inf")                  # fewer experts on than choices
    l[2::5, 8:40] = -float("inf")                # whole groups off
    l[3::5, ::2] = -float("inf")
    b = 0.1 * torch.randn(48, generator=g)
    b[7] = -float("inf")
    b[9] = float("inf")
    for score in ("sigmoid", "softmax"):
        for groups, top in ((1, 1), (6, 2)):
            _route(300, 48, 5, logits=l, bias=b, score=score, groups=groups, top_groups=top)
    _route(40, 48, 5, logits=torch.full((40, 48), -float("inf")))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_values_far_out(score):
    g = _gen(8)
    l = 60.0 * torch.randn(200, 64, generator=g)
    _route(200, 64, 4, logits=l, score=score, bias=None)
    l = torch.randn(60, 64, generator=g)
    l[3, 5] = float("nan")
    l[7, 9] = float("inf")
    l[9, :] = float("nan")
    b = 0.1 * torch.randn(64, generator=g)
    laga = _laga()
    r = laga.Router(64, 4, score=score, groups=4, top_groups=2, device=DEV)
    out = r.forward(l.to(DEV), b.to(DEV))
    e, w = oex.choose(as_f64(l), as_f64(b), top_k=4, groups=4, top_groups=2, score=score)
    assert np.array_equal(out.expert.cpu().numpy(), e)
    assert np.array_equal(np.isnan(as_f64(out.weight)), np.isnan(w))
    assert (e[9] == -1).all() and np.isnan(w[3]).all()


@pytest.mark.parametrize("shard", [(0, 32), (96, 32), (224, 32), (5, 1), (200, 56)])
@pytest.mark.parametrize("align", [1, 128])
def test_route_on_one_rank(shard, align):
    _route(257, 256, 8, shard=shard, align=align, groups=8, top_groups=4)


def test_route_many_tokens_twice_the_same():
    a = _route(5000, 64, 6, align=1)
    b = _route(5000, 64, 6, align=1)
    for x, y in zip(a[:5], b[:5]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,E,k,groups,score,io", [(200003, 64, 6, 4, "sigmoid", "fp32"),
                                                   (70001, 1000, 32, 1, "softmax", "fp32"),
                                                   (40000, 256, 8, 8, "sigmoid", "bf16")])
def test_route_a_long_batch(T, E, k, groups, score, io):
    """Chunks of more pairs than a block has threads, against torch in 64 bits."""
    laga = _laga()
    l = torch.randn(T, E, generator=torch.Generator(DEV).manual_seed(T), device=DEV).to(DT[io])
    b = 0.05 * torch.randn(E, generator=torch.Generator(DEV).manual_seed(E), device=DEV)
    top_groups = max(1, groups // 2)
    r = laga.Router(E, k, score=score, groups=groups, top_groups=top_groups, io_dtype=io, device=DEV)
    out = r.forward(l, b)
    _sync()
    s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), dim=1)
    c = s + b.double()
    if top_groups < groups:
        two = c.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        best = two.sort(dim=1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        c = c.masked_fill(~keep.repeat_interleave(E // groups, dim=1), -float("inf"))
    expert = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(out.expert.long(), expert)
    w = s.gather(1, expert)
    w = w / w.sum(dim=1, keepdim=True)
    assert ((out.weight.double() - w).abs() <= (24 + 4 * k + 4 * 8) * 2.0 ** -24 * w).all()
    flat = expert.reshape(-1)
    count = torch.bincount(flat, minlength=E)
    start = torch.cat([count.new_zeros(1), ((count + 127) // 128 * 128).cumsum(0)])
    assert torch.equal(out.start.long(), start)
    by = torch.argsort(flat, stable=True)
    before = torch.cat([count.new_zeros(1), count.cumsum(0)])[:-1]
    at = start[flat[by]] + torch.arange(len(by), device=DEV) - before[flat[by]]
    pair = torch.full((out.rows,), -1, dtype=torch.long, device=DEV)
    pair[at] = by
    assert torch.equal(out.pair.long(), pair)
    assert torch.equal(out.row.reshape(-1)[by].long(), at)


def test_route_no_tokens():
    r = _laga().Router(16, 2, device=DEV)
    out = r.forward(torch.zeros(0, 16, device=DEV))
    assert out.start.tolist() == [0] * 17 and out.rows == 0
    assert r.backward(torch.zeros(0, 16, device=DEV), out, torch.zeros(0, 2, device=DEV)).shape == (0, 16)


def test_route_backward_of_a_repeated_expert():
    g = _gen(9)
    l, dw = torch.randn(9, 16, generator=g), torch.randn(9, 3, generator=g)
    e = torch.randint(0, 16, (9, 3), generator=g, dtype=torch.int32)
    e[:, 2] = e[:, 0]
    e[4, 1] = -1
    laga = _laga()
    for score in ("sigmoid", "softmax"):
        r = laga.Router(16, 3, score=score, scale=0.5, device=DEV)
        out = r.forward(l.to(DEV))._replace(expert=e.to(DEV))
        got = as_f64(r.backward(l.to(DEV), out, dw.to(DEV)))
        want = oex.route_bwd(as_f64(l), e.numpy(), as_f64(dw), score=score, scale=0.5)
        assert np.abs(got - want).max() <= 64 * 2.0 ** -24 * np.abs(want).max()


# ------------------------------------------------------------------ products
def _codes(rows, d, g, scale=True):
    x = torch.randn(rows, d, generator=g)
    if scale:
        x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g))
    return ores.pack(as_f64(x))


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _seg(counts, align):
    start = [0]
    for c in counts:
        start.append(start[-1] + -(-c // align) * align)
    return np.array(start, np.int32)


def _routes(counts, align, spare=0):
    """Routes of one choice a token whose experts get so many rows; ``spare``
    rows behind the last one in use."""
    laga = _laga()
    start = _seg(counts, align)
    expert = np.repeat(np.arange(len(counts), dtype=np.int32), counts)
    row, pair, st = oex.order(expert[:, None], local=len(counts), align=align,
                              rows=int(start[-1]) + spare)
    assert np.array_equal(st, start)
    w = torch.ones(len(expert), 1, device=DEV)
    return laga.Routes(_dev(expert[:, None]), w, _dev(row), _dev(pair), _dev(start), align)


def _check_sum(got, want, mag, n, io, what):
    lim = (n + 64) * 2.0 ** -23 * mag + HALF[io] * np.abs(want) + 1e-37
    err = np.abs(as_f64(got) - want)
    assert np.array_equal(np.isnan(as_f64(got)), np.isnan(want)), what
    ok = ~np.isnan(want)
    assert (err <= lim)[ok].all(), (what, float((err / lim)[ok].max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,K,N", [(1, 1, 1), (1, 128, 128), (2, 130, 257), (3, 1001, 577),
                                   (1, 2048, 384), (2, 64, 1)])
def test_pack_weight_bit_for_bit(E, K, N, dtype):
    laga = _laga()
    w = (torch.randn(E, K, N, generator=_gen(E, K, N)) * 0.03).to(DT[dtype])
    w8 = laga.pack_weight8(w.to(DEV))
    fwd, bwd = oex.pack_weight(as_f64(w))
    assert np.array_equal(w8.fwd.cpu().numpy(), fwd) and np.array_equal(w8.bwd.cpu().numpy(), bwd)
    v = ores.unpack(bwd, N).reshape(E, K, N)
    assert np.array_equal(as_f64(w8.unpack()), v)
    only = laga.pack_weight8(w.to(DEV), backward=False)
    assert only.bwd is None and np.array_equal(as_f64(only.unpack(torch.float32)), v)
    assert torch.equal(laga.pack_weight8(w[0].to(DEV)).fwd, w8.fwd[:N])


def test_pack_weight_borders():
    w = torch.zeros(1, 256, 256)
    w[0, 0, 0], w[0, 130, 3], w[0, 3, 130] = 448.0, float("inf"), 2.0 ** -130
    w[0, 200, 200] = 3.0e38
    w8 = _laga().pack_weight8(w.to(DEV))
    fwd, bwd = oex.pack_weight(as_f64(w))
    assert np.array_equal(w8.fwd.cpu().numpy(), fwd) and np.array_equal(w8.bwd.cpu().numpy(), bwd)
    v = as_f64(w8.unpack())[0]
    assert np.isnan(v[128:, :128]).all() and v[0, 0] == 448.0 and np.isfinite(v[:, 128:]).all()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,K,N", [(1, 1, 1), (1, 7168, 256), (3, 129, 130), (16, 512, 1001),
                                      (17, 128, 64), (64, 2048, 96), (65, 300, 255),
                                      (127, 640, 128), (129, 1001, 257), (256, 896, 512),
                                      (257, 4096, 513), (300, 130, 7), (1000, 384, 1536), (130, 300, 200),
                                      (224, 2100, 1000), (225, 3000, 36), (449, 140, 8)])
def test_linear(rows, K, N, io):
    laga = _laga()
    g = _gen(rows, K, N)
    x, w = _codes(rows, K, g), torch.randn(1, K, N, generator=g) * K ** -0.5
    fwd, bwd = oex.pack_weight(as_f64(w))
    w8 = laga.Weight8((K, N), _dev(fwd), _dev(bwd))
    y = laga.linear8(laga.Checkpoint8(_dev(x), K), w8, dtype=DT[io])
    _sync()
    _check_sum(y, *oex.mm8(x, fwd, K, N), K, io, "y")
    dy = _codes(rows, N, g)
    dx = laga.linear8_dx(laga.Checkpoint8(_dev(dy), N), w8, dtype=DT[io])
    _sync()
    _check_sum(dx, *oex.mm8(dy, bwd, N, K), N, io, "dx")


COUNTS = [(0, 5, 0, 130, 1), (300,), (0, 0, 7), (64, 128, 1, 0, 257, 33), (1,) * 40, (0, 700, 2)]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("io,K,N", [("bf16", 256, 384), ("fp32", 333, 129)])
def test_linear_by_expert(counts, align, io, K, N):
    """Rows behind the last one in use keep what they held."""
    laga = _laga()
    g = _gen(len(counts), align, K)
    r = _routes(counts, align, spare=37)
    E, rows = len(counts), r.rows
    x, w = _codes(rows, K, g), torch.randn(E, K, N, generator=g) * K ** -0.5
    fwd, bwd = oex.pack_weight(as_f64(w))
    start = r.start.cpu().numpy()
    y = torch.full((rows, N), 7.0, dtype=DT[io], device=DEV)
    nb = laga._lib.mm8_workspace_bytes(rows, K, N, E, io)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=DEV)
    d_x, d_w = _dev(x), _dev(fwd)
    laga._lib.mm8(rows, K, N, E, io, d_x.data_ptr(), d_w.data_ptr(), r.start.data_ptr(), 0,
                  y.data_ptr(), ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    _sync()
    want, mag = oex.mm8(x, fwd, K, N, start)
    _check_sum(y[:start[-1]], want[:start[-1]], mag[:start[-1]], K, io, "y")
    assert (y[start[-1]:] == 7.0).all()
    w8 = laga.Weight8((E, K, N), d_w, _dev(bwd))
    live = (r.pair >= 0)[:, None]
    by_routes = laga.linear8(laga.Checkpoint8(d_x, K), w8, routes=r, dtype=DT[io])
    _sync()
    assert torch.equal(by_routes[:start[-1]], torch.where(live, y, 0.0)[:start[-1]])
    dy = _codes(rows, N, g)
    dx = laga.linear8_dx(laga.Checkpoint8(_dev(dy), N), w8, routes=r, dtype=DT[io])
    _sync()
    want, mag = oex.mm8(dy, bwd, N, K, start)
    want = np.where(live.cpu().numpy(), want, 0.0)
    _check_sum(dx[:start[-1]], want[:start[-1]], mag[:start[-1]], N, io, "dx")


def test_linear_values_without_an_end_stay_in_their_rows():
    """A NaN group of a row makes that row NaN, a NaN block of one expert's
    weight that expert's columns, and nothing else."""
    laga = _laga()
    g = _gen(11)
    r = _routes((70, 0, 140), 1)
    x, w = torch.randn(r.rows, 256, generator=g), torch.randn(3, 256, 384, generator=g)
    x[5, 130], x[75, 3] = float("nan"), float("inf")
    w[2, 200, 260] = float("inf")
    x8, (fwd, bwd) = ores.pack(as_f64(x)), oex.pack_weight(as_f64(w))
    y = laga.linear8(laga.Checkpoint8(_dev(x8), 256), laga.Weight8((3, 256, 384), _dev(fwd)),
                     routes=r, dtype=torch.float32)
    _sync()
    want, mag = oex.mm8(x8, fwd, 256, 384, r.start.cpu().numpy())
    assert np.isnan(want[5]).all() and np.isnan(want[70:, 256:]).all() and np.isfinite(want[71, :256]).all()
    _check_sum(y, want, mag, 256, "fp32", "y")


@pytest.mark.parametrize("dy_io", ["bf16", "fp32"])
@pytest.mark.parametrize("counts", [(0, 5, 0, 130, 1), (300,), (129, 128, 1, 0, 900, 33), (0, 0)])
@pytest.mark.parametrize("d,n", [(384, 200), (130, 577), (2048, 256), (1, 1)])
def test_weight_grad_by_expert(counts, d, n, dy_io):
    laga = _laga()
    g = _gen(len(counts), d, n)
    r = _routes(counts, 128, spare=128)
    live = (r.pair.cpu() >= 0)[:, None]
    x = torch.randn(r.rows, d, generator=g) * live
    dy = (torch.randn(r.rows, n, generator=g) * live).to(DT[dy_io])
    dy[int(r.start[-1]):] = float("nan")          # never read
    gamma = torch.randn(d, generator=g)
    x8 = ores.pack(as_f64(x))
    dw = laga.weight_grad8(laga.Checkpoint8(_dev(x8), d), dy.to(DEV), gamma.to(DEV), routes=r)
    _sync()
    want, mag = oex.weight_grad(x8, d, as_f64(dy), r.start.cpu().numpy(), as_f64(gamma))
    _check_sum(dw, want, mag, max(counts), "fp32", "dw")
    again = laga.weight_grad8(laga.Checkpoint8(_dev(x8), d), dy.to(DEV), gamma.to(DEV), routes=r)
    assert torch.equal(dw, again)


# ------------------------------------------------------------------ rows back
def _batch(T, E, k, align, seed=0, padded=True):
    """Routes of a router over random logits, some tokens padding, and the
    same as NumPy."""
    g = _gen(T, E, k, seed)
    l = torch.randn(T, E, generator=g)
    if padded and T > 2:
        l[1] = -float("inf")
        l[2, 1:] = -float("inf")
    r = _laga().Router(E, k, align=align, device=DEV).forward(l.to(DEV))
    return r, {n: getattr(r, n).cpu().numpy() for n in ("row", "pair", "start")}, as_f64(r.weight)


@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("T,E,k,d", [(1, 8, 2, 128), (37, 8, 3, 1001), (130, 16, 8, 2048), (5, 4, 4, 7168)])
def test_spread(T, E, k, d, align):
    laga = _laga()
    r, host, _ = _batch(T, E, k, align)
    x8 = _codes(T, d, _gen(T, d))
    out = laga.spread8(laga.Checkpoint8(_dev(x8), d), r)
    _sync()
    used = host["start"][-1]
    want = oex.spread(x8, host["pair"], k)
    assert np.array_equal(out.data.cpu().numpy()[:used], want[:used])
    assert out.shape == (r.rows, d)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("T,E,k,d", [(1, 8, 2, 128), (37, 8, 3, 1001), (130, 16, 8, 2048),
                                     (64, 40, 32, 8), (5, 4, 1, 16384), (3, 4, 2, 1)])
def test_combine_and_its_gradients(T, E, k, d, align, io):
    laga = _laga()
    r, host, weight = _batch(T, E, k, align)
    g = _gen(T, d, 1)
    y = torch.randn(r.rows, d, generator=g).to(DT[io])
    y[torch.from_numpy(host["pair"]) < 0] = float("nan")      # of no pair: not read
    dout = torch.randn(T, d, generator=g).to(DT[io])
    y64, d64 = as_f64(y), as_f64(dout)
    for weighted in (True, False):
        w = weight if weighted else np.ones_like(weight)
        out = laga.combine(y.to(DEV), r, weighted=weighted)
        _sync()
        want, mag = oex.combine(y64, w, host["row"])
        lim = (k + 2) * 2.0 ** -24 * mag + HALF[io] * np.abs(want) + 1e-37
        assert (np.abs(as_f64(out) - want) <= lim).all()
        dy, dw = laga.combine_grad(dout.to(DEV), r, y=y.to(DEV), weighted=weighted)
        _sync()
        used = host["start"][-1]
        want, dwant, dmag = oex.combine_bwd(d64, y64, w, host["row"])
        zero = host["pair"][:used] < 0
        got = as_f64(dy)[:used]
        assert (got[zero] == 0).all()
        lim = (2.0 ** -24 + HALF[io]) * np.abs(want[:used]) + 1e-37
        assert (np.abs(got - want[:used]) <= lim)[~zero].all()
        assert (np.abs(as_f64(dw) - dwant) <= (d + 2) * 2.0 ** -24 * dmag + 1e-37).all()
        only, none = laga.combine_grad(dout.to(DEV), r, weighted=weighted)
        assert none is None and torch.equal(only[:used], dy[:used])


# ------------------------------------------------------------------ activation
def _flips(got, want, exact):
    """Codes may differ from the oracle's where the exact value lies within
    fp32's error of the border between two: the value is then one of the two
    neighbours of the exact one.  Returns how many differ."""
    diff = got != want
    # both are a half step (2^-4 of the value, or of the least normal code) away
    assert (np.abs(got - exact)[diff] <= np.abs(want - exact)[diff] * (1 + 1e-4) + 1e-30).all()
    return int(diff.sum())


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,f", [(1, 1), (3, 129), (37, 1001), (130, 2048), (257, 128), (2, 16384)])
def test_swiglu_and_its_gradient(rows, f, io):
    laga = _laga()
    g = _gen(rows, f)
    gu = (2.0 * torch.randn(rows, 2 * f, generator=g)).to(DT[io])
    da = torch.randn(rows, f, generator=g).to(DT[io])
    ck = laga.swiglu8(gu.to(DEV))
    dgu = laga.swiglu8_grad(gu.to(DEV), da.to(DEV))
    _sync()
    a = oex.swiglu(as_f64(gu))
    got, want = as_f64(ck.unpack(torch.float32)), ores.unpack(ores.pack(a), f)
    assert ck.shape == (rows, f)
    # a value in 10^5 lies within 2^-22 of a border (steps are 2^-3 apart at most)
    assert _flips(got, want, a) <= 2 + rows * f * 1e-4
    cols, pitch = ores.row_layout(f)
    assert (ck.data[:, cols + cols // 128:] == 0).all()
    ref = oex.swiglu_bwd(as_f64(gu), as_f64(da))
    # each factor is within 8 units of the last place; 1 + g (1 - s) is a sum of
    # terms up to 1 + |g|
    g64, u64 = as_f64(gu)[:, :f], as_f64(gu)[:, f:]
    mag = np.abs(as_f64(da)) * np.concatenate([np.abs(u64) * (1 + np.abs(g64)), np.abs(g64)]).reshape(2, rows, f)
    lim = 24 * 2.0 ** -24 * np.concatenate([mag[0], mag[1]], axis=1) + HALF[io] * np.abs(ref) + 1e-37
    assert (np.abs(as_f64(dgu) - ref) <= lim).all()


def test_swiglu_values_far_out():
    laga = _laga()
    f = 256
    gu = torch.zeros(6, 2 * f)
    gu[0, :f], gu[0, f:] = -200.0, 3.0            # shut
    gu[1, :f], gu[1, f:] = 200.0, 3.0
    gu[2, 5], gu[2, f + 5] = float("nan"), 1.0
    gu[3, 130], gu[3, f + 130] = 1.0, float("inf")
    gu[4, :f], gu[4, f:] = 1e30, 1e30             # overflows
    ck = laga.swiglu8(gu.to(DEV))
    v = as_f64(ck.unpack(torch.float32))
    assert (v[0] == 0).all() and (v[1] == ores.unpack(ores.pack(np.full((1, f), 600.0)), f)).all()
    assert np.isnan(v[2, :128]).all() and (v[2, 128:] == 0).all()
    assert np.isnan(v[3, 128:]).all() and (v[3, :128] == 0).all()
    assert np.isnan(v[4]).all() and (v[5] == 0).all()
    d = as_f64(laga.swiglu8_grad(gu[:2].to(DEV), torch.ones(2, f, device=DEV)))
    assert (d[0, :] == 0).all() and np.allclose(d[1, :f], 3.0) and np.allclose(d[1, f:], 200.0)


def test_swiglu_of_the_rows_in_use():
    laga = _laga()
    r, host, _ = _batch(50, 8, 2, 128)
    used = int(host["start"][-1])
    gu = torch.randn(r.rows, 512, generator=_gen(1)).to(DEV)
    a, b = laga.swiglu8(gu, routes=r), laga.swiglu8(gu)
    assert torch.equal(a.data[:used], b.data[:used])
    da = torch.randn(r.rows, 256, generator=_gen(2)).to(DEV)
    assert torch.equal(laga.swiglu8_grad(gu, da, routes=r)[:used], laga.swiglu8_grad(gu, da)[:used])
