"""Calls on experts' rows that a program may make and the other tests do not:
trimmed routes, empty batches, inputs of other shapes and strides, one rank's
experts after the other's.

Tolerances: sums in fp32 of two ranks' parts differ from the whole's by the
roundings of at most top_k additions, 2^-24 of the terms' magnitudes each."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weights(d, f, E, dt, seed=0):
    g = _gen(seed)
    return [t.to(DEV) for t in (torch.randn(d, E, generator=g) * d ** -0.5,
                                (torch.randn(E, d, 2 * f, generator=g) * d ** -0.5).to(dt),
                                (torch.randn(E, f, d, generator=g) * f ** -0.5).to(dt))]


@pytest.mark.parametrize("align", [1, 128])
def test_trimmed_routes(align):
    """The same rows without the spare ones: every call gives the same values."""
    laga = _laga()
    T, E, k, d, f = 70, 6, 2, 256, 128
    l = torch.randn(T, E, generator=_gen(1))
    l[:30] = -float("inf")
    r = laga.Router(E, k, align=align, device=DEV).forward(l.to(DEV))
    t = r.trimmed()
    used = int(r.start[-1])
    assert t.rows == used < r.rows and t.pair.is_contiguous() and torch.equal(t.pair, r.pair[:used])
    assert t.tokens == T and t.top_k == k and t.experts == E and t.align == align
    x8 = laga.pack8(torch.randn(T, d, generator=_gen(2)).to(DEV))
    _, w_in, w_out = _weights(d, f, E, torch.bfloat16)
    w8 = laga.pack_weight8(w_in), laga.pack_weight8(w_out)
    dout = torch.randn(T, d, generator=_gen(3)).bfloat16().to(DEV)

    def run(r):
        xs = laga.spread8(x8, r)
        gu = laga.linear8(xs, w8[0], routes=r)
        a8 = laga.swiglu8(gu, routes=r)
        y = laga.linear8(a8, w8[1], routes=r)
        out = laga.combine(y, r)
        dy, dw = laga.combine_grad(dout, r, y=y)
        da = laga.linear8_dx(laga.pack8(dy, routes=r), w8[1], routes=r)
        dgu = laga.swiglu8_grad(gu, da, routes=r)
        grads = [laga.weight_grad8(a8, dy, routes=r)] if align == 128 else []
        return [out, dw, *grads], [xs.data, gu, a8.data, y, dy, da, dgu]

    a, b = run(r), run(t)
    laga._lib.sync_check()
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(len(y) == used and torch.equal(x[:used], y) for x, y in zip(a[1], b[1]))
    none = laga.Router(E, k, align=align, device=DEV).forward(
        torch.full((T, E), -float("inf"), device=DEV)).trimmed()
    assert none.rows == 0 and not laga.combine(torch.empty(0, d, device=DEV), none).any()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_no_tokens(io):
    laga = _laga()
    dt = dict(bf16=torch.bfloat16, fp32=torch.float32)[io]
    d, f, E = 256, 64, 4
    block = laga.RoutedExperts(E, 2, io_dtype=io, device=DEV)
    for shape in ((0, d), (3, 0, d)):
        y = block.forward(torch.empty(shape, dtype=dt, device=DEV), *_weights(d, f, E, dt))
        g = block.backward(torch.empty(shape, dtype=dt, device=DEV))
        laga._lib.sync_check()
        assert y.shape == shape and g["dh"].shape == shape
        for n, s in (("dw_router", (d, E)), ("dw_in", (E, d, 2 * f)), ("dw_out", (E, f, d))):
            assert g[n].shape == s and not g[n].any(), n


def test_every_token_masked():
    """No row in use at all: zero outputs and gradients."""
    laga = _laga()
    d, f, E = 256, 64, 4
    block = laga.RoutedExperts(E, 2, device=DEV)
    h = torch.randn(50, d, generator=_gen(4)).bfloat16().to(DEV)
    y = block.forward(h, *_weights(d, f, E, torch.bfloat16),
                      bias=torch.full((E,), -float("inf"), device=DEV))
    g = block.backward(h)
    laga._lib.sync_check()
    assert not y.any() and not any(v.any() for v in g.values())


def test_inputs_of_other_shapes_and_strides():
    laga = _laga()
    d, f, E = 256, 64, 4
    w = _weights(d, f, E, torch.bfloat16)
    h = torch.randn(6, 20, 2 * d, generator=_gen(5)).bfloat16().to(DEV)[..., ::2]
    dy = torch.randn(20, 6, d, generator=_gen(6)).bfloat16().to(DEV).transpose(0, 1)
    assert not h.is_contiguous() and not dy.is_contiguous()
    block = laga.RoutedExperts(E, 2, device=DEV)
    y = block.forward(h, *w)
    g = block.backward(dy)
    flat = laga.RoutedExperts(E, 2, device=DEV)
    y2 = flat.forward(h.reshape(-1, d).contiguous(), *w)
    g2 = flat.backward(dy.reshape(-1, d).contiguous())
    laga._lib.sync_check()
    assert y.shape == h.shape and torch.equal(y.reshape(-1, d), y2)
    assert torch.equal(g["dh"].reshape(-1, d), g2["dh"])
    assert all(torch.equal(g[n], g2[n]) for n in ("dw_router", "dw_in", "dw_out"))


def test_weights_packed_without_their_backward_order():
    laga = _laga()
    d, f, E = 256, 64, 4
    w_router, w_in, w_out = _weights(d, f, E, torch.bfloat16)
    block = laga.RoutedExperts(E, 2, device=DEV)
    h = torch.randn(9, d, generator=_gen(7)).bfloat16().to(DEV)
    block.forward(h, w_router, laga.pack_weight8(w_in, backward=False),
                  laga.pack_weight8(w_out, backward=False))
    with pytest.raises(ValueError, match="backward order"):
        block.backward(h)
    laga._lib.sync_check()


@pytest.mark.parametrize("align", [1, 128])
def test_two_ranks_parts_add_up(align):
    """The experts dealt out to two routers' shards, one after the other."""
    laga = _laga()
    T, E, k, d, f = 90, 6, 3, 256, 128
    l = torch.randn(T, E, generator=_gen(8)).to(DEV)
    x8 = laga.pack8(torch.randn(T, d, generator=_gen(9)).to(DEV))
    _, w_in, w_out = _weights(d, f, E, torch.float32)

    def part(first, count):
        r = laga.Router(E, k, shard=(first, count), align=align, device=DEV).forward(l)
        wi, wo = (laga.pack_weight8(w[first:first + count].contiguous()) for w in (w_in, w_out))
        gu = laga.linear8(laga.spread8(x8, r), wi, routes=r, dtype=torch.float32)
        y = laga.linear8(laga.swiglu8(gu, routes=r), wo, routes=r, dtype=torch.float32)
        return laga.combine(y, r), laga.combine(y.abs(), r)

    (whole, mag), (a, _), (b, _) = part(0, E), part(0, 2), part(2, 4)
    laga._lib.sync_check()
    assert ((a + b - whole).abs() <= 2 * (k + 1) * 2.0 ** -24 * mag).all()
