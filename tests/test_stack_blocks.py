"""What LagaResidualStack takes as a block: its own two kinds, blocks of the
user's own with their signatures, and wrappers around one, with no more than the
public calls.  The residual operators are computed by the oracle, on the CPU."""

import numpy as np
import pytest
import torch

import oracle
from test_sp_gloo import SMALL, OracleCompute
from test_stack_gloo import OracleResidualNorm, _layers, _unsharded

S, N_H, D = 12, 2, 7


@pytest.fixture
def block(monkeypatch):
    from sequence_latent_norm_gb300 import block
    monkeypatch.setattr(block, "ResidualNorm", OracleResidualNorm)
    return block


def _attention(block):
    return block.LagaAttentionBlock(OracleCompute(oracle.Dims(S=S, H=N_H, **SMALL)), N_H)


class Own:
    """A user's block: LagaAttentionBlock's calls, and nothing else of it."""

    def __init__(self, inner):
        self.inner, self.calls = inner, 0

    def forward(self, h, w_q, w_kva, gamma, w_kvb, w_o, cos, sin, *, kept=None, kept_gain=None):
        self.calls += 1
        return self.inner.forward(h, w_q, w_kva, gamma, w_kvb, w_o, cos, sin, kept=kept,
                                  kept_gain=kept_gain)

    def backward(self, dy):
        return self.inner.backward(dy)

    def _all_reduce(self, t, what):
        return t


class Wrapper:
    """A wrapper that hands on what it does not know."""

    def __init__(self, inner):
        self.inner, self.calls = inner, 0

    def forward(self, *a, **kw):
        self.calls += 1
        return self.inner.forward(*a, **kw)

    def __getattr__(self, name):
        return getattr(self.inner, name)


@pytest.mark.parametrize("kind", [Own, Wrapper])
def test_blocks_of_the_users_own(block, kind):
    rng = np.random.default_rng(4)
    layers = _layers(rng, 2, S, N_H, D, "none", "none")
    x, dx = rng.standard_normal((1, S, D)), rng.standard_normal((1, S, D))
    cos, sin = oracle.rope_tables(S, SMALL["d_rope"])
    norms = dict(norm_post="none", norm_pre="rms")
    want, want_dx, want_grads = _unsharded(x, dx, layers, oracle.Dims(S=S, H=N_H, **SMALL), cos, sin,
                                           norms)
    T = torch.from_numpy
    blocks = [kind(_attention(block)), _attention(block)]
    stack = block.LagaResidualStack(blocks, D, **norms)
    out = stack.forward(T(x), [{k: T(v) for k, v in w.items()} for w in layers], T(cos), T(sin))
    got_dx, got = stack.backward(T(dx))
    assert blocks[0].calls == 1                  # its own forward, not the one inside
    tol = dict(rtol=1e-10, atol=1e-10)
    np.testing.assert_allclose(out.numpy(), want, **tol)
    np.testing.assert_allclose(got_dx.numpy(), want_dx, **tol)
    for g, ref in zip(got, want_grads):
        assert set(g) == set(ref)
        for k in g:
            np.testing.assert_allclose(g[k].numpy(), ref[k], **tol, err_msg=k)


class Experts:
    """RoutedExperts' signature, computing y = h."""

    def __init__(self):
        self.seen = []

    def forward(self, h, w_router, w_in, w_out, *, bias=None, kept=None, kept_gain=None):
        self.seen.append((w_router, w_in, w_out, bias))
        return h

    def backward(self, dy):
        return dict(dh=dy)

    def _all_reduce(self, t, what):
        return t


def _routed():
    import sequence_latent_norm_gb300 as laga

    class Routed(laga.RoutedExperts):
        """The framework's class with that forward (it needs a CUDA device)."""

        def forward(self, *a, **kw):
            self.fake = getattr(self, "fake", None) or Experts()
            return self.fake.forward(*a, **kw)

        def backward(self, dy):
            return self.fake.backward(dy)

    return Routed(4, 2, device="cuda:0")


@pytest.mark.parametrize("make", [Experts, lambda: Wrapper(Experts()), _routed])
@pytest.mark.parametrize("bias", [None, "b"])
def test_experts_among_attention_blocks(block, make, bias):
    rng = np.random.default_rng(5)
    T = torch.from_numpy
    attn = {k: T(v) for k, v in _layers(rng, 1, S, N_H, D, "none", "none")[0].items()}
    experts = dict(w_router=1, w_in=2, w_out=3, gamma_pre=attn["gamma_pre"], alpha=attn["alpha"])
    if bias:
        experts["bias"] = bias
    cos, sin = (T(t) for t in oracle.rope_tables(S, SMALL["d_rope"]))
    e = make()
    stack = block.LagaResidualStack([_attention(block), e], D)
    stack.forward(T(rng.standard_normal((1, S, D))), [attn, experts], cos, sin)
    _, grads = stack.backward(T(rng.standard_normal((1, S, D))))
    seen = e.fake.seen if hasattr(e, "fake") else e.seen
    assert seen == [(1, 2, 3, bias)]
    assert "dw_q" in grads[0] and set(grads[1]) == {"dalpha", "dgamma_pre"}


def test_one_dict_may_hold_a_whole_layer(block):
    """Attention and experts of a layer may share a dict of weights."""
    rng = np.random.default_rng(6)
    T = torch.from_numpy
    w = {k: T(v) for k, v in _layers(rng, 1, S, N_H, D, "none", "none")[0].items()}
    w.update(w_router=1, w_in=2, w_out=3)
    cos, sin = (T(t) for t in oracle.rope_tables(S, SMALL["d_rope"]))
    e = _routed()
    stack = block.LagaResidualStack([_attention(block), e], D)
    stack.forward(T(rng.standard_normal((1, S, D))), [w, w], cos, sin)
    assert e.fake.seen == [(1, 2, 3, None)]
