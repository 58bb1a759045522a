"""The residual operators' halves against both in one call, and what the
stack's weight gradients are taken from.

Bounds: u = 2^-24 (a rounding to fp32), U half a step of the I/O type; an
element of a row is within ROW = 128 u of the size of the terms that make it
(at most 96 additions of a statistic's chain and 32 roundings of its own)."""

import numpy as np
import pytest
import torch

from laga_inputs import as_f64, config, make_block_inputs
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
ROW = 128 * 2.0 ** -24


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


@pytest.mark.parametrize("d", [333, 640, 2048, 7168])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm_post,norm_pre,gate", [("none", "rms", "none"), ("rms", "layer", "full"),
                                                     ("layer", "rms", "token")])
def test_both_halves_in_one_call_are_the_two(norm_post, norm_pre, gate, dtype, d):
    """The input half takes x' before its rounding, a call of its own the
    rounded one: x' is the same, and h is apart by what that rounding moves."""
    laga = _laga()
    rows, eps, U = 160, 1e-5, HALF[dtype]
    g = torch.Generator(device=DEV).manual_seed(d)
    x, y = (torch.randn(rows, d, generator=g, device=DEV).to(DT[dtype]) for _ in range(2))
    kw = dict(alpha=0.5 + torch.rand(1, generator=g, device=DEV),
              gamma_post=0.5 + torch.rand(d, generator=g, device=DEV),
              gate=torch.randn(rows, 1 if gate == "token" else d, generator=g, device=DEV).to(DT[dtype]))
    gamma = 0.5 + torch.rand(d, generator=g, device=DEV)
    opts = dict(norm_post=norm_post, norm_pre=norm_pre, gate=gate, io_dtype=dtype, eps=eps,
                device=DEV)
    one = laga.ResidualNorm(d, **opts).forward(x, y, gamma_pre=gamma, **kw)
    post = laga.ResidualNorm(d, pre=False, **opts).forward(x, y, **kw)
    pre = laga.ResidualNorm(d, post=False, **opts).forward(post.x, gamma_pre=gamma)
    laga._lib.sync_check()
    a, b = as_f64(one.x), as_f64(post.x)
    # either is within ROW of its terms and one rounding of x'
    size = np.abs(as_f64(x)) + 5 * np.abs(as_f64(y)).max(axis=1, keepdims=True) * \
        as_f64(post.saved.stat_post)[:, 1:]
    assert (np.abs(a - b) <= 2 * U * np.abs(b) + 2 * ROW * size).all()
    # With x' off by e = U |x'| (and what the last line allows), x^ = (x' - mean)
    # r moves by r (e + mean e), and r by r rms(e) at most of itself.
    st = as_f64(pre.saved.stat_pre)
    e = 3 * U * np.abs(b) + 2 * ROW * size
    hat = np.abs(ores.hat(b, st))
    r = st[:, 1:]
    move = r * (e + e.mean(axis=1, keepdims=True)) + \
        hat * r * np.sqrt((e ** 2).mean(axis=1, keepdims=True)) * 1.1
    own = 2 * ROW * r * (np.abs(b) + np.abs(b).max(axis=1, keepdims=True)) * 3
    h = np.abs(as_f64(pre.h))
    off = np.abs(as_f64(one.h) - as_f64(pre.h))
    assert (off <= as_f64(gamma) * (move + own) + 2 * U * h * 1.01).all()


@pytest.mark.parametrize("layer", [0, 1])
def test_stack_weight_gradients_are_of_the_checkpoint_and_its_gain(layer):
    """dW_q and dW_kv_a of a layer are diag(gamma_pre) v^T dy of the values v
    that its checkpoint stands for and the gradients that its block's compute
    gives: within the weight gradient's own bound, (rows + 64) 2^-23 of the
    terms' magnitudes, which they pass nearly everywhere without the gain."""
    laga = _laga()
    from sequence_latent_norm_gb300.block import LagaAttentionBlock, LagaResidualStack
    n, d_model = 2, 192
    layers, grads = [], {}
    for i in range(n):
        wl = config(1, S=160, H=2, n_h_total=2, seed=60 + i)
        b = {k: v.to(DEV) for k, v in make_block_inputs(wl, d_model).items()}
        w = {k: b[k] for k in ("w_q", "w_kva", "gamma", "w_kvb", "w_o")}
        g = torch.Generator(device=DEV).manual_seed(i)
        w["gamma_pre"] = 0.5 + torch.rand(d_model, generator=g, device=DEV)
        w["alpha"] = torch.tensor([0.7], device=DEV)
        layers.append(w)
        if i == 0:
            x, dx, cos, sin = b["h"], b["dy"], b["cos"], b["sin"]
    blocks = [LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV)) for _ in range(n)]
    for i, blk in enumerate(blocks):
        def backward(d_o, inner=blk.attn.backward, i=i):
            grads[i] = inner(d_o)
            return grads[i]
        blk.attn.backward = backward
    st = LagaResidualStack(blocks, d_model, ckpt=True, device=DEV)
    st.forward(x, layers, cos, sin)
    kept = blocks[layer]._saved[0]
    assert isinstance(kept, laga.Checkpoint8)
    v = as_f64(kept.unpack(torch.float32).reshape(-1, d_model))
    _, out = st.backward(dx)
    laga._lib.sync_check()
    rows = v.shape[0]
    gain = as_f64(layers[layer]["gamma_pre"])[:, None]
    for name, t in (("dw_q", grads[layer][0]), ("dw_kva", grads[layer][1])):
        t = as_f64(t.reshape(rows, -1))
        got = as_f64(out[layer][name])
        bound = (rows + 64) * 2.0 ** -23 * gain * (np.abs(v).T @ np.abs(t))
        assert (np.abs(got - gain * (v.T @ t)) <= bound).all(), name
        assert (np.abs(got - v.T @ t) > bound).mean() > 0.9, name
