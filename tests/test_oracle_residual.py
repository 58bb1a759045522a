"""Pins of the fp64 oracle of the residual stream and the 8-bit checkpoints:
central finite differences, torch's norms and torch's e4m3 cast."""

import itertools

import numpy as np
import pytest
import torch

from oracle import residual as ores

EPS = 1e-5


def _case(rng, T, d, gate, gain):
    t = dict(x=rng.standard_normal((T, d)) * 2 + 0.3, y=rng.standard_normal((T, d)) - 0.2,
             alpha=np.array([0.7]), gamma_pre=1 + 0.1 * rng.standard_normal(d))
    if gain:
        t["gamma_post"] = 1 + 0.1 * rng.standard_normal(d)
    if gate != "none":
        t["gate"] = rng.standard_normal((T, d if gate == "full" else 1))
    return t


@pytest.mark.parametrize("norm_post,norm_pre,gate", list(itertools.product(
    ["layer", "rms", "none"], ["layer", "rms"], ["none", "token", "full"])))
def test_backward_matches_finite_differences(norm_post, norm_pre, gate):
    rng = np.random.default_rng(5)
    T, d = 3, 6
    t = _case(rng, T, d, gate, norm_post != "none")
    dx_out, dh = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def loss(a):
        r = ores.forward(**a, norm_post=norm_post, norm_pre=norm_pre, eps=EPS)
        return (r["x"] * dx_out).sum() + (r["h"] * dh).sum()

    r = ores.forward(**t, norm_post=norm_post, norm_pre=norm_pre, eps=EPS)
    kw = {k: t[k] for k in ("gate", "alpha", "gamma_post", "gamma_pre") if k in t}
    g = ores.backward(dx_out=dx_out, dh=dh, y_hat=r["y_hat"], x_hat=r["x_hat"],
                      stat_post=r["stat_post"], stat_pre=r["stat_pre"], norm_post=norm_post,
                      norm_pre=norm_pre, **kw)
    for name, v in t.items():
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            h = 1e-5
            up, dn = dict(t), dict(t)
            up[name] = v.copy()
            dn[name] = v.copy()
            up[name][i] += h
            dn[name][i] -= h
            num[i] = (loss(up) - loss(dn)) / (2 * h)
        got = np.asarray(g["d" + name]).reshape(v.shape)
        assert np.linalg.norm(got - num) <= 1e-7 * np.linalg.norm(num), name


def test_forward_matches_torch_norms():
    rng = np.random.default_rng(6)
    x, y = rng.standard_normal((5, 33)), rng.standard_normal((5, 33)) * 3 + 1
    g = 1 + 0.1 * rng.standard_normal(33)
    tx, ty, tg = (torch.from_numpy(v) for v in (x, y, g))
    r = ores.forward(x, y, alpha=0.5, gamma_post=g, gamma_pre=g, norm_post="layer",
                     norm_pre="rms", eps=EPS)
    xo = tx + 0.5 * torch.nn.functional.layer_norm(ty, (33,), weight=tg, eps=EPS)
    assert np.abs(r["x"] - xo.numpy()).max() < 1e-12
    h = torch.nn.functional.rms_norm(xo, (33,), weight=tg, eps=EPS)
    assert np.abs(r["h"] - h.numpy()).max() < 1e-12


def test_pack_matches_torch_cast_and_its_scale_rule():
    rng = np.random.default_rng(7)
    v = rng.standard_normal((9, 300)) * 2.0 ** rng.integers(-20, 20, (9, 1))
    v = v.astype(np.float32)
    buf = ores.pack(v.astype(np.float64))
    cols, pitch = ores.row_layout(300)
    assert buf.shape == (9, pitch) and (cols, pitch) == (384, 400)
    assert (buf[:, 300:384] == 0).all() and (buf[:, 387:] == 0).all()
    for g in range(3):
        w = v[:, 128 * g:128 * (g + 1)]
        e = buf[:, cols + g].astype(int) - 127
        top = np.abs(w).max(axis=1).astype(np.float64)
        assert (top <= 448 * 2.0 ** e).all() and (top > 448 * 2.0 ** (e - 1)).all()
        t = torch.from_numpy(w / (2.0 ** e[:, None]).astype(np.float32))
        codes = t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert (codes == buf[:, 128 * g:128 * g + w.shape[1]]).all()
    # each value is off by at most half a step: 2^-4 of itself, or half of the
    # smallest step (2^-9 of the unit)
    unit = np.repeat(2.0 ** (buf[:, cols:cols + 3].astype(float) - 127), 128, axis=1)[:, :300]
    off = np.abs(ores.unpack(buf, 300) - v)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * unit)).all()


def test_pack_borders():
    """The scale's borders, its clamps, zeros, and groups that are not finite."""
    d = 128
    rows = np.zeros((8, d))
    rows[0, 3] = 448.0
    rows[1, 3] = np.nextafter(448.0, 1e9)
    rows[2, 3] = 2.0 ** -140
    rows[3, 3] = 3.0e38
    rows[4, 3] = np.inf
    rows[5, 3] = np.nan
    rows[6, :4] = [448.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11]
    buf = ores.pack(rows)
    s = buf[:, 128].astype(int)
    assert list(s[:2] - 127) == [0, 1] and s[2] - 127 == ores.E_MIN and s[3] - 127 == ores.E_MAX
    assert s[4] == 255 and s[5] == 255 and s[7] - 127 == ores.E_MIN
    v = ores.unpack(buf, d)
    assert np.isnan(v[4:6]).all() and (v[7] == 0).all()
    assert v[3, 3] == 448 * 2.0 ** 119                  # saturates
    assert list(v[6, :4]) == [448.0, 0.0, 2.0 ** -8, 0.0]   # ties to even, below half a step


def test_every_code_round_trips_in_bf16():
    """Packing a code's own value gives it back, and value * 2^e is a bf16 number."""
    vals = ores.e4m3_values()
    fin = vals[np.isfinite(vals)]
    for e in (-117, -9, 0, 7, 119):
        v = np.zeros((1, 256))
        v[0, :len(fin)] = fin * 2.0 ** e
        assert (ores.unpack(ores.pack(v), 256) == v).all()
        assert (torch.from_numpy(v).to(torch.bfloat16).double().numpy() == v).all()


def test_weight_grad_is_the_product_of_the_values():
    rng = np.random.default_rng(8)
    v, dy, g = rng.standard_normal((17, 130)), rng.standard_normal((17, 5)), rng.standard_normal(130)
    buf = ores.pack(v)
    dw, _ = ores.weight_grad(buf, 130, dy, g)
    ref = sum(np.outer(ores.unpack(buf, 130)[t] * g, dy[t]) for t in range(17))
    assert np.abs(dw - ref).max() < 1e-12
