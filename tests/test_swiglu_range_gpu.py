"""The gated activation over the whole range of its inputs: gates up to the
largest finite number are open (sigma = 1), and infinities and NaN give what the
formula gives.

Tolerances as for its other tests: each factor is within 8 units of its last
place, 24 of them in all (2^-24 each) of the terms' magnitudes, and half a step of
the output's type."""

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
INF, NAN = float("inf"), float("nan")
TOP = 2.0 ** 128 * (1 - 2.0 ** -8)                 # the largest bf16 number


def _run(gu, da):
    import sequence_latent_norm_gb300 as laga
    ck = laga.swiglu8(gu.to(DEV))
    dgu = laga.swiglu8_grad(gu.to(DEV), da.to(DEV))
    laga._lib.sync_check()
    return ck.data.cpu().numpy(), as_f64(dgu)


def _check(gu, da, io):
    f = da.shape[1]
    data, dgu = _run(gu, da)
    g, u, d = as_f64(gu)[:, :f], as_f64(gu)[:, f:], as_f64(da)
    with np.errstate(invalid="ignore"):
        a, ref = oex.swiglu(as_f64(gu)), oex.swiglu_bwd(as_f64(gu), d)
    # no value here is near a border between two codes: a is u times a gate of
    # few bits, and sigma is one or zero
    assert np.array_equal(data, ores.pack(a))
    assert np.array_equal(np.isnan(dgu), np.isnan(ref))
    assert np.array_equal(np.isinf(dgu), np.isinf(ref))
    ok = np.isfinite(ref)
    with np.errstate(invalid="ignore"):
        mag = np.concatenate([np.abs(d * u), np.abs(d * g)], axis=1)
        lim = 24 * 2.0 ** -24 * mag + HALF[io] * np.abs(ref)
    assert (np.abs(dgu[ok] - ref[ok]) <= lim[ok]).all()


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("f", [256, 129])
def test_gates_up_to_the_largest_number(f, io):
    """From where the exponential is far below one (g = 120) on."""
    gates = [128.0, 1024.0, 2.0 ** 100, 2.0 ** 127, 1.375 * 2.0 ** 127, 1.4375 * 2.0 ** 127,
             1.5 * 2.0 ** 127, TOP]
    gu = torch.zeros(len(gates) + 2, 2 * f)
    for r, g in enumerate(gates):
        gu[r, :f], gu[r, f:] = g, 2.0 ** -100
        gu[r, 1:f:3] = -g                          # shut beside open
    gu[-2, :f], gu[-2, f:] = torch.tensor(gates).repeat(f)[:f], 2.0 ** -120
    gu[-1, 5], gu[-1, f + 5] = TOP, 2.0 ** -126    # one alone in its group
    da = torch.full((len(gu), f), 0.5)
    da[:, ::2] = -0.25
    _check(gu.to(DT[io]), da.to(DT[io]), io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_the_largest_fp32_number_and_what_is_not_a_number(io):
    """An infinite gate is the formula's: sigma is one, g (1 - sigma) has no value."""
    f = 256
    gu = torch.zeros(7, 2 * f)
    gu[:, f:] = 2.0 ** -100
    gu[0, 3], gu[1, 130], gu[2, 5] = INF, -INF, NAN
    gu[3, 7], gu[4, f + 200] = TOP, INF
    gu[5, 9], gu[5, f + 9] = INF, 0.0              # no value: inf * 0
    gu[6, :f] = torch.finfo(torch.float32).max if io == "fp32" else TOP
    _check(gu.to(DT[io]), torch.ones(7, f, dtype=DT[io]), io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_sigmoids_between_open_and_shut(io):
    """Gates of -110 .. 110, where the exponential leaves the normal numbers."""
    f = 1024
    gu = torch.cat([torch.linspace(-110, 110, f), torch.ones(f)])[None].to(DT[io])
    da = torch.ones(1, f, dtype=DT[io])
    data, dgu = _run(gu, da)
    g = as_f64(gu)[0, :f]
    ref = oex.swiglu_bwd(as_f64(gu), as_f64(da))[0]
    # below -87.3 the sigmoid is zero where it would be subnormal, 2^-126 at most
    mag = np.concatenate([1 + np.abs(g), np.abs(g)])
    lim = 24 * 2.0 ** -24 * mag + HALF[io] * np.abs(ref) + 2.0 ** -126 * mag
    assert (np.abs(dgu[0] - ref) <= lim).all()
