"""fp64 oracle of the residual stream around a block and of the 8-bit
activation checkpoints: plain NumPy, written from the definitions.

    x' = x + alpha * sigmoid(gate) * N_post(y) * gamma_post
    h  = N_pre(x') * gamma_pre

Rows are tokens; N is LayerNorm (biased variance), the RMS norm or, for
N_post, the identity ("none").  The 8-bit form keeps e4m3 codes with one
power of two 2^e per 128 channels, the smallest with max|v| <= 448 2^e.
"""

from __future__ import annotations

import numpy as np

GROUP = 128
E_MIN, E_MAX = -117, 119


# ------------------------------------------------------------ norms
def stat(v, norm, eps):
    """[rows, 2]: mean and 1/std of each row."""
    v = np.asarray(v, np.float64)
    if norm == "none":
        return np.stack([np.zeros(len(v)), np.ones(len(v))], axis=1)
    mean = v.mean(axis=1) if norm == "layer" else np.zeros(len(v))
    var = ((v - mean[:, None]) ** 2).mean(axis=1)
    return np.stack([mean, 1.0 / np.sqrt(var + eps)], axis=1)


def hat(v, st):
    return (v - st[:, :1]) * st[:, 1:]


def norm_bwd(f, h, rstd, norm):
    """Gradient of the row before the norm; f = that of the normalised row h."""
    if norm == "none":
        return f
    out = f - h * (f * h).mean(axis=1, keepdims=True)
    if norm == "layer":
        out = out - f.mean(axis=1, keepdims=True)
    return out * rstd[:, None]


def sigmoid(a):
    return 1.0 / (1.0 + np.exp(-a))


def forward(x, y=None, *, gate=None, alpha=None, gamma_post=None, gamma_pre=None,
            norm_post="rms", norm_pre="rms", eps=1e-5):
    """post if y is given, pre if gamma_pre is.  Returns a dict of x, h,
    stat_post, stat_pre, y_hat, x_hat (what applies)."""
    out = {}
    if y is not None:
        out["stat_post"] = stat(y, norm_post, eps)
        out["y_hat"] = hat(y, out["stat_post"])
        z = out["y_hat"] * (1.0 if gamma_post is None else gamma_post)
        s = 1.0 if gate is None else sigmoid(gate)
        x = x + np.asarray(alpha).item() * s * z
    out["x"] = x
    if gamma_pre is not None:
        out["stat_pre"] = stat(x, norm_pre, eps)
        out["x_hat"] = hat(x, out["stat_pre"])
        out["h"] = out["x_hat"] * gamma_pre
    return out


def backward(*, dx_out=None, dh=None, y_hat=None, x_hat=None, stat_post=None, stat_pre=None,
             gate=None, alpha=None, gamma_post=None, gamma_pre=None, norm_post="rms",
             norm_pre="rms"):
    """Gradients for the given normalised rows; a column sum's entry
    ``<name>_abs`` is the sum of its terms' magnitudes."""
    out = {}
    D = 0.0 if dx_out is None else dx_out
    if dh is not None:
        out["dgamma_pre"] = (dh * x_hat).sum(axis=0)
        out["dgamma_pre_abs"] = np.abs(dh * x_hat).sum(axis=0)
        D = D + norm_bwd(dh * gamma_pre, x_hat, stat_pre[:, 1], norm_pre)
    out["dx"] = D
    if y_hat is not None:
        a = np.asarray(alpha).item()
        g = 1.0 if gamma_post is None else gamma_post
        s = 1.0 if gate is None else sigmoid(gate)
        z = y_hat * g
        dz = a * D * s
        if gate is not None:
            da = a * D * z * s * (1.0 - s)
            token = gate.shape[1] == 1 and y_hat.shape[1] != 1
            out["dgate"] = da.sum(axis=1, keepdims=True) if token else da
            out["dgate_abs"] = np.abs(da).sum(axis=1, keepdims=True) if token else np.abs(da)
        out["dalpha"] = np.array([(D * s * z).sum()])
        out["dalpha_abs"] = np.array([np.abs(D * s * z).sum()])
        if gamma_post is not None:
            out["dgamma_post"] = (dz * y_hat).sum(axis=0)
            out["dgamma_post_abs"] = np.abs(dz * y_hat).sum(axis=0)
        out["dy"] = norm_bwd(dz * g, y_hat, stat_post[:, 1], norm_post)
    return out


# ------------------------------------------------------------ 8 bits
def row_layout(d):
    """(code bytes, row bytes) of a checkpoint of d channels."""
    cols = -(-d // GROUP) * GROUP
    return cols, cols + -(-(cols // GROUP) // 16) * 16


def e4m3_values():
    """The 256 e4m3 codes' values (NaN for 0x7f and 0xff)."""
    b = np.arange(256)
    expo, frac = (b >> 3) & 15, b & 7
    v = np.where(expo > 0, (1 + frac / 8.0) * 2.0 ** (expo - 7.0), frac / 8.0 * 2.0 ** -6)
    v = np.where((b & 0x7f) == 0x7f, np.nan, v)
    return np.where(b >= 128, -v, v)


def group_exponents(v):
    """Exponent e of each group of fp64 rows [rows, d], and which are NaN."""
    rows, d = v.shape
    cols, _ = row_layout(d)
    g = np.zeros((rows, cols))
    g[:, :d] = v
    g = g.reshape(rows, -1, GROUP)
    bad = ~np.isfinite(g).all(axis=2)
    m, k = np.frexp(np.where(bad[:, :, None], 0.0, np.abs(g)).max(axis=2))
    e = np.where(m <= 448.0 / 512.0, k - 9, k - 8)     # m 2^k <= 448 2^e
    e = np.where(m == 0, E_MIN, np.clip(e, E_MIN, E_MAX))
    return e, bad, g


def pack(v):
    """The checkpoint rows (uint8 [rows, row bytes]) of fp64 rows."""
    rows, d = v.shape
    cols, pitch = row_layout(d)
    e, bad, g = group_exponents(v)
    t = np.where(bad[:, :, None], 0.0, g) / 2.0 ** e[:, :, None]
    t = np.clip(t, -448.0, 448.0).reshape(rows, cols)
    a = np.abs(t)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -7))), -6.0) - 3.0)
    a = np.rint(a / step) * step                       # ties to even
    table = e4m3_values()[:0x7f]
    code = np.searchsorted(table, a)
    assert (table[code] == a).all()
    out = np.zeros((rows, pitch), np.uint8)
    out[:, :cols] = code + np.where(np.signbit(t), 128, 0)
    out[:, cols:cols + e.shape[1]] = np.where(bad, 255, e + 127)
    return out


def unpack(buf, d):
    """fp64 values of checkpoint rows."""
    cols, _ = row_layout(d)
    s = buf[:, cols:cols + cols // GROUP].astype(np.float64)
    unit = np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return (e4m3_values()[buf[:, :cols]] * np.repeat(unit, GROUP, axis=1))[:, :d]


def weight_grad(buf, d, dy, gamma=None):
    """diag(gamma) v^T dy, and the sum of the terms' magnitudes."""
    v = unpack(buf, d)
    if gamma is not None:
        v = v * gamma
    return v.T @ dy, np.abs(v).T @ np.abs(dy)
