"""The residual-stream operators on the GPU against the fp64 oracle, and
their use together: forward, checkpoints, backward and weight gradient.

Tolerances.  u = 2^-24 (a rounding to fp32), U = half a step of the I/O type
(2^-8 bf16, 2^-24 fp32), relative to the value.
* A row statistic adds d terms: at most 96 additions of a chain (64 terms a
  thread, then a tree and 8 to 16 partial sums), so it is within 96 u of the
  mean magnitude of its terms; with the fewer than 32 further roundings of an
  element's own arithmetic every element is within ROW = 128 u of the size of
  the terms that make it.
* A column or whole sum of n terms adds (n + 64) u of the sum of their
  magnitudes, on top of ROW on each term.
* A stored output adds U of itself.
"""

import itertools

import numpy as np
import pytest
import torch

from laga_inputs import as_f64
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
U32 = 2.0 ** -24
ROW = 128 * U32
EPS = 1e-5
DEV = "cuda:0"


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _inputs(rows, d, dtype, gate, gain, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + rows * 31 + d)

    def rand(*s):
        return torch.randn(*s, generator=g)

    t = dict(x=(rand(rows, d) * 2 + 0.25).to(DT[dtype]), y=(rand(rows, d) - 0.5).to(DT[dtype]),
             dx_out=rand(rows, d).to(DT[dtype]), dh=rand(rows, d).to(DT[dtype]),
             alpha=torch.tensor([0.75]), gamma_pre=1 + 0.1 * rand(d))
    t["gamma_post"] = 1 + 0.1 * rand(d) if gain else None
    t["gate"] = None if gate == "none" else rand(rows, d if gate == "full" else 1).to(DT[dtype])
    return t


def _dev(t):
    return {k: None if v is None else v.to(DEV) for k, v in t.items()}


def _f64(t):
    return {k: None if v is None else as_f64(v) for k, v in t.items()}


def _close(got, ref, bound, what):
    got = as_f64(got).reshape(ref.shape)
    off = np.abs(got - ref)
    worst = float((off / np.maximum(bound, 1e-300)).max()) if off.size else 0.0
    assert np.isfinite(got).all() and (off <= bound).all(), f"{what}: {worst:.2f} of its bound"


def _size(v):
    """The size of the terms behind a row's elements: their magnitude and the
    row's largest."""
    a = np.abs(v)
    return a + (a.max(axis=1, keepdims=True) if a.size else 0)


def _check_stat(got, ref, v, what):
    """mean within ROW of the row's size; 1/std within ROW of itself (the
    squared terms are positive) and what the mean's error adds to them."""
    got = as_f64(got)
    top = np.abs(v).max(axis=1) if v.size else np.zeros(len(ref))
    assert (np.abs(got[:, 0] - ref[:, 0]) <= ROW * top).all(), what
    shift = ROW * top * ref[:, 1]
    assert (np.abs(got[:, 1] - ref[:, 1]) <= ref[:, 1] * (ROW + shift)).all(), what


def _check_hat8(ck, ref, top, d, what):
    """A checkpoint of normalised values: a scale that fits the group's
    maximum, and codes within half a step of the values."""
    buf = ck.data.cpu().numpy()
    cols, pitch = ores.row_layout(d)
    assert buf.shape[1] == pitch
    assert (buf[:, d:cols] == 0).all() and (buf[:, cols + cols // 128:] == 0).all(), what
    err = ROW * (np.abs(ref) + top)
    e = buf[:, cols:cols + cols // 128].astype(int) - 127
    for g in range(cols // 128):
        a, er = np.abs(ref[:, 128 * g:128 * g + 128]), err[:, 128 * g:128 * g + 128].max(axis=1)
        m, unit = a.max(axis=1), 2.0 ** e[:, g]
        assert (m - er <= 448 * unit).all(), what
        assert ((m + er > 448 * unit / 2) | (e[:, g] == ores.E_MIN)).all(), what
    unit = np.repeat(2.0 ** e, 128, axis=1)[:, :d]
    off = np.abs(ores.unpack(buf, d) - ref)
    assert (off <= np.maximum(2.0 ** -4 * (np.abs(ref) + err), 2.0 ** -10 * unit) + err).all(), what


def _plan(d, dtype="bf16", **kw):
    return _laga().ResidualNorm(d, io_dtype=dtype, eps=EPS, device=DEV, **kw)


def _forward(plan, dev):
    return plan.forward(dev["x"], dev["y"] if plan.post else None, gate=dev["gate"],
                        alpha=dev["alpha"], gamma_post=dev["gamma_post"],
                        gamma_pre=dev["gamma_pre"])


def _check(rows, d, dtype, post, pre, norm_post, norm_pre, gate, ckpt, seed=0):
    laga = _laga()
    what = f"{rows}x{d} {dtype} post={post} pre={pre} {norm_post}/{norm_pre} {gate} ckpt={ckpt}"
    gain = post and norm_post != "none"
    gate = gate if post else "none"
    t = _inputs(rows, d, dtype, gate, gain, seed)
    dev, a = _dev(t), _f64(t)
    plan = _plan(d, dtype, post=post, pre=pre, norm_post=norm_post, norm_pre=norm_pre, gate=gate,
                 ckpt=ckpt)
    r = _forward(plan, dev)
    laga._lib.sync_check()
    ref = ores.forward(a["x"], a["y"] if post else None, gate=a["gate"], alpha=a["alpha"],
                       gamma_post=a["gamma_post"], gamma_pre=a["gamma_pre"] if pre else None,
                       norm_post=norm_post, norm_pre=norm_pre, eps=EPS)
    H = HALF[dtype]
    if post:
        st = ref["stat_post"]
        _check_stat(r.saved.stat_post, st, a["y"], what + " stat_post")
        # an element of y^ is off by what y - mean and 1/std are
        top_y = _size(a["y"]) * st[:, 1:] if norm_post != "none" else np.abs(a["y"])
        size = np.abs(a["x"]) + 2 * top_y
        _close(r.x, ref["x"], H * np.abs(ref["x"]) + ROW * size, what + " x")
    else:
        assert r.x is dev["x"]
        size = np.abs(a["x"])
    if pre:
        st = ref["stat_pre"]
        _check_stat(r.saved.stat_pre, st, 3 * (size + size.max(axis=1, keepdims=True, initial=0)),
                    what + " stat_pre")
        top_x = 3 * _size(size) * st[:, 1:]
        _close(r.h, ref["h"], H * np.abs(ref["h"]) + 2 * ROW * top_x, what + " h")
    if ckpt:
        if post:
            _check_hat8(r.saved.y, ref["y_hat"], top_y, d, what + " y8")
        if pre:
            _check_hat8(r.saved.x, ref["x_hat"], top_x, d, what + " x8")

    # backward: the oracle starts from what the forward kept
    g = plan.backward(r.saved, dev["dx_out"], dev["dh"] if pre else None)
    laga._lib.sync_check()

    def kept(k, stat):
        if ckpt:
            return ores.unpack(k.data.cpu().numpy(), d)
        return ores.hat(as_f64(k).reshape(rows, d), as_f64(stat))

    y_hat = kept(r.saved.y, r.saved.stat_post) if post else None
    x_hat = kept(r.saved.x, r.saved.stat_pre) if pre else None
    s_post = as_f64(r.saved.stat_post) if post else None
    s_pre = as_f64(r.saved.stat_pre) if pre else None
    want = ores.backward(dx_out=a["dx_out"], dh=a["dh"] if pre else None, y_hat=y_hat, x_hat=x_hat,
                         stat_post=s_post, stat_pre=s_pre, gate=a["gate"], alpha=a["alpha"],
                         gamma_post=a["gamma_post"], gamma_pre=a["gamma_pre"], norm_post=norm_post,
                         norm_pre=norm_pre)
    size_D = np.abs(a["dx_out"])
    n_terms = (rows + 64) * U32
    if pre:
        big = np.abs(x_hat) + 1
        size_D = size_D + 3 * s_pre[:, 1:] * _size(a["dh"]) * _size(big)
        _close(g.dx, want["dx"], H * np.abs(want["dx"]) + ROW * size_D, what + " dx")
        _close(g.dgamma_pre, want["dgamma_pre"], (ROW + n_terms) * want["dgamma_pre_abs"] + 1e-30,
               what + " dgamma_pre")
    else:
        assert g.dx is dev["dx_out"]
    if post:
        big = np.abs(y_hat) + 1
        _close(g.dy, want["dy"], H * np.abs(want["dy"])
               + 6 * ROW * (s_post[:, 1:] * _size(size_D) * _size(big)), what + " dy")
        col = size_D * np.abs(y_hat) * 2
        if gain:
            _close(g.dgamma_post, want["dgamma_post"],
                   (ROW + n_terms) * col.sum(axis=0) + 1e-30, what + " dgamma_post")
        _close(g.dalpha, want["dalpha"], np.array([(2 * ROW + n_terms) * col.sum() + 1e-30]),
               what + " dalpha")
        if gate != "none":
            da = col.sum(axis=1, keepdims=True) if gate == "token" else col
            _close(g.dgate, want["dgate"], H * np.abs(want["dgate"]) + 2 * ROW * da, what + " dgate")


PARTS = [(True, True), (True, False), (False, True)]
SIZES = [(1, 1), (3, 7), (2, 8), (5, 127), (4, 129), (37, 256), (1, 1000), (333, 1001), (70, 1024),
         (19, 1032), (9, 2048), (155, 2056), (7, 4096), (5, 4104), (2, 7168), (3, 8192), (2, 8200),
         (2, 16384), (1, 16383)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sizes(rows, d, dtype):
    _check(rows, d, dtype, True, True, "layer", "rms", "full", True)
    _check(rows, d, dtype, True, True, "rms", "layer", "token", False)


@pytest.mark.parametrize("post,pre", PARTS)
@pytest.mark.parametrize("norm_post,norm_pre", list(itertools.product(["layer", "rms", "none"],
                                                                      ["layer", "rms"])))
@pytest.mark.parametrize("gate", ["none", "token", "full"])
@pytest.mark.parametrize("d", [200, 203])
def test_every_option(post, pre, norm_post, norm_pre, gate, d):
    for ckpt, dtype in itertools.product([False, True], ["bf16", "fp32"]):
        _check(21, d, dtype, post, pre, norm_post, norm_pre, gate, ckpt, seed=3)


@pytest.mark.parametrize("rows,d", [(5000, 512), (700, 7168), (3000, 333)])
def test_many_rows(rows, d):
    """More rows than a launch has places, so that every place walks several."""
    _check(rows, d, "bf16", True, True, "rms", "layer", "full", True)


@pytest.mark.parametrize("rows,d,ckpt", [(400, 7168, False), (320, 16384, False), (320, 16384, True),
                                         (1500, 4096, False), (2600, 1024, False)])
def test_many_rows_of_fp32(rows, d, ckpt):
    """fp32 rows: rings of one and two rows, and teams with several rows each."""
    _check(rows, d, "fp32", True, True, "layer", "rms", "full", ckpt)
    _check(rows, d, "fp32", False, True, "none", "layer", "none", ckpt)


@pytest.mark.parametrize("d", [512, 333])
def test_no_rows(d):
    """Zero tokens: empty tensors come back, and the sums over them are zero."""
    plan = _plan(d, gate="token", ckpt=True)
    dev = _dev(_inputs(0, d, "bf16", "token", True))
    r = _forward(plan, dev)
    g = plan.backward(r.saved, dev["dx_out"], dev["dh"])
    _laga()._lib.sync_check()
    assert r.x.shape == (0, d) and r.h.shape == (0, d) and g.dy.shape == (0, d)
    for s in (g.dalpha, g.dgamma_post, g.dgamma_pre):
        assert (s == 0).all()


def test_no_other_use_of_the_stream():
    """dx_out=None is a gradient of zeros."""
    for d in (512, 333):
        plan = _plan(d, gate="full")
        dev = _dev(_inputs(40, d, "bf16", "full", True))
        r = _forward(plan, dev)
        a = plan.backward(r.saved, None, dev["dh"])
        b = plan.backward(r.saved, torch.zeros_like(dev["dx_out"]), dev["dh"])
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_leading_dimensions_and_repeatability():
    plan = _plan(640, gate="token", ckpt=True)
    dev = _dev(_inputs(60, 640, "bf16", "token", True))
    r = _forward(plan, dev)
    g = plan.backward(r.saved, dev["dx_out"], dev["dh"])
    cut = {k: v.reshape(3, 20, -1) if k in ("x", "y", "gate", "dx_out", "dh") else v
           for k, v in dev.items()}
    r3 = _forward(plan, cut)
    g3 = plan.backward(r3.saved, cut["dx_out"], cut["dh"])
    assert r3.h.shape == (3, 20, 640) and g3.dgate.shape == (3, 20, 1)
    assert torch.equal(r.h, r3.h.reshape(60, 640)) and torch.equal(r.x, r3.x.reshape(60, 640))
    assert torch.equal(r.saved.x.data, r3.saved.x.data)
    for p, q in zip(g, g3):
        assert torch.equal(p.flatten(), q.flatten())


@pytest.mark.parametrize("d", [512, 333])
def test_non_finite_rows_stay_in_their_rows(d):
    """A NaN or an infinity in one token's y: its row, its groups and the sums
    over all rows are NaN; every other row is as without it."""
    t = _inputs(12, d, "bf16", "full", True)
    clean = _dev(t)
    t["y"][3, 5], t["y"][7, 200] = float("nan"), float("inf")
    dirty = _dev(t)
    plan = _plan(d, gate="full", ckpt=True)
    a, b = _forward(plan, clean), _forward(plan, dirty)
    keep = [i for i in range(12) if i not in (3, 7)]
    for p, q in ((a.x, b.x), (a.h, b.h), (a.saved.x.data, b.saved.x.data),
                 (a.saved.y.data, b.saved.y.data)):
        assert torch.equal(p[keep], q[keep])
    assert b.h[[3, 7]].isnan().all()
    assert b.saved.x.unpack()[[3, 7]].isnan().all()
    ga = plan.backward(a.saved, clean["dx_out"], clean["dh"])
    gb = plan.backward(b.saved, clean["dx_out"], clean["dh"])
    for p, q in ((ga.dx, gb.dx), (ga.dy, gb.dy), (ga.dgate, gb.dgate)):
        assert torch.equal(p[keep], q[keep])
        assert q[[3, 7]].isnan().all()
    assert gb.dgamma_pre.isnan().all() and gb.dalpha.isnan().all()


def test_backward_against_differences_of_the_forward():
    """<grad, direction> against central differences of the fp32 forward along
    random directions.  With a step of 2^-7 the third-order term of a loss of
    unit-scale pieces is below 1e-3 of the derivative, and the fp32 rounding of
    the loss (summed in fp64) far below that; the bound is 1e-2."""
    rows, d, h = 16, 192, 2.0 ** -7
    for norm_post, norm_pre, gate in (("layer", "rms", "full"), ("none", "layer", "token")):
        t = _inputs(rows, d, "fp32", gate, norm_post != "none", seed=9)
        dev = _dev(t)
        plan = _plan(d, "fp32", norm_post=norm_post, norm_pre=norm_pre, gate=gate)

        def loss(v):
            r = _forward(plan, v)
            return float((r.x.double() * dev["dx_out"].double()).sum()
                         + (r.h.double() * dev["dh"].double()).sum())

        r = _forward(plan, dev)
        g = plan.backward(r.saved, dev["dx_out"], dev["dh"])
        gen = torch.Generator().manual_seed(4)
        for name in ("x", "y", "gate", "alpha", "gamma_post", "gamma_pre"):
            if dev[name] is None:
                continue
            grad = getattr(g, "d" + name)
            # along the gradient's own signs the derivative is large
            u = grad.sign().cpu() * torch.rand(grad.shape, generator=gen)
            u = u.to(DEV)
            num = (loss({**dev, name: dev[name] + h * u}) - loss({**dev, name: dev[name] - h * u}))
            num /= 2 * h
            got = float((grad.double() * u.double()).sum())
            assert abs(num - got) <= 1e-2 * abs(got), (name, num, got)


def test_refusals_on_the_gpu():
    laga = _laga()
    plan = _plan(64, gate="full")
    dev = _dev(_inputs(6, 64, "bf16", "full", True))
    kw = dict(gate=dev["gate"], alpha=dev["alpha"], gamma_post=dev["gamma_post"],
              gamma_pre=dev["gamma_pre"])
    wide = torch.zeros(6, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        plan.forward(wide[:, ::2], dev["y"], **kw)
    with pytest.raises(ValueError, match="shape"):
        plan.forward(dev["x"], dev["y"][:5], **kw)
    with pytest.raises(ValueError, match="dtype"):
        plan.forward(dev["x"], dev["y"], **{**kw, "alpha": dev["alpha"].double()})
    with pytest.raises(TypeError):
        plan.forward(dev["x"], dev["y"], **{**kw, "gate": None})
    flat = torch.zeros(6 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(laga.LagaError) as e:            # 2 bytes off a 16-byte boundary
        plan.forward(flat[1:6 * 64 + 1].view(6, 64), dev["y"], **kw)
    assert e.value.status == laga._lib.LAGA_ERR_ALIGN
    r = plan.forward(dev["x"], dev["y"], **kw)
    with pytest.raises(ValueError, match="shape"):
        plan.backward(r.saved, dev["dx_out"], dev["dh"][:5].contiguous())
    with pytest.raises(TypeError):
        _plan(64, gate="full", ckpt=True).backward(r.saved, dev["dx_out"], dev["dh"])
    eight = _forward(_plan(64, gate="full", ckpt=True), dev)
    with pytest.raises(TypeError):
        plan.backward(eight.saved, dev["dx_out"], dev["dh"])
