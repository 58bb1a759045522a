"""The residual operators, the 8-bit checkpoints and the attention block
together, as a user runs them: LagaResidualStack against the fp64 oracles, the
block with an 8-bit checkpoint, a captured and replayed step, other streams,
and guard bands around every buffer.

Tolerances of the stack: every block may add BLOCK_REL_FRO = 1e-2 to what
passes through it (its own test's bound), forward and backward, so a gradient
of a stack of n blocks is held to 2 n 1e-2.  An e4m3 value is off by up to half
a step, uniformly: 2^-3 / sqrt(12) = 0.036 of its binade's base in the root
mean square, which bounds what 8-bit checkpoints add to a gradient that is a
sum of products with them."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from laga_inputs import as_f64, config, make_block_inputs
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCK_REL_FRO = 1e-2
E4M3_RMS = 2.0 ** -3 / np.sqrt(12.0)


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _rel(a, b):
    return float(np.linalg.norm(as_f64(a) - b) / max(np.linalg.norm(b), 1e-30))


def _stack_case(n, d_model, norm_post, gate):
    """Inputs of n layers (CPU): x, dx, the RoPE tables and the layers' dicts."""
    layers = []
    for i in range(n):
        wl = config(1, S=192, H=2, n_h_total=2, seed=40 + i)
        b = make_block_inputs(wl, d_model)
        g = torch.Generator().manual_seed(90 + i)
        w = {k: b[k] for k in ("w_q", "w_kva", "gamma", "w_kvb", "w_o")}
        w["gamma_pre"] = 1 + 0.1 * torch.randn(d_model, generator=g)
        w["alpha"] = torch.tensor([0.6 + 0.2 * i])
        if norm_post != "none":
            w["gamma_post"] = 1 + 0.1 * torch.randn(d_model, generator=g)
        if gate != "none":
            w["gate"] = torch.randn(1, wl.S, d_model if gate == "full" else 1,
                                    generator=g).to(torch.bfloat16)
        layers.append(w)
        if i == 0:
            x, dx, cos, sin = b["h"], b["dy"], b["cos"], b["sin"]
    return wl, x, dx, cos, sin, layers


def _stack(wl, n, d_model, ckpt, **kw):
    from sequence_latent_norm_gb300.block import LagaAttentionBlock, LagaResidualStack
    blocks = [LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV)) for _ in range(n)]
    return LagaResidualStack(blocks, d_model, ckpt=ckpt, device=DEV, **kw)


def _oracle_stack(x, dx, cos, sin, layers, wl, norm_post, norm_pre):
    from oracle import Dims
    from oracle.block import block_backward, block_forward
    dims = Dims(S=wl.S, H=wl.H)
    shape = x.shape
    flat = x.reshape(-1, shape[-1])
    saved = []
    for w in layers:
        pre = ores.forward(flat, gamma_pre=w["gamma_pre"], norm_pre=norm_pre)
        y, st = block_forward(pre["h"].reshape(shape), w["w_q"], w["w_kva"], w["gamma"], w["w_kvb"],
                              w["w_o"], cos, sin, dims)
        y = y.reshape(flat.shape)
        kw = dict(gate=w["gate"].reshape(len(flat), -1) if "gate" in w else None, alpha=w["alpha"],
                  gamma_post=w.get("gamma_post"))
        post = ores.forward(flat, y, norm_post=norm_post, **kw)
        saved.append((pre, st, post, kw))
        flat = post["x"]
    out = flat
    g = dx.reshape(flat.shape)
    grads = []
    for w, (pre, st, post, kw) in zip(reversed(layers), reversed(saved)):
        gp = ores.backward(dx_out=g, y_hat=post["y_hat"], stat_post=post["stat_post"],
                           norm_post=norm_post, **kw)
        gb = block_backward(st, gp["dy"].reshape(shape))
        gq = ores.backward(dx_out=g, dh=gb["dh"].reshape(flat.shape), x_hat=pre["x_hat"],
                           stat_pre=pre["stat_pre"], gamma_pre=w["gamma_pre"], norm_pre=norm_pre)
        g = gq["dx"]
        grads.append({**{k: v for k, v in gb.items() if k != "dh"}, "dgamma_pre": gq["dgamma_pre"],
                      **{k: gp[k] for k in ("dalpha", "dgamma_post", "dgate") if k in gp},
                      "dalpha_abs": gp["dalpha_abs"]})
    return out.reshape(shape), g.reshape(shape), grads[::-1]


@pytest.mark.parametrize("norm_post,norm_pre,gate", [("none", "rms", "none"),
                                                     ("rms", "layer", "full"),
                                                     ("layer", "rms", "token")])
def test_stack_matches_the_oracles(norm_post, norm_pre, gate):
    n, d_model = 2, 256
    wl, x, dx, cos, sin, layers = _stack_case(n, d_model, norm_post, gate)
    dev = [{k: v.to(DEV) for k, v in w.items()} for w in layers]
    f64 = [{k: as_f64(v) for k, v in w.items()} for w in layers]
    out, g0, grads = _oracle_stack(as_f64(x), as_f64(dx), as_f64(cos), as_f64(sin), f64, wl,
                                   norm_post, norm_pre)
    got = {}
    for ckpt in (False, True):
        st = _stack(wl, n, d_model, ckpt, norm_post=norm_post, norm_pre=norm_pre, gate=gate)
        y = st.forward(x.to(DEV), dev, cos.to(DEV), sin.to(DEV))
        gx, gl = st.backward(dx.to(DEV))
        _laga()._lib.sync_check()
        got[ckpt] = (y, gx, gl)
        tol = 2 * n * BLOCK_REL_FRO
        assert _rel(y, out) <= n * BLOCK_REL_FRO
        extra = 2 * n * E4M3_RMS if ckpt else 0.0
        assert _rel(gx, g0) <= tol + extra, ("dx", _rel(gx, g0))
        for i in range(n):
            for k, v in gl[i].items():
                ref = grads[i][k].reshape(v.shape)
                if k == "dalpha":   # one cancelling sum: against the size of its terms
                    off = abs(float(v) - ref.item()) / grads[i]["dalpha_abs"].item()
                else:
                    off = _rel(v, ref)
                assert off <= tol + extra, (ckpt, i, k, off)
    assert torch.equal(got[False][0], got[True][0])     # the forward is the same
    # and between the layers both halves in one kernel give what two give
    st = _stack(wl, n, d_model, True, norm_post=norm_post, norm_pre=norm_pre, gate=gate)
    y = st.forward(x.to(DEV), dev, cos.to(DEV), sin.to(DEV))
    assert torch.equal(y, got[True][0])


def test_stack_of_one_block_and_refusals():
    from sequence_latent_norm_gb300.block import LagaAttentionBlock, LagaResidualStack
    wl, x, dx, cos, sin, layers = _stack_case(1, 200, "none", "none")
    dev = [{k: v.to(DEV) for k, v in w.items()} for w in layers]
    st = _stack(wl, 1, 200, True)
    y = st.forward(x.to(DEV), dev, cos.to(DEV), sin.to(DEV))
    gx, gl = st.backward(dx.to(DEV))
    _laga()._lib.sync_check()
    assert y.shape == x.shape and gx.shape == x.shape and set(gl[0]) == {
        "dalpha", "dw_q", "dw_kva", "dw_o", "dw_kvb", "dgamma", "dgamma_pre"}
    with pytest.raises(ValueError):
        st.forward(x.to(DEV), dev + dev, cos.to(DEV), sin.to(DEV))
    with pytest.raises(ValueError):
        LagaResidualStack([], 200, device=DEV)
    with pytest.raises(ValueError):
        LagaAttentionBlock.single(2, 64, device=torch.device(DEV), checkpoint="int8")


def test_block_with_an_8_bit_checkpoint():
    """Everything but dW_q and dW_kv_a is as without the checkpoint; these two
    are the gradients of the 8-bit h, and hold no copy of h."""
    laga = _laga()
    from sequence_latent_norm_gb300.block import LagaAttentionBlock
    wl = config(1, S=384, H=2, n_h_total=2)
    t = {k: v.to(DEV) for k, v in make_block_inputs(wl, 256).items()}
    args = (t["w_q"], t["w_kva"], t["gamma"], t["w_kvb"], t["w_o"], t["cos"], t["sin"])
    runs = {}
    for ck in ("none", "fp8"):
        b = LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV), checkpoint=ck)
        y = b.forward(t["h"], *args)
        held = b._saved[0]
        runs[ck] = (y, b.backward(t["dy"]), held)
    laga._lib.sync_check()
    assert isinstance(runs["fp8"][2], laga.Checkpoint8)
    assert torch.equal(runs["none"][0], runs["fp8"][0])
    # an h with strides of its own is packed as what it holds
    wide = torch.zeros(*t["h"].shape[:-1], 2 * t["h"].shape[-1], dtype=t["h"].dtype, device=DEV)
    wide[..., ::2] = t["h"]
    b = LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV), checkpoint="fp8")
    b.forward(wide[..., ::2], *args)
    assert torch.equal(b._saved[0].data, runs["fp8"][2].data)
    for k, v in runs["none"][1].items():
        w = runs["fp8"][1][k]
        if k in ("dw_q", "dw_kva"):
            off = _rel(w, as_f64(v))
            assert 0 < off <= E4M3_RMS + BLOCK_REL_FRO, (k, off)
        else:
            assert torch.equal(v, w), k


def _step(plan, op, t):
    r = plan.forward(t["x"], t["y"], gate=t["gate"], alpha=t["alpha"], gamma_post=t["gamma_post"],
                     gamma_pre=t["gamma_pre"])
    g = plan.backward(r.saved, t["dx"], t["dh"])
    dw = op.weight_grad8(r.saved.x, t["dq"], gamma=t["gamma_pre"])
    x8 = op.pack8(t["x"]).unpack()
    return [r.x, r.h, *g, dw, x8]


def _step_inputs(rows, d, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)

    return dict(x=rand(rows, d), y=rand(rows, d), gate=rand(rows, d), dx=rand(rows, d),
                dh=rand(rows, d), dq=rand(rows, n), alpha=torch.rand(1, generator=g, device=DEV),
                gamma_post=rand(d).float(), gamma_pre=rand(d).float())


@pytest.mark.parametrize("rows,d,n", [(300, 640, 200), (70, 333, 51)])
def test_captured_step_replays_on_new_inputs(rows, d, n):
    """Two captured graphs of the same step, replayed on other values, give
    what eager calls give."""
    laga = _laga()
    plan = laga.ResidualNorm(d, gate="full", ckpt=True, device=DEV)
    t = _step_inputs(rows, d, n, 1)
    _step(plan, laga, t)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = _step(plan, laga, t)
        graphs.append((g, outs))
    for k, v in _step_inputs(rows, d, n, 2).items():
        t[k].copy_(v)
    want = _step(plan, laga, t)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    laga._lib.sync_check()
    for _, outs in graphs:
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_first_call_inside_a_capture():
    """A fresh process whose first call of each operator is captured."""
    code = """
import torch, sys
sys.path.insert(0, "tests")
from test_residual_stack_gpu import _step, _step_inputs
import sequence_latent_norm_gb300 as laga
t = _step_inputs(64, 512, 64, 3)
plan = laga.ResidualNorm(512, gate="full", ckpt=True, device="cuda:0")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = _step(plan, laga, t)
g.replay()
torch.cuda.synchronize()
want = _step(plan, laga, t)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, want))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_another_stream():
    """Calls on a stream of the caller's, beside work on the current one."""
    laga = _laga()
    plan = laga.ResidualNorm(640, gate="full", ckpt=True, device=DEV)
    t = _step_inputs(500, 640, 136, 5)
    want = _step(plan, laga, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    r = plan.forward(t["x"], t["y"], gate=t["gate"], alpha=t["alpha"],
                     gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], stream=s)
    busy = torch.randn(2048, 2048, device=DEV)
    for _ in range(5):
        busy = busy @ busy * 1e-3
    g = plan.backward(r.saved, t["dx"], t["dh"], stream=s)
    dw = laga.weight_grad8(r.saved.x, t["dq"], gamma=t["gamma_pre"], stream=s)
    x8 = laga.pack8(t["x"], stream=s).unpack(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip([r.x, r.h, *g, dw, x8], want):
        assert torch.equal(a, b)
    laga._lib.sync_check()


def test_weight_grad_many_times_over_ragged_sizes():
    """The pair's two CTAs hand tiles to one another; a hand-over that came
    too early would show as a value that is not the same every time."""
    laga = _laga()
    for rows, d, n, dt in ((129, 512, 257, torch.float32), (200, 640, 576, torch.float32),
                           (1000, 1408, 200, torch.bfloat16), (3000, 2048, 520, torch.bfloat16)):
        g = torch.Generator(device=DEV).manual_seed(rows)
        ck = laga.pack8(torch.randn(rows, d, generator=g, device=DEV))
        dy = torch.randn(rows, n, generator=g, device=DEV).to(dt)
        ref = ck.unpack(torch.float32).double().t() @ dy.double()
        size = ck.unpack(torch.float32).double().abs().t() @ dy.double().abs()
        first = laga.weight_grad8(ck, dy)
        assert ((first.double() - ref).abs() <= (rows + 64) * 2.0 ** -23 * size).all()
        junk = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        for i in range(60):
            if i % 4 == 0:
                junk.fill_(i)
            assert torch.equal(first, laga.weight_grad8(ck, dy)), (rows, d, n, i)
    laga._lib.sync_check()


def test_more_than_two_to_the_31_elements():
    """Rows behind the 2^31st element are as in a call of their own."""
    laga = _laga()
    rows, d, last = 301000, 7168, 160
    g = torch.Generator(device=DEV).manual_seed(8)
    tail = torch.randn(last, d, generator=g, device=DEV).to(torch.bfloat16)
    x = torch.ones(rows, d, dtype=torch.bfloat16, device=DEV)
    x[-last:] = tail
    gamma = torch.rand(d, generator=g, device=DEV)
    plan = laga.ResidualNorm(d, post=False, norm_pre="layer", ckpt=True, device=DEV)
    big, small = plan.forward(x, gamma_pre=gamma), plan.forward(tail, gamma_pre=gamma)
    assert torch.equal(big.h[-last:], small.h)
    assert torch.equal(big.saved.x.data[-last:], small.saved.x.data)
    gb, gs = plan.backward(big.saved, None, x), plan.backward(small.saved, None, tail)
    assert torch.equal(gb.dx[-last:], gs.dx)
    del gb, big
    ck = laga.pack8(x)
    assert torch.equal(ck.data[-last:], laga.pack8(tail).data)
    assert torch.equal(ck.unpack()[-last:], laga.pack8(tail).unpack())
    del x
    dy = torch.zeros(rows, 16, dtype=torch.bfloat16, device=DEV)
    dy[-last:] = tail[:, :16]
    v = laga.pack8(tail).unpack(torch.float32).double()
    ref, size = v.t() @ tail[:, :16].double(), v.abs().t() @ tail[:, :16].double().abs()
    got = laga.weight_grad8(ck, dy)
    assert ((got.double() - ref).abs() <= (last + 64) * 2.0 ** -23 * size).all()
    laga._lib.sync_check()


BAND, FILL = 4096, 0xA5


class _Banded:
    """A device buffer of nbytes between two bands of a fixed pattern."""

    def __init__(self, nbytes, fill=FILL):
        self.n = nbytes
        self.all = torch.full((2 * BAND + (nbytes + 255) // 256 * 256,), FILL, dtype=torch.uint8,
                              device=DEV)

    @property
    def ptr(self):
        return self.all.data_ptr() + BAND

    def view(self, dtype, shape):
        return self.all[BAND:BAND + self.n].view(dtype).view(shape)

    def intact(self):
        return bool((self.all[:BAND] == FILL).all()) and bool((self.all[BAND + self.n:] == FILL).all())


@pytest.mark.parametrize("rows,d", [(1, 8), (5, 200), (37, 333), (333, 1001), (160, 2048), (3, 7168),
                                    (2, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_guard_bands(rows, d, dtype):
    """No call writes outside its outputs and its workspace, whose size is
    exactly what the library asks for; inputs stay as they were."""
    laga = _laga()
    L = laga._lib
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    b, pitch, n = (2 if dtype == "bf16" else 4), L.ckpt_row_bytes(d), 77
    t = {k: (v if k.startswith(("alpha", "gamma")) else v.to(dt)) for k, v in
         _step_inputs(rows, d, n, 7).items()}
    before = {k: v.clone() for k, v in t.items()}
    p = {k: v.data_ptr() for k, v in t.items()}
    st = torch.cuda.current_stream().cuda_stream
    dims = L.make_res_dims(rows, d, gate="full", ckpt=True, io_dtype=dtype)
    o = {k: _Banded(rows * d * b) for k in ("x_out", "h", "dx_o", "dy", "dgate", "x8")}
    o.update({k: _Banded(rows * pitch) for k in ("ck_y", "ck_x", "ck")})
    o.update({k: _Banded(rows * 8) for k in ("s_post", "s_pre")})
    o.update({k: _Banded(d * 4) for k in ("dgp", "dgq")})
    o["dalpha"], o["dw"] = _Banded(4), _Banded(d * n * 4)
    o["ws"] = _Banded(L.res_workspace_bytes(dims))
    o["ws_dw"] = _Banded(L.ckpt_dw_workspace_bytes(rows, d, n, dtype))
    L.res_fwd(dims, p["x"], p["y"], p["gate"], p["alpha"], p["gamma_post"], p["gamma_pre"],
              o["x_out"].ptr, o["h"].ptr, o["ck_y"].ptr, o["ck_x"].ptr, o["s_post"].ptr,
              o["s_pre"].ptr, st)
    L.res_bwd(dims, p["dx"], p["dh"], o["ck_y"].ptr, o["ck_x"].ptr, o["s_post"].ptr,
              o["s_pre"].ptr, p["gate"], p["alpha"], p["gamma_post"], p["gamma_pre"],
              o["dx_o"].ptr, o["dy"].ptr, o["dgate"].ptr, o["dalpha"].ptr, o["dgp"].ptr,
              o["dgq"].ptr, o["ws"].ptr, o["ws"].n, st)
    L.ckpt_pack(rows, d, dtype, p["x"], o["ck"].ptr, st)
    L.ckpt_unpack(rows, d, dtype, o["ck"].ptr, o["x8"].ptr, st)
    L.ckpt_dw(rows, d, n, dtype, o["ck_x"].ptr, p["dq"], p["gamma_pre"], o["dw"].ptr,
              o["ws_dw"].ptr, o["ws_dw"].n, st)
    L.sync_check()
    for k, v in o.items():
        assert v.intact(), k
    for k, v in before.items():
        assert torch.equal(v, t[k]), k
    # and the same numbers as through the front end
    plan = laga.ResidualNorm(d, gate="full", ckpt=True, io_dtype=dtype, device=DEV)
    want = _step(plan, laga, t)
    got = [o["x_out"].view(dt, (rows, d)), o["h"].view(dt, (rows, d)), o["dx_o"].view(dt, (rows, d)),
           o["dy"].view(dt, (rows, d)), o["dgate"].view(dt, (rows, d)),
           o["dalpha"].view(torch.float32, (1,)), o["dgp"].view(torch.float32, (d,)),
           o["dgq"].view(torch.float32, (d,)), o["dw"].view(torch.float32, (d, n))]
    for i, (a, w) in enumerate(zip(got, want)):
        assert torch.equal(a, w), i
