"""What the documentation of the residual-stream operators and the 8-bit
checkpoints allows beyond one ordinary call at a time on the current stream:
two host threads at once, inputs dropped behind a call on another stream,
parameters that are slices of larger tensors, gate logits far from zero and
without an end."""

import ctypes
import threading

import numpy as np
import pytest
import torch

from laga_inputs import as_f64
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U32 = 2.0 ** -24        # half a step of fp32, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U32}


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _raw_calls(laga, rows, d, dtype, stream):
    """A forward and a backward of both halves with a full gate as C calls on
    buffers of their own, and the outputs."""
    L = laga._lib
    so, dt = L.load(), dict(bf16=torch.bfloat16, fp32=torch.float32)[dtype]
    g = torch.Generator(device=DEV).manual_seed(d)
    x, y, gate, dx, dh = (torch.randn(rows, d, generator=g, device=DEV).to(dt) for _ in range(5))
    alpha, post, pre = (0.5 + torch.rand(n, generator=g, device=DEV) for n in (1, d, d))
    x_out, h, dx_in, dy, dgate = (torch.empty_like(x) for _ in range(5))
    st_post, st_pre = (torch.empty(rows, 2, device=DEV) for _ in range(2))
    sums = [torch.empty(n, device=DEV) for n in (1, d, d)]
    dims = L.make_res_dims(rows, d, gate="full", io_dtype=dtype)
    ws = torch.empty(L.res_workspace_bytes(dims), dtype=torch.uint8, device=DEV)
    st = ctypes.c_void_p(stream.cuda_stream)
    ref = ctypes.byref(dims)

    def ptrs(*ts):
        return [None if t is None else ctypes.c_void_p(t.data_ptr()) for t in ts]

    fwd = ptrs(x, y, gate, alpha, post, pre, x_out, h, None, None, st_post, st_pre)
    bwd = ptrs(dx, dh, y, x_out, st_post, st_pre, gate, alpha, post, pre, dx_in, dy, dgate, *sums, ws)
    outs = [x_out, h, st_post, st_pre, dx_in, dy, dgate, *sums]
    keep = (x, y, gate, dx, dh, alpha, post, pre, ws, dims)
    return (lambda: so.laga_res_fwd(ref, *fwd, st),
            lambda: so.laga_res_bwd(ref, *bwd, ws.numel(), st), outs, keep)


# Rows and widths of one kernel instance whose launches need different amounts
# of shared memory: the rings of one team shape (one row a team, or several and
# the gains), and the scalar kernels.
SHARED = [((400, 8192), (20, 4104)), ((700, 4096), (20, 2056)), ((20, 5001), (20, 333)),
          ((20, 16383), (20, 8201))]


@pytest.mark.parametrize("one,other", SHARED)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_two_host_threads(one, other, dtype):
    """Calls of two sizes from two threads, each on a stream of its own, succeed
    and give what they give alone."""
    laga = _laga()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    made = [_raw_calls(laga, *size, dtype, s) for size, s in zip((one, other), streams)]
    torch.cuda.synchronize()
    for fwd, bwd, _, _ in made:
        assert fwd() == 0 and bwd() == 0
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, _, outs, _ in made]
    for which in (0, 1):
        start, bad = threading.Barrier(2), []

        def loop(call, stream):
            start.wait()
            for i in range(6000):
                status = call()
                if status:
                    bad.append((i, status))
                if i % 500 == 499:
                    stream.synchronize()

        threads = [threading.Thread(target=loop, args=(m[which], s)) for m, s in zip(made, streams)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not bad, (("forward", "backward")[which], len(bad), bad[0])
    for (_, _, outs, _), w in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    laga._lib.sync_check()


def test_inputs_dropped_behind_a_call_on_another_stream():
    """A call on another stream than the current one may be the last use of
    its inputs: while the other stream is still busy with what came before,
    memory that the caller has dropped is not handed out again."""
    laga = _laga()
    rows, d, n = 1000, 2048, 1024
    s = torch.cuda.Stream(DEV)
    plan = laga.ResidualNorm(d, gate="full", device=DEV)
    plan8 = laga.ResidualNorm(d, gate="full", ckpt=True, device=DEV)
    for p in (plan, plan8):        # whatever a first call loads or allocates
        z = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
        one = torch.ones(d, device=DEV)
        r = p.forward(z, z, gate=z, alpha=one[:1], gamma_post=one, gamma_pre=one, stream=s)
        p.backward(r.saved, z, z, stream=s)
        laga.weight_grad8(laga.pack8(z, stream=s), z, stream=s)
    del z, one, r
    torch.cuda.synchronize()

    def inputs():
        g = torch.Generator(device=DEV).manual_seed(3)
        t = {k: torch.randn(rows, d, generator=g, device=DEV).to(torch.bfloat16)
             for k in ("x", "y", "gate", "dx", "dh")}
        t["dq"] = torch.randn(rows, n, generator=g, device=DEV).to(torch.bfloat16)
        t.update({k: 0.5 + torch.rand(m, generator=g, device=DEV)
                  for k, m in (("alpha", 1), ("gamma_post", d), ("gamma_pre", d))})
        return t

    def fwd(p, t):
        return p.forward(t["x"], t["y"], gate=t["gate"], alpha=t["alpha"],
                         gamma_post=t["gamma_post"], gamma_pre=t["gamma_pre"], stream=s)

    def kept(p):
        t = inputs()
        r = fwd(p, t)
        torch.cuda.synchronize()
        return dict(saved=r.saved, dx=t["dx"], dh=t["dh"])

    def packed():
        ck = laga.pack8(inputs()["x"], stream=s)
        torch.cuda.synchronize()
        t = inputs()
        return dict(ck=ck, dq=t["dq"], gamma=t["gamma_pre"])

    def take(r):
        return [r.x, r.h, r.saved.stat_pre]

    cases = {
        "forward": (inputs, lambda t: take(fwd(plan, t))),
        "forward in 8 bits": (inputs, lambda t: take(fwd(plan8, t))),
        "backward": (lambda: kept(plan), lambda t: plan.backward(t["saved"], t["dx"], t["dh"],
                                                                 stream=s)),
        "backward in 8 bits": (lambda: kept(plan8),
                               lambda t: plan8.backward(t["saved"], t["dx"], t["dh"], stream=s)),
        "pack": (lambda: dict(x=inputs()["x"]), lambda t: [laga.pack8(t["x"], stream=s).data]),
        "unpack": (packed, lambda t: [t["ck"].unpack(stream=s)]),
        "weight gradient": (packed, lambda t: [laga.weight_grad8(t["ck"], t["dq"], t["gamma"],
                                                                 stream=s)]),
    }
    bad = []
    for name, (make, call) in cases.items():
        t = make()
        torch.cuda.synchronize()
        want = call(t)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)           # ~50 ms
        got = call(t)
        t.clear()                                    # the last references
        # what the current stream allocates and writes meanwhile
        junk = [torch.full((k,), 77, dtype=torch.uint8, device=DEV)
                for k in [rows * d * 2, rows * n * 2, rows * laga._lib.ckpt_row_bytes(d), rows * 8,
                          d * 4, 4] * 8]
        torch.cuda.synchronize()
        if not all(torch.equal(a, b) for a, b in zip(got, want) if a is not None):
            bad.append(name)
        del junk
    assert not bad, bad
    laga._lib.sync_check()


def test_a_captured_call_on_a_forked_stream():
    """A capture that forks to another stream and joins it again, with inputs
    made and dropped inside: replayed on other values it gives what eager calls
    give."""
    laga = _laga()
    rows, d = 300, 640
    plan = laga.ResidualNorm(d, gate="full", ckpt=True, device=DEV)
    gain = torch.rand(d + 1, device=DEV)[1:]          # off a 16-byte boundary
    alpha = torch.full((1,), 0.5, device=DEV)
    side = torch.cuda.Stream(DEV)

    def step(src, stream):
        x, y, gate, dx, dh = ((src * k).to(torch.bfloat16) for k in (1, 2, 3, 4, 5))
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        r = plan.forward(x, y, gate=gate, alpha=alpha, gamma_post=gain, gamma_pre=gain,
                         stream=stream)
        g = plan.backward(r.saved, dx, dh, stream=stream)
        dw = laga.weight_grad8(r.saved.x, dx, gain, stream=stream)
        v = laga.pack8(x, stream=stream).unpack(stream=stream)
        del x, y, gate, dx, dh
        junk = torch.full((rows, d), 9.0, dtype=torch.bfloat16, device=DEV)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return [r.x, r.h, *g, v, dw], junk

    src = torch.randn(rows, d, device=DEV)
    step(src, None)
    step(src, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, junk = step(src, side)
    src.copy_(torch.randn(rows, d, device=DEV))
    want, _ = step(src, side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    laga._lib.sync_check()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("d", [512, 333])
def test_parameters_that_are_slices(d):
    """alpha, the gains and a weight gradient's gain as a model holds them: one
    layer's entries of a tensor of all layers', wherever they start."""
    laga = _laga()
    rows, layers = 40, 4
    g = torch.Generator(device=DEV).manual_seed(d)
    x, y, dx, dh = (torch.randn(rows, d, generator=g, device=DEV).to(torch.bfloat16)
                    for _ in range(4))
    alpha = 0.5 + torch.rand(layers, generator=g, device=DEV)
    gains = 0.5 + torch.rand(2 * layers * d + 1, generator=g, device=DEV)
    post, pre = gains[1:1 + layers * d].view(layers, d), gains[1 + layers * d:].view(layers, d)
    for ckpt in (False, True):
        plan = laga.ResidualNorm(d, ckpt=ckpt, device=DEV)
        for i in range(layers):
            outs = []
            for own in (lambda v: v.clone(), lambda v: v):
                par = dict(alpha=own(alpha[i:i + 1]), gamma_post=own(post[i]),
                           gamma_pre=own(pre[i]))
                r = plan.forward(x, y, **par)
                out = [r.x, r.h, *plan.backward(r.saved, dx, dh)]
                if ckpt:
                    out.append(laga.weight_grad8(r.saved.x, dx, par["gamma_pre"]))
                outs.append([v for v in out if v is not None])
            assert all(torch.equal(a, b) for a, b in zip(*outs))
    laga._lib.sync_check()


# Error of sigmoid(a) = 1 / (1 + e^-a) and of 1 - sigmoid(a) relative to
# themselves, in units of u = 2^-24.  e^-a = 2^t with t = -a log2 e: the
# rounded constant (0.23 u) and the rounded product (1 u) are each off by
# their share of a log2 e, which moves 2^t by 1.23 |a| u of itself; the
# hardware's exponential is within 2^-22 = 4 u; 1 + e^-a and its reciprocal
# (2^-23) add 3 u, the product that makes 1 - sigmoid(a) one more.
def _sigmoid_u(a):
    return (1.25 * np.abs(a) + 9.0) * U32


# below this the sigmoid is no normal fp32 number any more; it may be zero
TINY = 2.0 ** -126

FINITE = [-100.0, -95.0, -90.0, -88.0, -87.0, -86.0, -80.0, -60.0, -40.0, -20.0, -10.0, -5.0, -1.0,
          -0.125, 0.0, 0.125, 1.0, 5.0, 10.0, 20.0, 40.0, 60.0, 80.0, 86.0, 87.0, 88.0, 90.0, 100.0]


def _gate_run(gate, d, kind, dtype, x0=0.0):
    """alpha = y = dx_out = 1 and no norm: x' = x + s, dy = s and dgate = s (1 -
    s), each summed over the row for a token gate."""
    plan = _laga().ResidualNorm(d, pre=False, norm_post="none", gate=kind, device=DEV,
                                io_dtype="bf16" if dtype == torch.bfloat16 else "fp32")
    rows = gate.shape[0]
    x = torch.full((rows, d), x0, dtype=dtype, device=DEV)
    y = torch.ones(rows, d, dtype=dtype, device=DEV)
    r = plan.forward(x, y, gate=gate.to(DEV), alpha=torch.ones(1, device=DEV))
    g = plan.backward(r.saved, y)
    _laga()._lib.sync_check()
    return as_f64(r.x), as_f64(g.dy), as_f64(g.dgate)


@pytest.mark.parametrize("d", [512, 333])
@pytest.mark.parametrize("kind", ["full", "token"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gate_logits_far_from_zero(d, kind, dtype):
    a = torch.tensor(FINITE)
    gate = (a.repeat(1 + d // len(a))[:d].repeat(5, 1) if kind == "full" else a[:, None]).to(dtype)
    v = as_f64(gate)
    s, c, u = ores.sigmoid(v), ores.sigmoid(-v), _sigmoid_u(v)
    x, dy, dgate = _gate_run(gate, d, kind, dtype)
    tol = s * (u + HALF[dtype]) * (1 + 2.0 ** -7) + TINY
    assert (np.abs(x - s) <= tol).all() and (np.abs(dy - s) <= tol).all()
    # s (1 - s): two of the errors and three products; d terms add d u at most
    n, add = (d, d * U32) if kind == "token" else (1, 0.0)
    tol = n * (s * c * (2 * u + 3 * U32 + add + HALF[dtype]) * (1 + 2.0 ** -7) + TINY)
    assert (np.abs(dgate - n * s * c) <= tol).all()


@pytest.mark.parametrize("d", [512, 333])
@pytest.mark.parametrize("kind", ["full", "token"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gate_logits_without_an_end(d, kind, dtype):
    """-inf shuts a gate and +inf opens it, exactly, and neither has a
    gradient; a NaN is one in what it gates."""
    inf, nan = float("inf"), float("nan")
    if kind == "full":
        gate = torch.zeros(4, d)
        gate[0, 3], gate[1, 5], gate[2, d - 1] = -inf, inf, nan
        at = (np.array([0, 1, 2]), np.array([3, 5, d - 1]))
    else:
        gate = torch.tensor([-inf, inf, nan, 0.0])[:, None]
        at = (np.array([0, 1, 2]), slice(None))
    for x0 in (0.0, 3.0):
        x, dy, dgate = _gate_run(gate.to(dtype), d, kind, dtype, x0)
        want = np.full((4, d), 0.5)
        for i, s in enumerate((0.0, 1.0, nan)):
            want[at[0][i], at[1] if kind == "token" else at[1][i]] = s
        assert np.array_equal(x, x0 + want, equal_nan=True)
        assert np.array_equal(dy, want, equal_nan=True)
        want = want * (1 - want)
        if kind == "token":     # rounded once: 333/4 = 83.25 has a bit more than bf16 holds
            want = as_f64(torch.from_numpy(want.sum(axis=1, keepdims=True)).to(dtype))
        assert np.array_equal(dgate, want, equal_nan=True)
