"""The experts' operators as they are used: the routed block against the fp64
oracle, blocks of both kinds on a residual stream, 8-bit projections of the
attention block; captured and replayed, on other streams, from two host
threads, inside guard bands.

Tolerances.  The block's oracle makes the same roundings, to 8 bits and to bf16;
what is left are sums in another order, which move a bf16 value by one step
(2^-8) or an 8-bit one by one (2^-3) where they fall next to a border: of n
values, a fraction of some 2^-24 sqrt(K) / 2^-9 of the bf16 ones, each by 2^-8 of
itself.  Every bf16 boundary is allowed 2^-9 (the rounding it makes), five of
them on the longest way: 1e-2, as for the attention block."""

import threading

import numpy as np
import pytest
import torch

from laga_inputs import as_f64, config, make_block_inputs
from oracle import experts as oex
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
REL_FRO = 1e-2


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _rel(a, b):
    return float(np.linalg.norm(as_f64(a) - b) / max(np.linalg.norm(b), 1e-30))


def _inputs(T, d, f, E, seed=0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return dict(h=torch.randn(T, d, generator=g).to(dtype),
                w_router=torch.randn(d, E, generator=g) * d ** -0.5,
                w_in=(torch.randn(E, d, 2 * f, generator=g) * d ** -0.5).to(dtype),
                w_out=(torch.randn(E, f, d, generator=g) * f ** -0.5).to(dtype),
                bias=0.1 * torch.randn(E, generator=g), dy=torch.randn(T, d, generator=g).to(dtype))


def _dev(x):
    return {k: v.to(DEV) for k, v in x.items()}


def _run(block, x):
    y = block.forward(x["h"], x["w_router"], x["w_in"], x["w_out"], bias=x["bias"])
    return y, block.backward(x["dy"])


@pytest.mark.parametrize("T,d,f,E,k,kw", [(100, 256, 192, 8, 2, {}),
                                          (37, 200, 136, 12, 3, dict(groups=4, top_groups=2, scale=2.5)),
                                          (300, 384, 128, 5, 5, dict(score="softmax", renormalise=False)),
                                          (1, 128, 64, 16, 4, {})])
def test_block_matches_the_oracle(T, d, f, E, k, kw):
    laga = _laga()
    x = _inputs(T, d, f, E, seed=T)
    y, g = _run(laga.RoutedExperts(E, k, device=DEV, **kw), _dev(x))
    laga._lib.sync_check()
    a = {n: as_f64(v) for n, v in x.items()}
    want, st = oex.block_fwd(a["h"], a["w_router"], a["bias"], a["w_in"], a["w_out"], top_k=k, **kw)
    assert _rel(y, want) <= REL_FRO
    for n, v in oex.block_bwd(st, a["dy"]).items():
        assert g[n].shape == v.shape and _rel(g[n], v) <= REL_FRO, (n, _rel(g[n], v))


def test_block_in_fp32_and_with_packed_weights():
    """fp32 in and out: nothing but the 8-bit roundings; weights packed once give
    the same bits as weights packed in the call."""
    laga = _laga()
    x = _dev(_inputs(64, 256, 128, 6, dtype=torch.float32))
    block = laga.RoutedExperts(6, 2, io_dtype="fp32", device=DEV)
    y, g = _run(block, x)
    y2, g2 = _run(block, dict(x, w_in=laga.pack_weight8(x["w_in"]), w_out=laga.pack_weight8(x["w_out"])))
    laga._lib.sync_check()
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    a = {n: as_f64(v) for n, v in x.items()}
    want, st = oex.block_fwd(a["h"], a["w_router"], a["bias"], a["w_in"], a["w_out"], top_k=2,
                             io="fp32")
    assert y.dtype == torch.float32 and _rel(y, want) <= REL_FRO
    for n, v in oex.block_bwd(st, a["dy"]).items():
        assert _rel(g[n], v) <= REL_FRO, n


def test_transposed_weights():
    """Weights that are views of another order give the same bits."""
    from sequence_latent_norm_gb300.block import LagaAttentionBlock
    laga = _laga()

    def turned(w):
        return w.transpose(-1, -2).contiguous().transpose(-1, -2)

    x = _dev(_inputs(40, 256, 128, 4))
    block = laga.RoutedExperts(4, 2, device=DEV)
    y, g = _run(block, x)
    y2, g2 = _run(block, dict(x, w_in=turned(x["w_in"]), w_out=turned(x["w_out"])))
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    wl = config(1, S=130, H=2, n_h_total=2, seed=6)
    b = {n: v.to(DEV) for n, v in make_block_inputs(wl, 320).items()}
    for n in ("h", "w_q", "w_kva", "w_kvb", "w_o", "dy"):
        b[n] = b[n].to(torch.bfloat16)
    blk = LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV), projections="fp8")
    names = ("h", "w_q", "w_kva", "gamma", "w_kvb", "w_o", "cos", "sin")
    y = blk.forward(*(b[n] for n in names))
    t = dict(b, **{n: turned(b[n]) for n in ("w_q", "w_kva", "w_o")})
    assert not t["w_q"].is_contiguous()
    y2 = blk.forward(*(t[n] for n in names))
    laga._lib.sync_check()
    assert torch.equal(y, y2)


def test_kept_checkpoint_serves_the_weight_gradients():
    laga = _laga()
    x = _dev(_inputs(90, 256, 64, 4))
    gain = 0.5 + torch.rand(256, device=DEV)
    kept = laga.pack8((x["h"].float() / gain).to(torch.bfloat16))
    block = laga.RoutedExperts(4, 2, device=DEV)
    _, g = _run(block, x)
    block.forward(x["h"], x["w_router"], x["w_in"], x["w_out"], bias=x["bias"], kept=kept,
                  kept_gain=gain)
    g2 = block.backward(x["dy"])
    laga._lib.sync_check()
    assert torch.equal(g["dh"], g2["dh"]) and torch.equal(g["dw_out"], g2["dw_out"])
    # two 8-bit roundings of h: 2^-3 / sqrt(12) of the values in the mean, each
    for n in ("dw_in", "dw_router"):
        assert not torch.equal(g[n], g2[n])
        assert _rel(g2[n], as_f64(g[n])) <= 2 * 0.036, n


def test_captured_step_follows_its_inputs():
    """A captured forward and backward, replayed with other tokens, other
    choices and another number of rows a expert, gives what an eager step gives."""
    laga = _laga()
    block, eager = laga.RoutedExperts(8, 2, device=DEV), laga.RoutedExperts(8, 2, device=DEV)
    x = _dev(_inputs(130, 256, 128, 8))
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(block, x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, g = _run(block, x)
    for seed in (1, 2):
        new = _dev(_inputs(130, 256, 128, 8, seed=seed))
        if seed == 2:
            new["bias"][3:] = -float("inf")           # five experts without rows
        for n in x:
            x[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        y2, g2 = _run(eager, new)
        laga._lib.sync_check()
        assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_padding_tokens_take_no_part():
    """Tokens whose logits are all -inf: no rows, zero outputs, no gradient."""
    laga = _laga()
    T, E = 40, 6
    g = torch.Generator().manual_seed(3)
    l = torch.randn(T, E, generator=g)
    l[10:20] = -float("inf")
    r = laga.Router(E, 2, device=DEV)
    routes = r.forward(l.to(DEV))
    assert (routes.row[10:20] == -1).all() and int((routes.pair >= 0).sum()) == 60
    y = torch.randn(routes.rows, 64, generator=g).to(DEV)
    assert (laga.combine(y, routes)[10:20] == 0).all()
    dy, dw = laga.combine_grad(torch.randn(T, 64, generator=g).to(DEV), routes, y=y)
    assert (dw[10:20] == 0).all()
    dl = r.backward(l.to(DEV), routes, dw)
    assert (dl[10:20] == 0).all() and torch.isfinite(dl).all()


@pytest.mark.parametrize("ckpt", [False, True])
def test_stack_of_attention_and_experts(ckpt):
    """A transformer layer on a residual stream equals its parts called one by
    one, and keeps no activation but in 8 bits with ``ckpt``."""
    from sequence_latent_norm_gb300.block import LagaAttentionBlock, LagaResidualStack
    laga = _laga()
    d, E = 256, 6
    wl = config(1, S=192, H=2, n_h_total=2, seed=5)
    b = {n: v.to(DEV) for n, v in make_block_inputs(wl, d).items()}
    e = _dev(_inputs(wl.S, d, 128, E))
    gen = torch.Generator().manual_seed(8)
    layers = [{n: b[n] for n in ("w_q", "w_kva", "gamma", "w_kvb", "w_o")},
              {n: e[n] for n in ("w_router", "w_in", "w_out", "bias")}]
    for w in layers:
        w["gamma_pre"] = (1 + 0.1 * torch.randn(d, generator=gen)).to(DEV)
        w["alpha"] = torch.tensor([0.7], device=DEV)

    def blocks():
        return [LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV)),
                laga.RoutedExperts(E, 2, device=DEV)]

    stack = LagaResidualStack(blocks(), d, ckpt=ckpt, device=DEV)
    y = stack.forward(b["h"], layers, b["cos"], b["sin"])
    dx, grads = stack.backward(b["dy"])
    laga._lib.sync_check()
    assert set(grads[1]) == {"dw_router", "dw_in", "dw_out", "dalpha", "dgamma_pre"}

    # the parts
    kw = dict(ckpt=ckpt, norm_post="none", device=DEV)
    first, mid, last = (laga.ResidualNorm(d, post=p, pre=q, **kw) for p, q in
                        ((False, True), (True, True), (True, False)))
    attn, exp = blocks()
    r0 = first.forward(b["h"], gamma_pre=layers[0]["gamma_pre"])
    held = [dict(kept=r.x, kept_gain=w["gamma_pre"]) if ckpt else {} for r, w in
            ((r0.saved, layers[0]),)][0]
    y0 = attn.forward(r0.h, *(b[n] for n in ("w_q", "w_kva", "gamma", "w_kvb", "w_o", "cos", "sin")),
                      **held)
    r1 = mid.forward(r0.x, y0, alpha=layers[0]["alpha"], gamma_pre=layers[1]["gamma_pre"])
    held = dict(kept=r1.saved.x, kept_gain=layers[1]["gamma_pre"]) if ckpt else {}
    y1 = exp.forward(r1.h, e["w_router"], e["w_in"], e["w_out"], bias=e["bias"], **held)
    r2 = last.forward(r1.x, y1, alpha=layers[1]["alpha"])
    assert torch.equal(r2.x, y)
    g2 = last.backward(r2.saved, b["dy"])
    ge = exp.backward(g2.dy)
    g1 = mid.backward(r1.saved, g2.dx, ge["dh"])
    ga = attn.backward(g1.dy)
    g0 = first.backward(r0.saved, g1.dx, ga["dh"])
    laga._lib.sync_check()
    assert torch.equal(g0.dx, dx)
    for n in ("dw_router", "dw_in", "dw_out"):
        assert torch.equal(ge[n], grads[1][n]), n
    assert torch.equal(g1.dgamma_pre, grads[1]["dgamma_pre"])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_projections_in_8_bits(io):
    """Every projection of the attention block equals the product of what its
    operands' codes stand for, and every gradient theirs."""
    from sequence_latent_norm_gb300.block import LagaAttentionBlock
    laga = _laga()
    d = 320
    dt = dict(bf16=torch.bfloat16, fp32=torch.float32)[io]
    half = dict(bf16=2.0 ** -8, fp32=2.0 ** -24)[io]
    wl = config(1, S=130, H=2, n_h_total=2, seed=6)
    b = {n: v.to(DEV) for n, v in make_block_inputs(wl, d).items()}
    for n in ("h", "w_q", "w_kva", "w_kvb", "w_o", "dy"):
        b[n] = b[n].to(dt)
    blk = LagaAttentionBlock.single(wl.H, wl.S, device=torch.device(DEV), projections="fp8",
                                    io_dtype=io)
    seen = {}
    inner = blk.attn

    class Spy:
        def forward(self, q, c, *a):
            seen["q"], seen["c"] = q, c
            seen["out"], lse = inner.forward(q, c, *a)
            return seen["out"], lse

        def backward(self, d_out):
            seen["d_out"] = d_out
            seen["grads"] = inner.backward(d_out)
            return seen["grads"]

    blk.attn = Spy()
    y = blk.forward(*(b[n] for n in ("h", "w_q", "w_kva", "gamma", "w_kvb", "w_o", "cos", "sin")))
    g = blk.backward(b["dy"])
    laga._lib.sync_check()
    T = wl.S

    def codes(t):
        return as_f64(laga.pack8(t.reshape(T, -1).contiguous()).unpack(torch.float32))

    def weight(t):
        return as_f64(laga.pack_weight8(t).unpack(torch.float32))

    def check(got, a, m, extra=0.0):
        want, mag = a @ m, np.abs(a) @ np.abs(m)
        lim = (a.shape[1] + 64) * 2.0 ** -23 * mag + half * np.abs(want) + extra
        assert (np.abs(as_f64(got).reshape(want.shape) - want) <= lim).all()

    check(seen["q"], codes(b["h"]), weight(b["w_q"]))
    check(seen["c"], codes(b["h"]), weight(b["w_kva"]))
    check(y, codes(seen["out"]), weight(b["w_o"]))
    check(seen["d_out"], codes(b["dy"]), weight(b["w_o"]).T)
    dq, dc = seen["grads"][0], seen["grads"][1].to(dt)
    one, two = (codes(t) @ weight(w).T for t, w in ((dq, b["w_q"]), (dc, b["w_kva"])))
    mags = [np.abs(codes(t)) @ np.abs(weight(w)).T for t, w in ((dq, b["w_q"]), (dc, b["w_kva"]))]
    lim = sum(700 * 2.0 ** -23 * m for m in mags) + 2 * half * (np.abs(one) + np.abs(two))
    assert (np.abs(as_f64(g["dh"]).reshape(T, d) - one - two) <= lim).all()
    check(g["dw_q"], codes(b["h"]).T, as_f64(dq).reshape(T, -1))
    check(g["dw_kva"], codes(b["h"]).T, as_f64(dc).reshape(T, -1))
    check(g["dw_o"], codes(seen["out"]).T, as_f64(b["dy"]).reshape(T, -1))


def test_other_stream_and_dropped_inputs():
    """Calls on a stream of the caller's whose inputs are dropped as soon as they
    return."""
    laga = _laga()
    side = torch.cuda.Stream(DEV)
    x = _dev(_inputs(500, 512, 256, 8))
    l = torch.randn(500, 8, generator=torch.Generator().manual_seed(1)).to(DEV)
    router = laga.Router(8, 2, device=DEV)

    def chain(stream):
        h, w = x["h"].clone(), x["w_in"].clone()
        logits = l.clone()
        torch.cuda.synchronize()
        r = router.forward(logits, stream=stream)
        del logits
        h8 = laga.pack8(h, stream=stream)
        del h
        w8 = laga.pack_weight8(w, stream=stream)
        del w
        xs = laga.spread8(h8, r, stream=stream)
        del h8
        gu = laga.linear8(xs, w8, routes=r, stream=stream)
        del xs
        a8 = laga.swiglu8(gu, routes=r, stream=stream)
        dgu = laga.swiglu8_grad(gu, gu[:, :256].contiguous() if stream is None else _half(gu, stream),
                                routes=r, stream=stream)
        del gu
        dw = laga.weight_grad8(a8, dgu, stream=stream, routes=r)
        out = laga.combine(dgu, r, stream=stream)
        junk_now = [torch.full((4 << 20,), 7.0, device=DEV) for _ in range(8)]   # of the current stream
        torch.cuda.synchronize()
        del junk_now
        return r, out, dw

    def _half(gu, stream):
        with torch.cuda.stream(stream):
            return gu[:, :256].contiguous()

    a, b = chain(None), chain(side)
    laga._lib.sync_check()
    for s, t in zip(a[0][:5], b[0][:5]):
        assert torch.equal(s, t)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_two_host_threads():
    """Two threads, each on a stream of its own, with products of other sizes:
    the kernels' shared-memory limits and scratch belong to no one call."""
    laga = _laga()
    cases = [(_dev(_inputs(400, 256, 128, 8, seed=1)), 8), (_dev(_inputs(3, 512, 64, 40, seed=2)), 40)]
    want = [_run(laga.RoutedExperts(E, 2, device=DEV), x) for x, E in cases]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            x, E = cases[i]
            s = torch.cuda.Stream(DEV)
            with torch.cuda.stream(s):
                block = laga.RoutedExperts(E, 2, device=DEV)
                for _ in range(20):
                    got[i] = _run(block, x)
            s.synchronize()
        except Exception as e:                        # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    laga._lib.sync_check()
    for (y, g), (y2, g2) in zip(want, got):
        assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)


BAND = 4096


class Banded:
    """A buffer of so many bytes between two bands of a fixed pattern."""

    def __init__(self, nbytes):
        self.n = max(int(nbytes), 16)
        self.buf = torch.full((self.n + 2 * BAND,), 0xA5, dtype=torch.uint8, device=DEV)
        self.ptr = self.buf.data_ptr() + BAND

    def intact(self):
        return bool((self.buf[:BAND] == 0xA5).all() and (self.buf[BAND + self.n:] == 0xA5).all())


@pytest.mark.parametrize("T,d,n,E,k,align", [(37, 129, 257, 5, 2, 1), (1, 1001, 64, 8, 3, 128),
                                             (300, 256, 384, 3, 2, 128), (9, 7168, 33, 2, 1, 1),
                                             (260, 300, 200, 2, 2, 128)])
def test_nothing_is_written_outside(T, d, n, E, k, align):
    laga = _laga()
    L = laga._lib
    gen = torch.Generator().manual_seed(T)
    st = torch.cuda.current_stream().cuda_stream
    l = torch.randn(T, E, generator=gen).to(DEV)
    dims = L.make_route_dims(T, E, k, align=align)
    rows = L.route_rows(dims)
    nb = L.route_workspace_bytes(dims)
    out = {name: Banded(b) for name, b in [("expert", 4 * T * k), ("weight", 4 * T * k),
           ("row", 4 * T * k), ("pair", 4 * rows), ("start", 4 * (E + 1)), ("ws", nb),
           ("dlogits", 4 * T * E)]}
    p = {name: b.ptr for name, b in out.items()}
    L.route_fwd(dims, l.data_ptr(), 0, p["expert"], p["weight"], p["row"], p["pair"], p["start"],
                p["ws"], nb, st)
    L.route_bwd(dims, l.data_ptr(), p["expert"], p["weight"], p["dlogits"], st)
    end = p["start"] + 4 * E
    row_x, row_n = L.ckpt_row_bytes(d), L.ckpt_row_bytes(n)
    for dtype, size, dt in (("bf16", 2, torch.bfloat16), ("fp32", 4, torch.float32)):
        x8 = laga.pack8(torch.randn(T, d, generator=gen).to(DEV))
        w = torch.randn(E, d, n, generator=gen).to(DEV).to(dt)
        dy = torch.randn(T, n, generator=gen).to(DEV).to(dt)
        mm, dwb = L.mm8_workspace_bytes(rows, d, n, E, dtype), 0
        more = [("fwd", E * n * row_x), ("bwd", E * d * row_n), ("xs", rows * row_x),
                ("y", rows * n * size), ("mm_ws", mm), ("out", T * n * size),
                ("dys", rows * n * size), ("dweight", 4 * T * k), ("dw", 4 * E * d * n)]
        if align == 128:
            dwb = L.experts_dw_workspace_bytes(rows, d, n, E, dtype)
            more.append(("dw_ws", dwb))
        if n % 2 == 0:
            more += [("a8", rows * L.ckpt_row_bytes(n // 2)), ("dgu", rows * n * size)]
        out.update({f"{name} {dtype}": Banded(b) for name, b in more})
        q = {name: out[f"{name} {dtype}"].ptr for name, _ in more}
        L.weight_pack(E, d, n, dtype, w.data_ptr(), q["fwd"], q["bwd"], st)
        L.spread8(rows, T, k, d, x8.data.data_ptr(), p["pair"], end, q["xs"], st)
        L.mm8(rows, d, n, E, dtype, q["xs"], q["fwd"], p["start"], p["pair"] if align > 1 else 0,
              q["y"], q["mm_ws"], mm, st)
        L.combine_fwd(T, k, rows, n, dtype, q["y"], p["weight"], p["row"], q["out"], st)
        L.combine_bwd(T, k, rows, n, dtype, dy.data_ptr(), q["y"], p["weight"], p["row"], p["pair"],
                      end, q["dys"], q["dweight"], st)
        if align == 128:
            L.experts_dw(rows, d, n, E, dtype, q["xs"], q["dys"], 0, p["start"], q["dw"], q["dw_ws"],
                         dwb, st)
        if n % 2 == 0:
            L.swiglu_fwd(rows, n // 2, dtype, q["y"], end, q["a8"], st)
            L.swiglu_bwd(rows, n // 2, dtype, q["y"], q["y"], end, q["dgu"], st)
    L.sync_check()
    assert [name for name, b in out.items() if not b.intact()] == []


def test_launch_counts_and_error_leave_nothing_behind():
    laga = _laga()
    x8, w8 = laga.pack8(torch.randn(4, 1024, device=DEV)), laga.pack_weight8(torch.randn(1024, 512, device=DEV))
    laga.linear8(x8, w8)
    assert laga._lib.last_launch_count() == 2            # a split product and its join
    with pytest.raises(ValueError):
        laga.linear8(laga.pack8(torch.randn(4, 128, device=DEV)), w8)
    with pytest.raises(laga.LagaError):
        laga._lib.mm8(4, 1024, 512, 0, "bf16", x8.data.data_ptr(), 0, 0, 0, x8.data.data_ptr(), 0, 0)
    assert laga._lib.last_launch_count() == 0
    laga._lib.sync_check()


def test_values_at_the_ends_of_the_scales():
    """Rows and weights whose scales are the largest and smallest there are:
    products beyond fp32 are infinite, below it zero, and rows beside them keep
    their values."""
    laga = _laga()
    x = torch.ones(5, 256)
    x[0] *= 2.0 ** 119
    x[1] *= 2.0 ** -120
    x[3] = 0.0
    w = torch.eye(256)
    w[:, 200:] *= 2.0 ** 100
    x8, w8 = ores.pack(as_f64(x)), oex.pack_weight(as_f64(w[None]))
    y = laga.linear8(laga.Checkpoint8(torch.from_numpy(x8).to(DEV), 256),
                     laga.Weight8((256, 256), torch.from_numpy(w8[0]).to(DEV)), dtype=torch.float32)
    laga._lib.sync_check()
    want, _ = oex.mm8(x8, w8[0], 256, 256)
    y = as_f64(y)
    small = np.abs(want) < 2.0 ** -120
    big = np.abs(want) >= 2.0 ** 128
    assert np.isinf(y[big]).all() and (np.abs(y[small]) <= 2.0 ** -119).all()
    rest = ~small & ~big
    assert (y[rest] == want[rest]).all() and (y[3] == 0).all()


def test_more_than_2_31_elements():
    """Outputs, rows and codes whose offsets do not fit 32 bits; values that tell
    the rows apart."""
    laga = _laga()
    T, n = 140000, 16384                               # 2.3e9 elements
    x = torch.zeros(T, 128, device=DEV)
    r = torch.arange(T, device=DEV)
    for c in range(18):                                # the row number in bits: exact codes
        x[:, c] = (r >> c & 1).float()
    w = torch.zeros(128, n, device=DEV)
    w[:18, -1] = w[:18, 5] = 1.0
    w[:18, -2] = torch.arange(1, 19, device=DEV).float().clamp(max=16)
    y = laga.linear8(laga.pack8(x), laga.pack_weight8(w, backward=False))
    laga._lib.sync_check()
    ones, weighted = x.sum(dim=1), x[:, :18] @ w[:18, -2]
    assert torch.equal(y[:, -1].float(), ones) and torch.equal(y[:, 5].float(), ones)
    assert torch.equal(y[:, -2].float(), weighted.to(torch.bfloat16).float())
    assert not y[:, 6:-2].any()
    a8 = laga.swiglu8(y)                               # u = silu's partner: columns 8192 on
    laga._lib.sync_check()
    assert a8.shape == (T, n // 2) and not a8.data[:, :n // 2].any()
    routes = laga.Routes(torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(T, 1, device=DEV),
                         r.flip(0)[:, None].int().contiguous(), r.flip(0).int().contiguous(),
                         torch.tensor([0, T], dtype=torch.int32, device=DEV), 1)
    out = laga.combine(y, routes)
    dy, dw = laga.combine_grad(out, routes, y=y)
    laga._lib.sync_check()
    assert torch.equal(out[:, -1], y[:, -1].flip(0)) and torch.equal(dy, y)
    want = 2 * ones.flip(0).double() ** 2 + weighted.to(torch.bfloat16).flip(0).double() ** 2
    assert ((dw[:, 0].double() - want).abs() <= 2.0 ** -22 * want).all()
    back = laga.spread8(a8, routes)
    laga._lib.sync_check()
    assert back.data.shape == a8.data.shape and torch.equal(back.data[-1], a8.data[0])
