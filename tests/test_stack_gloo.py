"""LagaResidualStack on CPU ranks (gloo): which gradients are summed over the
ranks and which stay a rank's own.

The residual operators run on a CUDA device only, so a stand-in computes them
from the fp64 oracle here, as the oracle's head shard does the per-rank
attention.  Every rank holds the same weights and its own chunk of the
sequence; the unsharded oracles give what the ranks together must."""

import math
import os

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import oracle
from oracle import residual as ores
from oracle.block import block_backward, block_forward
from test_sp_gloo import SMALL, OracleCompute, _free_port


class OracleResidualNorm:
    """sequence_latent_norm_gb300.ResidualNorm's calls, by the oracle."""

    def __init__(self, d, *, post=True, pre=True, norm_post="rms", norm_pre="rms", gate="none",
                 ckpt=False, io_dtype="bf16", eps=1e-5, device=None):
        assert not ckpt
        self.d, self.post, self.pre, self.ckpt, self.gate = d, post, pre, ckpt, gate
        self.norms, self.eps = dict(norm_post=norm_post, norm_pre=norm_pre), eps

    def forward(self, x, y=None, *, gate=None, alpha=None, gamma_post=None, gamma_pre=None):
        from sequence_latent_norm_gb300.residual import ResidualOut

        def flat(t):
            return None if t is None else t.numpy().reshape(-1, t.shape[-1])

        kw = dict(gate=flat(gate) if self.post and self.gate != "none" else None,
                  alpha=alpha if self.post else None,
                  gamma_post=gamma_post.numpy() if self.post and gamma_post is not None else None,
                  gamma_pre=gamma_pre.numpy() if self.pre else None)
        out = ores.forward(flat(x), flat(y) if self.post else None, eps=self.eps, **self.norms, **kw)

        def tensor(a):
            return torch.from_numpy(a.reshape(x.shape)) if a is not None else None

        return ResidualOut(tensor(out["x"]), tensor(out.get("h")), (out, kw, gate))

    def backward(self, saved, dx_out=None, dh=None):
        from sequence_latent_norm_gb300.residual import ResidualGrads
        out, kw, gate = saved

        def flat(t):
            return None if t is None else t.numpy().reshape(-1, self.d)

        g = ores.backward(dx_out=flat(dx_out), dh=flat(dh) if self.pre else None,
                          **{k: out.get(k) for k in ("y_hat", "x_hat", "stat_post", "stat_pre")},
                          **self.norms, **kw)
        shape = dx_out.shape

        def tensor(name, shape=None):
            a = g.get(name)
            return None if a is None else torch.from_numpy(np.array(a.reshape(shape or a.shape)))

        return ResidualGrads(tensor("dx", shape), tensor("dy", shape),
                             tensor("dgate", gate.shape) if "dgate" in g else None,
                             tensor("dalpha"), tensor("dgamma_post"), tensor("dgamma_pre"))


def _layers(rng, n, S, n_h, d_model, norm_post, gate):
    qk, hkv = SMALL["d_nope"] + SMALL["d_rope"], SMALL["d_nope"] + SMALL["d_v"]

    def rand(*s, scale=1.0):
        return rng.standard_normal(s) * scale

    out = []
    for i in range(n):
        w = dict(w_q=rand(d_model, n_h * qk, scale=1 / math.sqrt(d_model)),
                 w_kva=rand(d_model, SMALL["d_kv"] + SMALL["d_rope"], scale=1 / math.sqrt(d_model)),
                 gamma=1 + rand(SMALL["d_kv"], scale=0.1),
                 w_kvb=rand(SMALL["d_kv"], n_h * hkv, scale=1 / math.sqrt(SMALL["d_kv"])),
                 w_o=rand(n_h * SMALL["d_v"], d_model, scale=1 / math.sqrt(n_h * SMALL["d_v"])),
                 gamma_pre=1 + rand(d_model, scale=0.1), alpha=np.array([0.6 + 0.2 * i]))
        if norm_post != "none":
            w["gamma_post"] = 1 + rand(d_model, scale=0.1)
        if gate != "none":
            w["gate"] = rand(1, S, d_model if gate == "full" else 1)
        out.append(w)
    return out


def _unsharded(x, dx, layers, dims, cos, sin, norms):
    """The stream behind the last layer, dx in front of the first, and per
    layer the gradients, all over the whole sequence."""
    shape, d = x.shape, x.shape[-1]
    flat, saved = x.reshape(-1, d), []
    for w in layers:
        pre = ores.forward(flat, gamma_pre=w["gamma_pre"], **norms)
        y, st = block_forward(pre["h"].reshape(shape), w["w_q"], w["w_kva"], w["gamma"], w["w_kvb"],
                              w["w_o"], cos, sin, dims)
        kw = dict(gate=w["gate"].reshape(len(flat), -1) if "gate" in w else None, alpha=w["alpha"],
                  gamma_post=w.get("gamma_post"))
        post = ores.forward(flat, y.reshape(flat.shape), **norms, **kw)
        saved.append((pre, st, post, kw))
        flat = post["x"]
    g, grads = dx.reshape(flat.shape), []
    for w, (pre, st, post, kw) in zip(reversed(layers), reversed(saved)):
        gp = ores.backward(dx_out=g, y_hat=post["y_hat"], stat_post=post["stat_post"], **norms, **kw)
        gb = block_backward(st, gp["dy"].reshape(shape))
        gq = ores.backward(dx_out=g, dh=gb["dh"].reshape(flat.shape), x_hat=pre["x_hat"],
                           stat_pre=pre["stat_pre"], gamma_pre=w["gamma_pre"], **norms)
        g = gq["dx"]
        grads.append({**{k: v for k, v in gb.items() if k != "dh"}, "dgamma_pre": gq["dgamma_pre"],
                      **{k: gp[k] for k in ("dalpha", "dgamma_post", "dgate") if k in gp}})
    return flat.reshape(shape), g.reshape(shape), grads[::-1]


def _rank_stack(rank, world, port, norm_post, norm_pre, gate):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        from sequence_latent_norm_gb300 import block
        from sequence_latent_norm_gb300.sp import SequenceParallelLaga
        block.ResidualNorm = OracleResidualNorm
        n, S, n_h, d_model = 2, 12, 4, 7
        rng = np.random.default_rng(23)
        layers = _layers(rng, n, S, n_h, d_model, norm_post, gate)
        x, dx = rng.standard_normal((1, S, d_model)), rng.standard_normal((1, S, d_model))
        cos, sin = oracle.rope_tables(S, SMALL["d_rope"])
        norms = dict(norm_post=norm_post, norm_pre=norm_pre)
        want, want_dx, want_grads = _unsharded(x, dx, layers, oracle.Dims(S=S, H=n_h, **SMALL), cos,
                                               sin, norms)
        Sr, H = S // world, n_h // world
        seq = slice(rank * Sr, (rank + 1) * Sr)
        T = torch.from_numpy

        def mine(a):
            return T(np.ascontiguousarray(a[:, seq]))

        dims = oracle.Dims(S=S, H=H, n_h_total=n_h, head_offset=rank * H, **SMALL)
        blocks = [block.LagaAttentionBlock(SequenceParallelLaga(n_h, S, compute=OracleCompute(dims),
                                                                **SMALL), n_h, distributed=True)
                  for _ in range(n)]
        stack = block.LagaResidualStack(blocks, d_model, gate=gate, **norms)
        local = [{k: mine(v) if k == "gate" else T(v) for k, v in w.items()} for w in layers]
        out = stack.forward(mine(x), local, T(cos), T(sin))
        got_dx, got = stack.backward(mine(dx))
        tol = dict(rtol=1e-10, atol=1e-10)
        np.testing.assert_allclose(out.numpy(), want[:, seq], **tol)
        np.testing.assert_allclose(got_dx.numpy(), want_dx[:, seq], **tol)
        for i in range(n):
            assert set(got[i]) == set(want_grads[i])
            for k, v in got[i].items():
                ref = want_grads[i][k]
                if k == "dgate":       # of this rank's own logits
                    ref = ref.reshape(1, S, -1)[:, seq]
                np.testing.assert_allclose(v.numpy(), ref, **tol, err_msg=f"layer {i} {k}")
            # ring bytes of the summed fp64 parameters of the residual stream
            for k in ("dalpha", "dgamma_pre", "dgamma_post"):
                if k in got[i]:
                    size = got[i][k].numel() * 8
                    assert blocks[i].sent["all_reduce_" + k] == 2 * (world - 1) * size // world
            assert "all_reduce_dgate" not in blocks[i].sent
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("norm_post,norm_pre,gate", [("none", "rms", "none"),
                                                     ("rms", "layer", "full"),
                                                     ("layer", "rms", "token")])
def test_stack_over_ranks_matches_the_unsharded_oracles(norm_post, norm_pre, gate):
    mp.spawn(_rank_stack, args=(2, _free_port(), norm_post, norm_pre, gate), nprocs=2, join=True)


def test_stack_over_four_ranks():
    mp.spawn(_rank_stack, args=(4, _free_port(), "rms", "rms", "full"), nprocs=4, join=True)
