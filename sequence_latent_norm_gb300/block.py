"""The full MLA attention block around the per-rank LAGA compute.

Algorithm 1 of the LAGA page ("A Training-Memory Regression in MLA Sequence
Parallelism ... LAGA", Section 3.3), on one rank of P:

  step 1     q = h W_q and [latent | k_pe] = h W_kv_a on the rank's chunk
             of the sequence (the latent norm is applied by the compute,
             after the gather: it is per token, so the result is the same)
  steps 2-6  ``attn``: ``sp.SequenceParallelLaga`` (the q / O all-to-alls
             and the latent all-gather around laga_fwd), or, at one rank
             without a process group, the library directly
  step 7     y = reshape(out) W_o on the rank's chunk

W_q, W_kv_a and W_o are plain bias-free dense GEMMs: they run as torch
matmuls (cuBLAS on the GPU, in the I/O dtype with fp32 accumulation).
Every step of the LAGA compute itself runs in the library's kernels.

Backward, for the loss sum(y * dy):
  dW_o = out^T dy,  d_out = dy W_o^T,
  (dq, dc, dW_kv_b, dgamma) = attn.backward(d_out),
  dW_q = h^T dq,  dW_kv_a = h^T dc,  dh = dq W_q^T + dc W_kv_a^T.
Every rank holds the same W_q, W_kv_a and W_o and a different chunk of the
sequence, so their gradients are summed over the ranks (all-reduce);
``attn`` already assembles dW_kv_b along the head axis and sums dgamma.
The weight gradients come out of the GEMMs in the I/O dtype and are
returned in (at least) fp32.

What the block holds of h between the passes serves dW_q and dW_kv_a alone.
``checkpoint="fp8"`` holds it in 8 bits (``checkpoint.py``) and takes both
gradients, in fp32, straight from the codes.

``LagaResidualStack`` puts blocks on a residual stream, each with its norm in
front, and its norm, gate and residual scale behind (``residual.py``); between
two blocks both run in one kernel.  The paper leaves this part of the
transformer open.
"""

from __future__ import annotations

import collections

import torch.distributed as dist

from .sp import LibraryCompute, SequenceParallelLaga
from .api import Shard
from .checkpoint import Checkpoint8, pack8, weight_grad8
from .residual import ResidualNorm


def _wide(t):
    """A weight gradient in at least fp32."""
    return t.float() if t.element_size() < 4 else t


class LagaAttentionBlock:
    """One rank's attention block.  ``attn`` runs steps 2-6 (``forward(q,
    c, w_kvb, gamma, cos, sin) -> (out, lse)`` on the rank's chunk,
    ``backward(d_out) -> (dq, dc, dw_kvb, dgamma)``); ``group`` is the
    process group whose ranks share the weights (None: one rank, no
    collective); ``checkpoint`` how h is held between the passes ("none": as
    given, "fp8": in 8 bits, on a CUDA device)."""

    def __init__(self, attn, n_h: int, group=None, distributed: bool = False,
                 checkpoint: str = "none"):
        if checkpoint not in ("none", "fp8"):
            raise ValueError(f"checkpoint={checkpoint!r}: one of none, fp8")
        self.checkpoint = checkpoint
        self.attn = attn
        self.n_h = n_h
        self.group = group
        self.distributed = distributed
        self.sent = collections.Counter()
        self._saved = None

    @classmethod
    def sequence_parallel(cls, n_h: int, S: int, *, group=None, device=None,
                          checkpoint: str = "none", **dims):
        """A rank of a sequence-parallel group (torch.distributed must be
        initialised): the library on its n_h/P heads behind sp.py's
        exchanges."""
        return cls(SequenceParallelLaga(n_h, S, group=group, device=device, **dims), n_h, group,
                   distributed=True, checkpoint=checkpoint)

    @classmethod
    def single(cls, n_h: int, S: int, *, device=None, B: int = 1, checkpoint: str = "none",
               **dims):
        """All n_h heads and the whole sequence on one device, no process
        group: the library directly."""
        shard = Shard(S=S, H=n_h, n_h_total=n_h, B=B, **dims)
        return cls(LibraryCompute(shard, device), n_h, checkpoint=checkpoint)

    def forward(self, h, w_q, w_kva, gamma, w_kvb, w_o, cos, sin, *, kept=None, kept_gain=None):
        """h [B, S_r, d_model] (this rank's chunk); w_q [d_model, n_h (d_nope
        + d_rope)]; w_kva [d_model, d_kv + d_rope]; gamma [d_kv] fp32;
        w_kvb [d_kv, n_h (d_nope + d_v)]; w_o [n_h d_v, d_model]; cos/sin
        [S, d_rope/2] fp32 for the full sequence.  Returns y [B, S_r,
        d_model] in h's dtype.  ``kept``, a Checkpoint8 with h = kept *
        kept_gain (fp32 [d_model] or None), is held instead of h."""
        B, S_r, d_model = h.shape
        if kept is None:
            if kept_gain is not None:
                raise ValueError("kept_gain without kept: h is held as given")
        elif not isinstance(kept, Checkpoint8):
            raise TypeError("kept must be a Checkpoint8")
        elif (kept.rows, kept.d) != (B * S_r, d_model):
            raise ValueError(f"kept: a checkpoint of {kept.rows} rows of {kept.d}, expected "
                             f"{B * S_r} of {d_model}")
        h_flat = h.reshape(B * S_r, d_model)
        q = (h_flat @ w_q).reshape(B, S_r, self.n_h, -1)
        c = (h_flat @ w_kva).reshape(B, S_r, -1)
        out, _ = self.attn.forward(q, c, w_kvb, gamma, cos, sin)
        out_flat = out.reshape(B * S_r, -1)
        if kept is None and self.checkpoint == "fp8":
            kept = pack8(h_flat.contiguous())
        elif kept is None:
            kept = h_flat
        self._saved = (kept, kept_gain, w_q, w_kva, w_o, out_flat, out.shape, h.shape)
        return (out_flat @ w_o).reshape(B, S_r, d_model)

    def _all_reduce(self, t, what):
        if not self.distributed:
            return t
        P = dist.get_world_size(self.group)
        self.sent[what] += 2 * (P - 1) * t.numel() * t.element_size() // P
        dist.all_reduce(t, group=self.group)
        return t

    def backward(self, dy):
        """dy [B, S_r, d_model] (the rank's chunk).  Returns a dict: dh
        [B, S_r, d_model] in h's dtype; dw_q, dw_kva, dw_o (fp32, summed
        over the ranks); dw_kvb [d_kv, n_h (d_nope + d_v)] and dgamma
        [d_kv] (fp32, from ``attn``)."""
        kept, gain, w_q, w_kva, w_o, out_flat, out_shape, h_shape = self._saved
        rows = out_flat.shape[0]
        dy_flat = dy.reshape(rows, -1)
        dw_o = _wide(out_flat.t() @ dy_flat)
        d_out = (dy_flat @ w_o.t()).reshape(out_shape)
        dq, dc, dw_kvb, dgamma = self.attn.backward(d_out)
        dq_flat = dq.reshape(rows, -1)
        dc_flat = dc.reshape(rows, -1)
        dc_io = dc_flat.to(dq.dtype)
        dh = (dq_flat @ w_q.t() + dc_io @ w_kva.t()).reshape(h_shape)
        if isinstance(kept, Checkpoint8):
            dw_q = weight_grad8(kept, dq_flat, gain)
            dw_kva = weight_grad8(kept, dc_flat, gain)
        else:
            dw_q = _wide(kept.t() @ dq_flat)
            dw_kva = _wide(kept.t() @ dc_io)
        return dict(dh=dh, dw_q=self._all_reduce(dw_q, "all_reduce_dw_q"),
                    dw_kva=self._all_reduce(dw_kva, "all_reduce_dw_kva"),
                    dw_o=self._all_reduce(dw_o, "all_reduce_dw_o"),
                    dw_kvb=dw_kvb, dgamma=dgamma)


class LagaResidualStack:
    """Attention blocks on a residual stream x [B, S_r, d_model] (contiguous):

        h_l = N_pre(x_l) gamma_pre,  y_l = block_l(h_l),
        x_{l+1} = x_l + alpha s N_post(y_l) gamma_post

    ``blocks``: one LagaAttentionBlock a layer.  norm_pre, norm_post ("none":
    a plain gated residual add) and gate as for ResidualNorm.  ``ckpt`` holds
    the normalised x and y of every layer as 8-bit checkpoints; the one of x
    also serves the layer's dW_q and dW_kv_a, so neither x nor h is held in
    the I/O type.  Gate logits are given as tensors and their gradients given
    back; a gate that is computed from x or h on the way needs ResidualNorm in
    the caller's own loop."""

    def __init__(self, blocks, d_model: int, *, norm_pre: str = "rms", norm_post: str = "none",
                 gate: str = "none", ckpt: bool = False, io_dtype: str = "bf16", eps: float = 1e-5,
                 device="cuda"):
        if not blocks:
            raise ValueError("at least one block")
        kw = dict(norm_pre=norm_pre, norm_post=norm_post, gate=gate, ckpt=ckpt, io_dtype=io_dtype,
                  eps=eps, device=device)
        self.blocks = list(blocks)
        self.first = ResidualNorm(d_model, post=False, **kw)
        self.between = ResidualNorm(d_model, **kw)
        self.last = ResidualNorm(d_model, pre=False, **kw)
        self._saved = None

    def forward(self, x, layers, cos, sin):
        """``layers``: per block a dict of w_q, w_kva, gamma, w_kvb, w_o (see
        LagaAttentionBlock.forward), gamma_pre [d_model] and alpha [1] fp32,
        and, where they apply, gamma_post [d_model] fp32 and gate logits [B,
        S_r, d_model or 1].  Returns x behind the last block."""
        if len(layers) != len(self.blocks):
            raise ValueError(f"{len(layers)} layers for {len(self.blocks)} blocks")
        r = self.first.forward(x, gamma_pre=layers[0]["gamma_pre"])
        kept = [r.saved]                      # of the norm in front of block l
        behind = []                           # of the residual half behind block l
        for i, (block, w) in enumerate(zip(self.blocks, layers)):
            in_bits = self.first.ckpt
            y = block.forward(r.h, w["w_q"], w["w_kva"], w["gamma"], w["w_kvb"], w["w_o"], cos, sin,
                              kept=kept[i].x if in_bits else None,
                              kept_gain=w["gamma_pre"] if in_bits else None)
            ends = i + 1 == len(layers)
            step = self.last if ends else self.between
            r = step.forward(r.x, y, gate=w.get("gate"), alpha=w["alpha"],
                             gamma_post=w.get("gamma_post"),
                             gamma_pre=None if ends else layers[i + 1]["gamma_pre"])
            behind.append(r.saved)
            kept.append(r.saved)
        self._saved = (kept[0], behind)
        return r.x

    def backward(self, dx):
        """dx of the stream behind the last block.  Returns (dx in front of the
        first block, per block a dict: the block's weight gradients, and
        dgamma_pre, dalpha, dgamma_post and dgate where they apply; those of
        the shared parameters summed over the ranks)."""
        first, behind = self._saved
        grads = [None] * len(self.blocks)
        g = self.last.backward(behind[-1], dx)
        for i in reversed(range(len(self.blocks))):
            block = self.blocks[i]
            out = {k: block._all_reduce(v, "all_reduce_" + k) for k, v in
                   (("dalpha", g.dalpha), ("dgamma_post", g.dgamma_post)) if v is not None}
            if g.dgate is not None:
                out["dgate"] = g.dgate
            out.update(block.backward(g.dy))
            dh = out.pop("dh")
            g = (self.between.backward(behind[i - 1], g.dx, dh) if i else
                 self.first.backward(first, g.dx, dh))
            out["dgamma_pre"] = block._all_reduce(g.dgamma_pre, "all_reduce_dgamma_pre")
            grads[i] = out
        return g.dx, grads
