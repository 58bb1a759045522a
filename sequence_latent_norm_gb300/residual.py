"""The residual stream around a block.

    x' = x + alpha * sigmoid(gate) * N_post(y) * gamma_post     (post)
    h  = N_pre(x') * gamma_pre                                  (pre)

y is a block's output, h the next block's input; a step between two blocks
does both, the one in front of the first block only ``pre``, the one behind
the last only ``post``.  ``ckpt=True`` keeps the normalised y and x' for the
backward as 8-bit checkpoints instead of y and x' themselves; the
checkpoint of x' is also the activation of the weight gradients behind h
(``weight_grad8(saved.x, dq, gamma=gamma_pre)``).
"""

from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import _lib
from .api import _TORCH_DT
from .checkpoint import Checkpoint8, empty_checkpoint, need, on_16, on_stream, rows_of


class ResidualSaved(NamedTuple):
    """What the backward reads.  y and x: the forward's y and x' (x without
    ``post``), or their checkpoints after the norm; stat_*: [rows, 2] fp32
    mean and 1/std; the rest as given to the forward."""

    y: torch.Tensor | Checkpoint8 | None = None
    x: torch.Tensor | Checkpoint8 | None = None
    stat_post: torch.Tensor | None = None
    stat_pre: torch.Tensor | None = None
    gate: torch.Tensor | None = None
    alpha: torch.Tensor | None = None
    gamma_post: torch.Tensor | None = None
    gamma_pre: torch.Tensor | None = None


class ResidualOut(NamedTuple):
    x: torch.Tensor                # x' (x itself without ``post``)
    h: torch.Tensor | None
    saved: ResidualSaved


class ResidualGrads(NamedTuple):
    """Gradients of x, y, the gate logits, alpha and the gains (None: off)."""

    dx: torch.Tensor
    dy: torch.Tensor | None = None
    dgate: torch.Tensor | None = None
    dalpha: torch.Tensor | None = None
    dgamma_post: torch.Tensor | None = None
    dgamma_pre: torch.Tensor | None = None


class ResidualNorm:
    """One place of the residual stream, for rows of d channels.

    norm_post "layer", "rms" or "none" (a plain gated residual add);
    norm_pre "layer" or "rms"; gate "none", "token" (logits [..., 1]) or
    "full" (logits [..., d]); io_dtype "bf16" or "fp32" of x, y, gate, h and
    their gradients.  Gains and alpha ([1]) are fp32 and may start anywhere (one
    layer's entry of a tensor of all layers'); the other tensors start on a
    16-byte boundary.  What is off is ignored where it is given.  A call takes
    any number of rows and keeps none of its data in the object."""

    def __init__(self, d: int, *, post: bool = True, pre: bool = True, norm_post: str = "rms",
                 norm_pre: str = "rms", gate: str = "none", ckpt: bool = False,
                 io_dtype: str = "bf16", eps: float = 1e-5, device="cuda"):
        for what, v, known in (("norm_post", norm_post, _lib.POST_NORMS),
                               ("norm_pre", norm_pre, _lib.NORMS), ("gate", gate, _lib.GATES),
                               ("io_dtype", io_dtype, _lib.DTYPES)):
            if v not in known:
                raise ValueError(f"{what}={v!r}: one of {', '.join(known)}")
        self.d, self.post, self.pre, self.ckpt = d, bool(post), bool(pre), bool(ckpt)
        self.gate = gate if post else "none"
        self.gain = self.post and norm_post != "none"
        self.dtype = _TORCH_DT[io_dtype]
        self._dims = dict(post=post, pre=pre, norm_post=norm_post, norm_pre=norm_pre, eps=eps,
                          gate=gate, ckpt=ckpt, io_dtype=io_dtype)
        if not (self.post or self.pre):
            raise ValueError("post or pre, or both")
        if not 1 <= d <= 16384:
            raise ValueError(f"{d} channels: 1 .. 16384")
        if not (0.0 < eps < math.inf):
            raise ValueError(f"eps={eps}: positive and finite")
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device {self.device}: a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._last = None

    def _c_dims(self, rows):
        """The C dims for so many rows and their backward's scratch bytes; the
        last ones are kept (and never changed), since calls mostly repeat."""
        last = self._last
        if last is None or last[0] != rows:
            dims = _lib.make_res_dims(rows, self.d, **self._dims)
            last = self._last = (rows, dims, _lib.res_workspace_bytes(dims))
        return last[1], last[2]

    @staticmethod
    def _shape(t, name):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        return rows_of(t.shape)[0], tuple(t.shape)

    def _io(self, t, name, shape):
        return need(t, name, self.dtype, self.device, shape)

    def _f32(self, t, name, shape):
        return need(t, name, torch.float32, self.device, shape)

    def _used(self, gate, alpha, gamma_post, gamma_pre):
        """The gate logits, alpha and the gains, None where they are off."""
        return (gate if self.gate != "none" else None, alpha if self.post else None,
                gamma_post if self.gain else None, gamma_pre if self.pre else None)

    def _params(self, shape, gate, alpha, gamma_post, gamma_pre):
        """Addresses of the gate logits, alpha and the gains (0: off)."""
        d = (self.d,)
        gate_shape = shape if self.gate == "full" else (*shape[:-1], 1)
        return (self._io(gate, "gate", gate_shape) if self.gate != "none" else 0,
                self._f32(alpha, "alpha", (1,)) if self.post else 0,
                self._f32(gamma_post, "gamma_post", d) if self.gain else 0,
                self._f32(gamma_pre, "gamma_pre", d) if self.pre else 0)

    @staticmethod
    def _aligned(params, used):
        """The addresses again, of copies of alpha and the gains where these start
        off a 16-byte boundary; and the copies, to be held up to the launch."""
        moved = [on_16(t) for t in used[1:]]
        return (params[0], *(0 if t is None else t.data_ptr() for t in moved)), moved

    def forward(self, x, y=None, *, gate=None, alpha=None, gamma_post=None, gamma_pre=None,
                stream=None) -> ResidualOut:
        """x, y [..., d]; see the class and the module for the rest."""
        rows, shape = self._shape(x, "x")
        full = (*shape[:-1], self.d)
        if not self.post:
            y = None
        used = self._used(gate, alpha, gamma_post, gamma_pre)
        px = self._io(x, "x", full)
        py = self._io(y, "y", full) if self.post else 0
        params = self._params(full, *used)
        dev = self.device
        with on_stream(dev, stream, x, y, *used) as st:
            x_out = torch.empty_like(x) if self.post else x
            h = torch.empty_like(x) if self.pre else None
            ck_y = empty_checkpoint(full, dev) if self.ckpt and self.post else None
            ck_x = empty_checkpoint(full, dev) if self.ckpt and self.pre else None
            s_post = torch.empty(rows, 2, dtype=torch.float32, device=dev) if self.post else None
            s_pre = torch.empty(rows, 2, dtype=torch.float32, device=dev) if self.pre else None
            if (params[1] | params[2] | params[3]) % 16:
                params, moved = self._aligned(params, used)
            _lib.res_fwd(self._c_dims(rows)[0], px, py, *params,
                         x_out.data_ptr() if self.post else 0, h.data_ptr() if self.pre else 0,
                         ck_y.data.data_ptr() if ck_y else 0, ck_x.data.data_ptr() if ck_x else 0,
                         s_post.data_ptr() if self.post else 0,
                         s_pre.data_ptr() if self.pre else 0, st)
        saved = ResidualSaved(ck_y or y, (ck_x or x_out) if self.pre else None, s_post, s_pre, *used)
        return ResidualOut(x_out, h, saved)

    def _kept(self, t, name, shape, rows):
        if not self.ckpt:
            return self._io(t, name, shape)
        if not isinstance(t, Checkpoint8):
            raise TypeError(f"{name} must be a Checkpoint8")
        if t.d != self.d or t.rows != rows:
            raise ValueError(f"{name}: a checkpoint of {t.rows} rows of {t.d}, expected {rows} "
                             f"of {self.d}")
        return need(t.data, name, torch.uint8, self.device)

    def backward(self, saved: ResidualSaved, dx_out=None, dh=None, *, stream=None) -> ResidualGrads:
        """Gradients for dx_out [..., d] of x' (None with ``pre``: x' has no
        other use) and dh [..., d] of h.  Without ``pre``, dx is dx_out."""
        lead = dh if self.pre else dx_out
        rows, shape = self._shape(lead, "dh" if self.pre else "dx_out")
        full = (*shape[:-1], self.d)
        p_dh = self._io(dh, "dh", full) if self.pre else 0
        p_dx = 0 if dx_out is None and self.pre else self._io(dx_out, "dx_out", full)
        k_y = self._kept(saved.y, "saved.y", full, rows) if self.post else 0
        k_x = self._kept(saved.x, "saved.x", full, rows) if self.pre else 0
        s_post = self._f32(saved.stat_post, "saved.stat_post", (rows, 2)) if self.post else 0
        s_pre = self._f32(saved.stat_pre, "saved.stat_pre", (rows, 2)) if self.pre else 0
        used = self._used(saved.gate, saved.alpha, saved.gamma_post, saved.gamma_pre)
        params = self._params(full, *used)
        dev, (dims, nb) = self.device, self._c_dims(rows)
        read = []
        if stream is not None:       # what on_stream records there
            read = [dx_out, *used]
            if self.post:
                read += [saved.y.data, saved.stat_post]
            if self.pre:
                read += [dh, saved.x.data, saved.stat_pre]
        with on_stream(dev, stream, *read) as st:
            def f32(on, n):
                return torch.empty(n, dtype=torch.float32, device=dev) if on else None

            dx = torch.empty_like(dh) if self.pre else dx_out
            dy = torch.empty_like(lead) if self.post else None
            dgate = torch.empty_like(saved.gate) if self.gate != "none" else None
            dalpha, dg_post = f32(self.post, 1), f32(self.gain, self.d)
            dg_pre = f32(self.pre, self.d)
            ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
            if (params[1] | params[2] | params[3]) % 16:
                params, moved = self._aligned(params, used)

            def ptr(t):
                return 0 if t is None else t.data_ptr()

            _lib.res_bwd(dims, p_dx, p_dh, k_y, k_x, s_post, s_pre, *params,
                         ptr(dx) if self.pre else 0, ptr(dy), ptr(dgate), ptr(dalpha),
                         ptr(dg_post), ptr(dg_pre), ptr(ws), nb, st)
        return ResidualGrads(dx, dy, dgate, dalpha, dg_post, dg_pre)
