"""Rows to experts and back, their gated activation, and the routed block.

    h_t -> rows of its experts (spread8) -> [g | u] = row W_in[e] (linear8)
        -> a = silu(g) u in 8 bits (swiglu8) -> a W_out[e] (linear8)
        -> y_t = sum_j weight_tj row_tj (combine)

:class:`RoutedExperts` runs all of it, forward and backward, as a block of
``LagaResidualStack``.
"""

from __future__ import annotations

import torch

from . import _lib
from .api import _TORCH_DT
from .checkpoint import (IO_NAME, Checkpoint8, empty_checkpoint, need, on_stream, pack8, rows_of,
                         weight_grad8)
from .linear8 import Weight8, linear8, linear8_dx, pack_weight8
from .routing import Router


def _matrix(t, name, device=None, shape=None):
    """Check a bf16 or fp32 tensor: its address, rows and width."""
    if not isinstance(t, torch.Tensor) or t.dtype not in IO_NAME:
        raise TypeError(f"{name} must be a bf16 or fp32 tensor")
    rows, d = rows_of(t.shape)
    if not 1 <= d <= 16384:
        raise ValueError(f"{name}: {d} channels, 1 .. 16384")
    return need(t, name, t.dtype, device, shape), rows, d


def spread8(x: Checkpoint8, routes, *, stream=None) -> Checkpoint8:
    """x's rows (one per token) as the experts' rows; rows of no pair are zero."""
    if not isinstance(x, Checkpoint8):
        raise TypeError("spread8 takes a Checkpoint8")
    if x.rows != routes.tokens:
        raise ValueError(f"spread8: {x.rows} rows for {routes.tokens} tokens")
    _, pair, _, end = routes.check(x.device)
    with on_stream(x.device, stream, x.data, routes.pair, routes.start) as st:
        out = empty_checkpoint((routes.rows, x.d), x.device)
        _lib.spread8(routes.rows, x.rows, routes.top_k, x.d, x.data.data_ptr(), pair, end,
                     out.data.data_ptr(), st)
    return out


def _weight(routes, weighted, device):
    if not weighted:
        return 0
    return need(routes.weight, "routes.weight", torch.float32, device, tuple(routes.row.shape))


def combine(y: torch.Tensor, routes, *, weighted: bool = True, stream=None) -> torch.Tensor:
    """sum_j weight_tj y[row_tj] [tokens, d] of the experts' rows y [rows, d];
    ``weighted=False`` takes weights of 1 (the gradient of spread8).  A token
    that a NaN left without an expert (a row of -2) comes out as NaN."""
    p, rows, d = _matrix(y, "y")
    if rows != routes.rows:
        raise ValueError(f"y has {rows} rows, the routes {routes.rows}")
    dev, T = y.device, routes.tokens
    row = routes.check(dev)[0]
    w = _weight(routes, weighted, dev)
    with on_stream(dev, stream, y, routes.weight, routes.row) as st:
        out = torch.empty(T, d, dtype=y.dtype, device=dev)
        _lib.combine_fwd(T, routes.top_k, rows, d, IO_NAME[y.dtype], p, w, row, out.data_ptr(), st)
    return out


def combine_grad(dout: torch.Tensor, routes, *, y=None, weighted: bool = True, stream=None):
    """(dy [rows, d], dweight [tokens, k] fp32) of combine for dout [tokens, d];
    dweight needs the forward's y, and is None without it.  Rows of no pair
    get zeros."""
    p, T, d = _matrix(dout, "dout")
    if T != routes.tokens:
        raise ValueError(f"dout has {T} rows, the routes {routes.tokens} tokens")
    dev = dout.device
    row, pair, _, end = routes.check(dev)
    py = 0 if y is None else need(y, "y", dout.dtype, dev, (routes.rows, d))
    w = _weight(routes, weighted, dev)
    with on_stream(dev, stream, dout, y, routes.weight, routes.row, routes.pair,
                   routes.start) as st:
        dy = torch.empty(routes.rows, d, dtype=dout.dtype, device=dev)
        dweight = None
        if y is not None:
            dweight = torch.empty(T, routes.top_k, dtype=torch.float32, device=dev)
        _lib.combine_bwd(T, routes.top_k, routes.rows, d, IO_NAME[dout.dtype], p, py, w, row, pair,
                         end, dy.data_ptr(), 0 if y is None else dweight.data_ptr(), st)
    return dy, dweight


def _gated(gu, routes):
    p, rows, d = _matrix_2f(gu)
    if routes is None:
        return p, rows, d, 0
    if rows != routes.rows:
        raise ValueError(f"gu has {rows} rows, the routes {routes.rows}")
    return p, rows, d, routes.check(gu.device)[3]


def _matrix_2f(gu):
    if not isinstance(gu, torch.Tensor) or gu.dtype not in IO_NAME:
        raise TypeError("gu must be a bf16 or fp32 tensor")
    rows, d = rows_of(gu.shape)
    if d % 2 or not 2 <= d <= 32768:
        raise ValueError(f"gu: [g | u] of {d} channels, an even number up to 32768")
    return need(gu, "gu", gu.dtype), rows, d // 2


def swiglu8(gu: torch.Tensor, *, routes=None, stream=None) -> Checkpoint8:
    """silu(g) u of gu [..., 2 f] = [g | u] in 8 bits; with ``routes``, of the
    rows in use."""
    p, rows, f, end = _gated(gu, routes)
    with on_stream(gu.device, stream, gu, routes and routes.start) as st:
        ck = empty_checkpoint((*gu.shape[:-1], f), gu.device)
        _lib.swiglu_fwd(rows, f, IO_NAME[gu.dtype], p, end, ck.data.data_ptr(), st)
    return ck


def swiglu8_grad(gu: torch.Tensor, da: torch.Tensor, *, routes=None, stream=None) -> torch.Tensor:
    """Gradient [..., 2 f] of gu for da [..., f]."""
    p, rows, f, end = _gated(gu, routes)
    pa = need(da, "da", gu.dtype, gu.device, (*gu.shape[:-1], f))
    with on_stream(gu.device, stream, gu, da, routes and routes.start) as st:
        dgu = torch.empty_like(gu)
        _lib.swiglu_bwd(rows, f, IO_NAME[gu.dtype], p, pa, end, dgu.data_ptr(), st)
    return dgu


class RoutedExperts:
    """Feed-forward experts behind a router, all on this device:

        logits = h W_router (fp32),  routes = Router(logits, bias),
        y_t = sum_j weight_tj W_out[e]^T (silu(g) u),  [g | u] = W_in[e]^T h_t

    with the experts' products in 8 bits.  Options of the router as for
    Router (score, groups, top_groups, renormalise, scale).  What is held
    between the passes: h in 8 bits (or ``kept``), [g | u], logits and routes;
    the activation and the experts' outputs are computed again."""

    distributed = False

    def __init__(self, n_experts: int, top_k: int, *, io_dtype: str = "bf16", device="cuda",
                 **router):
        for k in ("shard", "align"):
            if k in router:
                raise ValueError(f"RoutedExperts sets {k} itself")
        if io_dtype not in _TORCH_DT:
            raise ValueError(f"io_dtype={io_dtype!r}: one of {', '.join(_TORCH_DT)}")
        self.router = Router(n_experts, top_k, device=device, **router)
        self.dtype = _TORCH_DT[io_dtype]
        self._saved = None

    def forward(self, h, w_router, w_in, w_out, *, bias=None, kept=None, kept_gain=None):
        """h [..., d]; w_router [d, n_experts] fp32; w_in [n_experts, d, 2 f] and
        w_out [n_experts, f, d], in the I/O dtype or as Weight8; bias
        [n_experts] fp32 or None.  Returns y [..., d].  ``kept`` and
        ``kept_gain`` as for LagaAttentionBlock.forward."""
        if h.dtype != self.dtype:
            raise ValueError(f"h: dtype {h.dtype} != {self.dtype}")
        rows, d = rows_of(h.shape)
        if kept is None:
            if kept_gain is not None:
                raise ValueError("kept_gain without kept: h is held as given")
        elif not isinstance(kept, Checkpoint8):
            raise TypeError("kept must be a Checkpoint8")
        elif (kept.rows, kept.d) != (rows, d):
            raise ValueError(f"kept: a checkpoint of {kept.rows} rows of {kept.d}, expected "
                             f"{rows} of {d}")
        w_in, w_out = (w if isinstance(w, Weight8) else pack_weight8(w.contiguous())
                       for w in (w_in, w_out))
        h_flat = h.reshape(rows, d).contiguous()
        logits = h_flat.float() @ w_router
        routes = self.router.forward(logits, bias)
        h8 = pack8(h_flat)
        gu = linear8(spread8(h8, routes), w_in, routes=routes, dtype=self.dtype)
        y = self._outputs(swiglu8(gu, routes=routes), w_out, routes)
        self._saved = (h8 if kept is None else kept, kept_gain, logits, routes, gu, w_router, w_in,
                       w_out, h.shape)
        return combine(y, routes).reshape(h.shape)

    def _outputs(self, a8, w_out, routes):
        return linear8(a8, w_out, routes=routes, dtype=self.dtype)

    def _all_reduce(self, t, what):
        return t

    def backward(self, dy):
        """dy [..., d].  Returns a dict: dh [..., d]; dw_router [d, n_experts],
        dw_in and dw_out of their weights' shapes, fp32."""
        kept, gain, logits, routes, gu, w_router, w_in, w_out, shape = self._saved
        dy_flat = dy.reshape(-1, shape[-1]).contiguous()
        a8 = swiglu8(gu, routes=routes)
        d_rows, dweight = combine_grad(dy_flat, routes, y=self._outputs(a8, w_out, routes))
        dw_out = weight_grad8(a8, d_rows, routes=routes)
        da = linear8_dx(pack8(d_rows, routes=routes), w_out, routes=routes, dtype=self.dtype)
        dgu = swiglu8_grad(gu, da, routes=routes)
        dw_in = weight_grad8(spread8(kept, routes), dgu, gain, routes=routes)
        dx = linear8_dx(pack8(dgu, routes=routes), w_in, routes=routes, dtype=self.dtype)
        dlogits = self.router.backward(logits, routes, dweight)
        dh = combine(dx, routes, weighted=False) + (dlogits @ w_router.t()).to(self.dtype)
        return dict(dh=dh.reshape(shape), dw_router=weight_grad8(kept, dlogits, gain), dw_in=dw_in,
                    dw_out=dw_out)
