"""Linear maps of 8-bit operands.

A :class:`Weight8` holds W [k, n], or one per expert, as e4m3 codes with one
power-of-two scale per block of 128 x 128, in the two orders that a product
with it and with its transpose read.  :func:`linear8` multiplies the codes of
a :class:`Checkpoint8` with it, :func:`linear8_dx` is the gradient of its
input; the weight's is :func:`weight_grad8`'s.  With ``routes`` every row
takes its expert's weight.
"""

from __future__ import annotations

import torch

from . import _lib
from .checkpoint import IO_NAME, Checkpoint8, need, on_stream


class Weight8:
    """A weight in 8 bits: ``shape`` (k, n) or (experts, k, n); ``fwd`` uint8
    [experts n, row bytes of k], the rows of W^T; ``bwd`` uint8 [experts k, row
    bytes of n], the rows of W, or None (no input gradient)."""

    __slots__ = ("shape", "fwd", "bwd")

    def __init__(self, shape, fwd: torch.Tensor, bwd: torch.Tensor | None = None):
        shape = tuple(shape)
        if len(shape) not in (2, 3):
            raise ValueError(f"a weight of shape {shape}: [k, n] or [experts, k, n]")
        k, n = shape[-2:]
        if not (1 <= k <= 16384 and 1 <= n <= 16384):
            raise ValueError(f"a weight of {k} x {n}: 1 .. 16384 each")
        if len(shape) == 3 and not 1 <= shape[0] <= 1024:
            raise ValueError(f"{shape[0]} experts: 1 .. 1024")
        e = shape[0] if len(shape) == 3 else 1
        need(fwd, "fwd", torch.uint8, shape=(e * n, _lib.ckpt_row_bytes(k)))
        if bwd is not None:
            need(bwd, "bwd", torch.uint8, fwd.device, (e * k, _lib.ckpt_row_bytes(n)))
        self.shape, self.fwd, self.bwd = shape, fwd, bwd

    @property
    def experts(self):
        return self.shape[0] if len(self.shape) == 3 else 0

    @property
    def device(self):
        return self.fwd.device

    @property
    def nbytes(self):
        return self.fwd.numel() + (0 if self.bwd is None else self.bwd.numel())

    def unpack(self, dtype=torch.bfloat16, stream=None):
        """The values, [*shape], in bf16 or fp32 (both hold them exactly)."""
        *lead, k, n = self.shape
        if self.bwd is not None:
            return Checkpoint8(self.bwd, n, self.shape).unpack(dtype, stream)
        with on_stream(self.device, stream, self.fwd):
            v = Checkpoint8(self.fwd, k, (*lead, n, k)).unpack(dtype, stream)
            return v.transpose(-1, -2).contiguous()


def pack_weight8(w: torch.Tensor, *, backward: bool = True, stream=None) -> Weight8:
    """w [k, n] or [experts, k, n] (bf16 or fp32, contiguous, on a CUDA device)
    in 8 bits; ``backward=False`` leaves out what the input gradient reads."""
    if not isinstance(w, torch.Tensor) or w.dtype not in IO_NAME:
        raise TypeError("pack_weight8 takes a bf16 or fp32 tensor")
    if w.dim() not in (2, 3):
        raise ValueError(f"w: shape {tuple(w.shape)}, expected [k, n] or [experts, k, n]")
    p = need(w, "w", w.dtype)
    e, (k, n) = w.shape[0] if w.dim() == 3 else 1, w.shape[-2:]
    pk, pn = _lib.ckpt_row_bytes(k), _lib.ckpt_row_bytes(n)
    if not pk or not pn or not 1 <= e <= 1024:
        raise ValueError(f"w: shape {tuple(w.shape)}: widths of 1 .. 16384, 1 .. 1024 experts")
    with on_stream(w.device, stream, w) as st:
        fwd = torch.empty(e * n, pk, dtype=torch.uint8, device=w.device)
        bwd = torch.empty(e * k, pn, dtype=torch.uint8, device=w.device) if backward else None
        _lib.weight_pack(e, k, n, IO_NAME[w.dtype], p, fwd.data_ptr(),
                         bwd.data_ptr() if backward else 0, st)
    return Weight8(w.shape, fwd, bwd)


def _product(x, w, routes, dtype, stream, matrix, k, n, what):
    if not isinstance(x, Checkpoint8):
        raise TypeError(f"{what} takes a Checkpoint8")
    if dtype not in IO_NAME:
        raise ValueError(f"{what} into {dtype}: bf16 or fp32")
    if x.d != k:
        raise ValueError(f"{what}: rows of {x.d} channels, expected {k}")
    dev = x.device
    if w.device != dev:
        raise ValueError(f"{what}: the weight on {w.device}, expected {dev}")
    if (routes is None) != (w.experts == 0):
        raise ValueError(f"{what}: routes go with the weights of experts, and these with routes")
    start = pair = 0
    lead = x.shape[:-1]
    if routes is not None:
        if routes.experts != w.experts:
            raise ValueError(f"{what}: routes to {routes.experts} experts, weights of {w.experts}")
        pair, start = routes.check(dev)[1:3]
        if routes.align == 1:            # every row in use has a pair
            pair = 0
        if x.rows != routes.rows:
            raise ValueError(f"{what}: {x.rows} rows, expected the routes' {routes.rows}")
    with on_stream(dev, stream, x.data, matrix, *(routes[3:5] if routes is not None else ())) as st:
        y = torch.empty(*lead, n, dtype=dtype, device=dev)
        nb = _lib.mm8_workspace_bytes(x.rows, k, n, w.experts, IO_NAME[dtype])
        ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
        _lib.mm8(x.rows, k, n, w.experts, IO_NAME[dtype], x.data.data_ptr(), matrix.data_ptr(),
                 start, pair, y.data_ptr(), ws.data_ptr() if nb else 0, nb, st)
    return y


def linear8(x: Checkpoint8, w: Weight8, *, routes=None, dtype=torch.bfloat16, stream=None):
    """x W [..., n] in ``dtype`` (bf16 or fp32); with ``routes`` (a Routes; x
    has its rows, as :func:`spread8` makes them) row by row with its
    expert's W; rows of no pair are zero."""
    if not isinstance(w, Weight8):
        raise TypeError("linear8 takes a Weight8")
    k, n = w.shape[-2:]
    return _product(x, w, routes, dtype, stream, w.fwd, k, n, "linear8")


def linear8_dx(dy: Checkpoint8, w: Weight8, *, routes=None, dtype=torch.bfloat16, stream=None):
    """dy W^T [..., k]: the gradient of linear8's x for an output gradient in
    8 bits."""
    if not isinstance(w, Weight8):
        raise TypeError("linear8_dx takes a Weight8")
    if w.bwd is None:
        raise ValueError("linear8_dx: the weight was packed without its backward order")
    k, n = w.shape[-2:]
    return _product(dy, w, routes, dtype, stream, w.bwd, n, k, "linear8_dx")
