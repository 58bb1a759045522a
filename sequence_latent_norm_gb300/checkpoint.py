"""Activations kept in 8 bits between the passes.

A :class:`Checkpoint8` holds a [..., d] activation as e4m3 codes with one
power-of-two scale per 128 channels of a row (the byte layout is that of
``include/laga.h``): about one byte per element instead of two, every value
exact in bf16.  :func:`pack8` makes one, ``unpack`` reads it back and
:func:`weight_grad8` takes a weight gradient straight from the codes.

``stream`` (a torch.cuda.Stream; None: the current one) is where a call runs
and what its outputs' memory belongs to.  The caller orders it behind the work
that makes the inputs, and other streams behind the call.  With a stream given,
the inputs may be dropped as soon as the call returns, whichever stream their
memory belongs to; without one that holds for memory of the current stream, as
for torch's own operators.
"""

from __future__ import annotations

import math

import torch

from . import _lib

IO_NAME = {torch.bfloat16: "bf16", torch.float32: "fp32"}


class on_stream:
    """Run on ``device`` and ``stream`` (None: the device's current stream);
    entering gives the stream's handle.  What is allocated inside belongs to
    that stream, so its memory is reused in that stream's order.  ``inputs``
    (tensors or None) are read there: with a stream of the caller's they are
    recorded on it, so that the caller may drop them behind the call."""

    __slots__ = ("device", "stream", "inner", "inputs")

    def __init__(self, device, stream, *inputs):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream on {stream.device}, tensors on {device}")
        self.device, self.stream, self.inner, self.inputs = device, stream, None, inputs

    def __enter__(self):
        if self.stream is not None:
            for t in self.inputs:
                if t is not None:
                    t.record_stream(self.stream)
            self.inner = torch.cuda.stream(self.stream)   # its device, too
        elif torch.cuda.current_device() != self.device.index:
            self.inner = torch.cuda.device(self.device)
        if self.inner is not None:
            self.inner.__enter__()
        return (self.stream or torch.cuda.current_stream(self.device)).cuda_stream

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def need(t, name, dtype, device=None, shape=None):
    """Check one CUDA tensor argument and return its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: on {t.device}, expected {device if device else 'a CUDA device'}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def on_16(t):
    """``t``, or a copy of it (of the current stream) if it starts off a 16-byte
    boundary, as one layer's entry of a parameter tensor of all layers may."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.detach().clone()


def rows_of(shape):
    """Rows and width of a [..., d] tensor seen as a matrix."""
    if len(shape) < 1:
        raise ValueError("an activation has at least one dimension, its channels")
    rows = math.prod(shape[:-1])
    if rows > 2 ** 31 - 1:
        raise ValueError(f"{rows} rows: at most 2^31 - 1")
    return rows, shape[-1]


class Checkpoint8:
    """One activation in 8 bits: ``data``, uint8 [rows, row bytes], contiguous
    on a CUDA device, standing for values of shape ``shape`` (default [rows,
    d]; its last dimension is d)."""

    __slots__ = ("data", "d", "shape")

    def __init__(self, data: torch.Tensor, d: int, shape=None):
        row_bytes = _lib.ckpt_row_bytes(d)
        if row_bytes == 0:
            raise ValueError(f"no checkpoint of {d} channels (1 .. 16384)")
        shape = (data.shape[0], d) if shape is None else tuple(shape)
        rows, last = rows_of(shape)
        need(data, "checkpoint data", torch.uint8, shape=(rows, row_bytes))
        if last != d:
            raise ValueError(f"shape {shape} does not end in {d} channels")
        self.data, self.d, self.shape = data, d, shape

    @property
    def rows(self):
        return self.data.shape[0]

    @property
    def device(self):
        return self.data.device

    @property
    def nbytes(self):
        return self.data.numel()

    def unpack(self, dtype=torch.bfloat16, stream=None):
        """The values, [*shape], in bf16 or fp32 (both hold them exactly)."""
        if dtype not in IO_NAME:
            raise ValueError(f"unpack to {dtype}: bf16 or fp32")
        with on_stream(self.device, stream, self.data) as st:
            x = torch.empty(self.shape, dtype=dtype, device=self.device)
            _lib.ckpt_unpack(self.rows, self.d, IO_NAME[dtype], self.data.data_ptr(),
                             x.data_ptr(), st)
        return x


def empty_checkpoint(shape, device):
    """An unwritten checkpoint for values of ``shape``."""
    rows, d = rows_of(shape)
    data = torch.empty(rows, _lib.ckpt_row_bytes(d), dtype=torch.uint8, device=device)
    return Checkpoint8(data, d, shape)


def pack8(x: torch.Tensor, stream=None) -> Checkpoint8:
    """x [..., d] (bf16 or fp32, contiguous, on a CUDA device) in 8 bits."""
    if not isinstance(x, torch.Tensor) or x.dtype not in IO_NAME:
        raise TypeError("pack8 takes a bf16 or fp32 tensor")
    ptr = need(x, "x", x.dtype)
    rows, d = rows_of(x.shape)
    with on_stream(x.device, stream, x) as st:
        ck = empty_checkpoint(x.shape, x.device)
        _lib.ckpt_pack(rows, d, IO_NAME[x.dtype], ptr, ck.data.data_ptr(), st)
    return ck


def weight_grad8(ck: Checkpoint8, dy: torch.Tensor, gamma=None, stream=None) -> torch.Tensor:
    """dW [d, n] fp32 = diag(gamma) v^T dy of the checkpointed activation v
    [rows, d] and dy [..., n] (bf16 or fp32, as many rows): the gradient of W
    in (v gamma) W.  gamma [d] fp32 (it may start anywhere), or None for 1."""
    if not isinstance(ck, Checkpoint8):
        raise TypeError("weight_grad8 takes a Checkpoint8")
    if not isinstance(dy, torch.Tensor) or dy.dtype not in IO_NAME:
        raise TypeError("dy must be a bf16 or fp32 tensor")
    rows, n = rows_of(dy.shape)
    if rows != ck.rows:
        raise ValueError(f"dy has {rows} rows, the checkpoint {ck.rows}")
    dev, name = ck.device, IO_NAME[dy.dtype]
    dy_ptr = need(dy, "dy", dy.dtype, dev)
    g_ptr = 0 if gamma is None else need(gamma, "gamma", torch.float32, dev, (ck.d,))
    with on_stream(dev, stream, ck.data, dy, gamma) as st:
        dw = torch.empty(ck.d, n, dtype=torch.float32, device=dev)
        nb = _lib.ckpt_dw_workspace_bytes(rows, ck.d, n, name)
        ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
        if g_ptr % 16:
            gamma = on_16(gamma)
            g_ptr = gamma.data_ptr()
        _lib.ckpt_dw(rows, ck.d, n, name, ck.data.data_ptr(), dy_ptr, g_ptr, dw.data_ptr(),
                     ws.data_ptr() if nb else 0, nb, st)
    return dw
