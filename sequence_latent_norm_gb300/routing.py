"""Routing of tokens to experts.

    s = sigmoid(logits) or softmax(logits),   c = s + bias  (it chooses only)
    groups with the best sums of their two best c, of these the top_k best c
    weight = scale * s / (sum of the chosen s + 1e-20)  (or scale * s)

and the order in which the experts take their rows: the (token, choice) pairs
sorted by expert.  Calls order their work on ``stream`` as those of
``checkpoint.py`` do.
"""

from __future__ import annotations

import math
from typing import NamedTuple

import torch

from . import _lib
from .api import _TORCH_DT
from .checkpoint import need, on_16, on_stream


class Routes(NamedTuple):
    """A batch's choices and the rows that experts take them in.

    expert [T, k] int32 (best first; -1: no expert was on); weight [T, k]
    fp32 (0 there; NaN throughout a token that holds a NaN); row [T, k] int32:
    the pair's row, -1 where it has none (on this rank), -2 where a token with
    a NaN has no expert (combine makes that token NaN); pair [R] int32: the
    row's pair t k + j, -1 where it has none; start [E + 1] int32: expert e (of
    this rank's) takes the rows start[e] .. start[e + 1] - 1, of which the ones
    behind its pairs belong to none.  start[e] are multiples of ``align``.  R
    rows are the most that a batch can need; buffers of rows have that many, and
    what is behind row start[E] - 1 is never written or read."""

    expert: torch.Tensor
    weight: torch.Tensor
    row: torch.Tensor
    pair: torch.Tensor
    start: torch.Tensor
    align: int

    @property
    def tokens(self):
        return self.row.shape[0]

    @property
    def top_k(self):
        return self.row.shape[1]

    @property
    def rows(self):
        return self.pair.shape[0]

    @property
    def experts(self):
        return self.start.shape[0] - 1

    def check(self, device):
        """Check the row order's tensors; addresses of row, pair, start, and of
        start's last entry."""
        T, k = self.row.shape
        i32 = torch.int32
        p = [need(self.row, "routes.row", i32, device, (T, k)),
             need(self.pair, "routes.pair", i32, device, (self.rows,)),
             need(self.start, "routes.start", i32, device, (self.experts + 1,))]
        if not 1 <= k <= 32:
            raise ValueError(f"routes of {k} choices: 1 .. 32")
        if self.align not in (1, 128):
            raise ValueError(f"routes.align={self.align}: 1 or 128")
        return (*p, p[2] + 4 * self.experts)

    def trimmed(self):
        """The same without the rows behind the last one in use.  Waits for the
        GPU; for programs that keep rows and know their number anyway."""
        return self._replace(pair=self.pair[:int(self.start[-1])].contiguous())


class Router:
    """Chooses ``top_k`` of ``n_experts`` experts a token.

    score "sigmoid" or "softmax"; groups equal groups of neighbouring experts,
    of which a token's top_groups best are looked at (None: all);
    renormalise divides a token's weights by their sum; scale multiplies them.
    shard=(first, count): the experts of this rank, whose pairs alone get
    rows (None: all).  align: 128 for training (the weight gradient by expert
    needs it), 1 for the fewest rows.  io_dtype "fp32" or "bf16" of the
    logits.  Up to 1024 experts, 32 choices and 32 groups; 32 choices are settled
    in fp64 throughout and take some eight times as long as 31."""

    def __init__(self, n_experts: int, top_k: int, *, score: str = "sigmoid", groups: int = 1,
                 top_groups: int | None = None, renormalise: bool = True, scale: float = 1.0,
                 shard=None, align: int = 128, io_dtype: str = "fp32", device="cuda"):
        for what, v, known in (("score", score, _lib.SCORES), ("io_dtype", io_dtype, _lib.DTYPES)):
            if v not in known:
                raise ValueError(f"{what}={v!r}: one of {', '.join(known)}")
        top_groups = groups if top_groups is None else top_groups
        if not 1 <= n_experts <= 1024:
            raise ValueError(f"{n_experts} experts: 1 .. 1024")
        if not 1 <= groups <= 32 or n_experts % groups:
            raise ValueError(f"{groups} groups of {n_experts} experts: 1 .. 32 equal ones")
        if not 1 <= top_groups <= groups:
            raise ValueError(f"top_groups={top_groups}: 1 .. {groups}")
        if not 1 <= top_k <= min(32, n_experts // groups * top_groups):
            raise ValueError(f"top_k={top_k}: 1 .. 32, and no more than the chosen groups hold")
        if not math.isfinite(scale):
            raise ValueError(f"scale={scale}: finite")
        if align not in (1, 128):
            raise ValueError(f"align={align}: 1 or 128")
        first, count = (0, n_experts) if shard is None else shard
        if first < 0 or count < 1 or first + count > n_experts:
            raise ValueError(f"shard={shard}: experts within 0 .. {n_experts - 1}")
        self.n_experts, self.top_k, self.align = n_experts, top_k, align
        self.first, self.local = first, count
        self.dtype = _TORCH_DT[io_dtype]
        self._dims = dict(experts=n_experts, top_k=top_k, groups=groups, top_groups=top_groups,
                          score=score, renormalise=bool(renormalise), scale=scale, first=first,
                          local=count, align=align, io_dtype=io_dtype)
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"device {self.device}: a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._last = None

    def _c_dims(self, tokens):
        """The C dims, rows and scratch bytes of so many tokens; the last ones
        are kept (and never changed), since calls mostly repeat."""
        last = self._last
        if last is None or last[0] != tokens:
            if tokens * self.top_k > 2 ** 31 - 1:
                raise ValueError(f"{tokens} tokens of {self.top_k} choices: at most 2^31 - 1 pairs")
            dims = _lib.make_route_dims(tokens, **self._dims)
            last = self._last = (tokens, dims, _lib.route_rows(dims),
                                 _lib.route_workspace_bytes(dims))
        return last[1:]

    def rows(self, tokens: int) -> int:
        """Rows that so many tokens' pairs can need."""
        return self._c_dims(tokens)[1]

    def _logits(self, logits):
        if not isinstance(logits, torch.Tensor):
            raise TypeError("logits must be a torch.Tensor")
        if logits.dim() < 1 or logits.shape[-1] != self.n_experts:
            raise ValueError(f"logits: shape {tuple(logits.shape)} does not end in "
                             f"{self.n_experts} experts")
        return (need(logits, "logits", self.dtype, self.device),
                math.prod(logits.shape[:-1]))

    def forward(self, logits, bias=None, *, stream=None) -> Routes:
        """logits [..., n_experts]; bias [n_experts] fp32 (it may start anywhere)."""
        p, T = self._logits(logits)
        dev, k = self.device, self.top_k
        pb = 0 if bias is None else need(bias, "bias", torch.float32, dev, (self.n_experts,))
        dims, rows, nb = self._c_dims(T)
        with on_stream(dev, stream, logits, bias) as st:
            i32 = dict(dtype=torch.int32, device=dev)
            expert, row = torch.empty(T, k, **i32), torch.empty(T, k, **i32)
            weight = torch.empty(T, k, dtype=torch.float32, device=dev)
            pair, start = torch.empty(rows, **i32), torch.empty(self.local + 1, **i32)
            ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
            if pb % 16:
                bias = on_16(bias)
                pb = bias.data_ptr()
            _lib.route_fwd(dims, p, pb, expert.data_ptr(), weight.data_ptr(), row.data_ptr(),
                           pair.data_ptr(), start.data_ptr(), ws.data_ptr() if nb else 0, nb, st)
        return Routes(expert, weight, row, pair, start, self.align)

    def backward(self, logits, routes: Routes, dweight, *, stream=None):
        """Gradient of the logits (their shape and dtype) for dweight [T, k]
        fp32, with the choice held fixed; the bias has none.  NaN for a token
        whose logits all are."""
        p, T = self._logits(logits)
        pe = need(routes.expert, "routes.expert", torch.int32, self.device, (T, self.top_k))
        pw = need(dweight, "dweight", torch.float32, self.device, (T, self.top_k))
        dims = self._c_dims(T)[0]
        with on_stream(self.device, stream, logits, routes.expert, dweight) as st:
            out = torch.empty_like(logits)
            _lib.route_bwd(dims, p, pe, pw, out.data_ptr(), st)
        return out
