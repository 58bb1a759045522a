"""ctypes binding of liblaga.so: argument marshalling only.

Every step of the compute runs in the library's CUDA kernels; this module
turns Python values into the C structs and pointers of ``include/laga.h``
and raises on a non-OK status.  It never falls back to another
implementation: if the library is missing, loading raises.
"""

from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liblaga.so")

LAGA_OK, LAGA_ERR_ARG, LAGA_ERR_ALIGN, LAGA_ERR_WORKSPACE = 0, 1, 2, 3
LAGA_ERR_UNSUPPORTED, LAGA_ERR_CUDA, LAGA_ERR_TIMEOUT = 4, 5, 6
FORMS = {"laga": 0, "explicit": 1, "absorbed": 2, "laga_fused": 3}
DTYPES = {"bf16": 0, "fp32": 1}
NORMS = {"layer": 0, "rms": 1}
POST_NORMS = {**NORMS, "none": 2}
GATES = {"none": 0, "token": 1, "full": 2}
SCORES = {"sigmoid": 0, "softmax": 1}
WS_SAVED, WS_BWD, WS_FWD = 0, 1, 2

EXPORTED = ("laga_workspace_bytes", "laga_workspace_tensor", "laga_fwd", "laga_fwd_scratch",
            "laga_bwd",
            "laga_bwd_overlap", "laga_sync_check", "laga_status_string", "laga_last_launch_count",
            "laga_profile_enable", "laga_profile_reset", "laga_profile_read",
            "laga_norm_rope_bwd_noalloc", "laga_selftest_wait_timeout", "laga_diag_mma_rate",
            "laga_res_fwd", "laga_res_bwd", "laga_res_workspace_bytes", "laga_ckpt_row_bytes",
            "laga_ckpt_pack", "laga_ckpt_pack_rows", "laga_ckpt_unpack", "laga_ckpt_dw",
            "laga_ckpt_dw_workspace_bytes",
            "laga_route_rows", "laga_route_workspace_bytes", "laga_route_fwd", "laga_route_bwd",
            "laga_weight_pack", "laga_mm8", "laga_mm8_workspace_bytes", "laga_experts_dw",
            "laga_experts_dw_workspace_bytes", "laga_spread8", "laga_combine_fwd",
            "laga_combine_bwd", "laga_swiglu_fwd", "laga_swiglu_bwd")


class LagaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("S", ctypes.c_int), ("n_h_total", ctypes.c_int),
                ("head_offset", ctypes.c_int), ("n_h_shard", ctypes.c_int),
                ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_v", ctypes.c_int),
                ("d_kv", ctypes.c_int), ("scale", ctypes.c_float), ("ln_eps", ctypes.c_float),
                ("causal", ctypes.c_int), ("io_dtype", ctypes.c_int), ("form", ctypes.c_int),
                ("norm", ctypes.c_int)]


class LagaResDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("d", ctypes.c_int), ("post", ctypes.c_int),
                ("pre", ctypes.c_int), ("norm_post", ctypes.c_int), ("norm_pre", ctypes.c_int),
                ("eps", ctypes.c_float), ("gate", ctypes.c_int), ("ckpt", ctypes.c_int),
                ("io_dtype", ctypes.c_int)]


class LagaRouteDims(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("experts", ctypes.c_int), ("top_k", ctypes.c_int),
                ("groups", ctypes.c_int), ("top_groups", ctypes.c_int), ("score", ctypes.c_int),
                ("renormalise", ctypes.c_int), ("scale", ctypes.c_float), ("first", ctypes.c_int),
                ("local", ctypes.c_int), ("align", ctypes.c_int), ("io_dtype", ctypes.c_int)]


class LagaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"liblaga.so not found at {path}: build it with "
                           "sequence_latent_norm_gb300.build.build_library()")
    lib = ctypes.CDLL(path)
    P, S, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_float)
    D = ctypes.POINTER(LagaDims)
    lib.laga_workspace_bytes.argtypes = [D, I]
    lib.laga_workspace_bytes.restype = S
    lib.laga_workspace_tensor.argtypes = [D, I, I, ctypes.POINTER(ctypes.c_char_p),
                                          ctypes.POINTER(S), ctypes.POINTER(S)]
    lib.laga_workspace_tensor.restype = I
    lib.laga_fwd.argtypes = [D, P, P, P, P, P, P, P, P, P, S, P]
    lib.laga_fwd.restype = I
    lib.laga_fwd_scratch.argtypes = [D, P, P, P, P, P, P, P, P, P, S, P, S, P]
    lib.laga_fwd_scratch.restype = I
    lib.laga_bwd.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P, S, P]
    lib.laga_bwd.restype = I
    lib.laga_bwd_overlap.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P, S, P,
                                     P, P, P]
    lib.laga_bwd_overlap.restype = I
    lib.laga_sync_check.argtypes = [P]
    lib.laga_sync_check.restype = I
    lib.laga_selftest_wait_timeout.argtypes = [P]
    lib.laga_selftest_wait_timeout.restype = I
    lib.laga_status_string.argtypes = [I]
    lib.laga_status_string.restype = ctypes.c_char_p
    lib.laga_last_launch_count.argtypes = []
    lib.laga_last_launch_count.restype = I
    lib.laga_profile_enable.argtypes = [I]
    lib.laga_profile_enable.restype = None
    lib.laga_profile_reset.argtypes = []
    lib.laga_profile_reset.restype = None
    lib.laga_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p),
                                      ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I), I]
    lib.laga_profile_read.restype = I
    lib.laga_norm_rope_bwd_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P]
    lib.laga_norm_rope_bwd_noalloc.restype = I
    lib.laga_diag_mma_rate.argtypes = [I, I, I, I, I, I, P, P]
    lib.laga_diag_mma_rate.restype = I
    R = ctypes.POINTER(LagaResDims)
    lib.laga_res_fwd.argtypes = [R] + [P] * 13
    lib.laga_res_fwd.restype = I
    lib.laga_res_bwd.argtypes = [R] + [P] * 17 + [S, P]
    lib.laga_res_bwd.restype = I
    lib.laga_res_workspace_bytes.argtypes = [R]
    lib.laga_res_workspace_bytes.restype = S
    lib.laga_ckpt_row_bytes.argtypes = [I]
    lib.laga_ckpt_row_bytes.restype = S
    lib.laga_ckpt_pack.argtypes = [I, I, I, P, P, P]
    lib.laga_ckpt_pack.restype = I
    lib.laga_ckpt_pack_rows.argtypes = [I, I, I, P, P, P, P]
    lib.laga_ckpt_pack_rows.restype = I
    lib.laga_ckpt_unpack.argtypes = [I, I, I, P, P, P]
    lib.laga_ckpt_unpack.restype = I
    lib.laga_ckpt_dw.argtypes = [I, I, I, I, P, P, P, P, P, S, P]
    lib.laga_ckpt_dw.restype = I
    lib.laga_ckpt_dw_workspace_bytes.argtypes = [I, I, I, I]
    lib.laga_ckpt_dw_workspace_bytes.restype = S
    Q = ctypes.POINTER(LagaRouteDims)
    for name, args in (("route_fwd", [Q] + [P] * 8 + [S, P]), ("route_bwd", [Q] + [P] * 5),
                       ("weight_pack", [I] * 4 + [P] * 4), ("mm8", [I] * 5 + [P] * 6 + [S, P]),
                       ("experts_dw", [I] * 5 + [P] * 6 + [S, P]), ("spread8", [I] * 4 + [P] * 5),
                       ("combine_fwd", [I] * 5 + [P] * 5), ("combine_bwd", [I] * 5 + [P] * 9),
                       ("swiglu_fwd", [I] * 3 + [P] * 4), ("swiglu_bwd", [I] * 3 + [P] * 5)):
        f = getattr(lib, "laga_" + name)
        f.argtypes, f.restype = args, I
    for name, args in (("route_rows", [Q]), ("route_workspace_bytes", [Q]),
                       ("mm8_workspace_bytes", [I] * 5), ("experts_dw_workspace_bytes", [I] * 5)):
        f = getattr(lib, "laga_" + name)
        f.argtypes, f.restype = args, S
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().laga_status_string(int(status)).decode()


def make_dims(S, n_h_shard, *, B=1, n_h_total=None, head_offset=0, d_nope=128, d_rope=64,
              d_v=128, d_kv=512, scale=0.0, ln_eps=1e-5, causal=1, io_dtype="bf16",
              form="laga", norm="layer") -> LagaDims:
    return LagaDims(B, S, n_h_shard if n_h_total is None else n_h_total, head_offset, n_h_shard,
                    d_nope, d_rope, d_v, d_kv, scale, ln_eps, causal, DTYPES[io_dtype],
                    FORMS[form], NORMS[norm])


def workspace_bytes(dims: LagaDims, pass_: int) -> int:
    return int(load().laga_workspace_bytes(ctypes.byref(dims), pass_))


def workspace_tensors(dims: LagaDims, pass_: int):
    """[(name, offset, bytes)] of the tensors inside one workspace."""
    lib = load()
    out, i = [], 0
    name, off, nb = ctypes.c_char_p(), ctypes.c_size_t(), ctypes.c_size_t()
    while lib.laga_workspace_tensor(ctypes.byref(dims), pass_, i, ctypes.byref(name),
                                    ctypes.byref(off), ctypes.byref(nb)) == LAGA_OK:
        out.append((name.value.decode(), off.value, nb.value))
        i += 1
    return out


def _check(status: int, what: str):
    if status != LAGA_OK:
        raise LagaError(status, what)


def fwd(dims: LagaDims, q, c, w, gamma, cos, sin, o, lse, ws_saved, saved_bytes, stream=0):
    """laga_fwd with raw device addresses (ints)."""
    _check(load().laga_fwd(ctypes.byref(dims), q, c, w, gamma, cos, sin, o, lse, ws_saved,
                           saved_bytes, stream), "laga_fwd")


def fwd_scratch(dims: LagaDims, q, c, w, gamma, cos, sin, o, lse, ws_saved, saved_bytes, ws_fwd,
                fwd_bytes, stream=0):
    """laga_fwd_scratch with raw device addresses (ints)."""
    _check(load().laga_fwd_scratch(ctypes.byref(dims), q, c, w, gamma, cos, sin, o, lse, ws_saved,
                                   saved_bytes, ws_fwd, fwd_bytes, stream), "laga_fwd_scratch")


def bwd(dims: LagaDims, q, c, w, gamma, cos, sin, o, lse, d_o, dq, dc, dw, dgamma, ws_saved,
        saved_bytes, ws_bwd, bwd_bytes, stream=0):
    """laga_bwd with raw device addresses (ints)."""
    _check(load().laga_bwd(ctypes.byref(dims), q, c, w, gamma, cos, sin, o, lse, d_o, dq, dc, dw,
                           dgamma, ws_saved, saved_bytes, ws_bwd, bwd_bytes, stream), "laga_bwd")


def bwd_overlap(dims: LagaDims, q, c, w, gamma, cos, sin, o, lse, d_o, dq, dc, dw, dgamma,
                ws_saved, saved_bytes, ws_bwd, bwd_bytes, stream, aux_stream, fork_event,
                join_event):
    """laga_bwd_overlap with raw device addresses and stream/event handles (ints)."""
    _check(load().laga_bwd_overlap(ctypes.byref(dims), q, c, w, gamma, cos, sin, o, lse, d_o, dq,
                                   dc, dw, dgamma, ws_saved, saved_bytes, ws_bwd, bwd_bytes,
                                   stream, aux_stream, fork_event, join_event),
           "laga_bwd_overlap")


def sync_check(stream=0):
    _check(load().laga_sync_check(stream), "laga_sync_check")


def selftest_wait_timeout(stream=0):
    """Enqueue the bounded-wait self-test (see include/laga.h)."""
    _check(load().laga_selftest_wait_timeout(stream), "laga_selftest_wait_timeout")


def last_launch_count() -> int:
    return int(load().laga_last_launch_count())


def profile_enable(on: bool):
    load().laga_profile_enable(1 if on else 0)


def profile_reset():
    load().laga_profile_reset()


def profile_read():
    """{kernel name: (total ms, launches)} since the last reset (waits for the events)."""
    lib = load()
    n = 64
    names = (ctypes.c_char_p * n)()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    k = lib.laga_profile_read(names, ms, cnt, n)
    return {names[i].decode(): (ms[i], cnt[i]) for i in range(min(k, n))}


def norm_rope_bwd_noalloc(dims: LagaDims, c, gamma, cos, sin, d_latent, d_kpe_rot, dc, dgamma,
                          stream=0):
    """laga_norm_rope_bwd_noalloc with raw device addresses (ints): the
    LayerNorm + RoPE backward using the library's own fixed scratch."""
    _check(load().laga_norm_rope_bwd_noalloc(ctypes.byref(dims), c, gamma, cos, sin, d_latent,
                                             d_kpe_rot, dc, dgamma, stream),
           "laga_norm_rope_bwd_noalloc")


def diag_mma_rate(form: int, n: int, n_acc: int, run: int, n_instr: int, n_cta: int, cycles,
                  stream=0):
    """laga_diag_mma_rate: SM clocks per CTA for n_instr MMAs into `cycles`
    (a device address of n_cta uint64)."""
    _check(load().laga_diag_mma_rate(form, n, n_acc, run, n_instr, n_cta, cycles, stream),
           "laga_diag_mma_rate")


def make_res_dims(rows, d, *, post=True, pre=True, norm_post="rms", norm_pre="rms", eps=1e-5,
                  gate="none", ckpt=False, io_dtype="bf16") -> LagaResDims:
    return LagaResDims(rows, d, int(post), int(pre), POST_NORMS[norm_post], NORMS[norm_pre], eps,
                       GATES[gate], int(ckpt), DTYPES[io_dtype])


def res_fwd(dims: LagaResDims, x, y, gate, alpha, gamma_post, gamma_pre, x_out, h, ck_y, ck_x,
            stat_post, stat_pre, stream=0):
    """laga_res_fwd with raw device addresses (ints; 0 for what is off)."""
    _check(load().laga_res_fwd(ctypes.byref(dims), x, y, gate, alpha, gamma_post, gamma_pre, x_out,
                               h, ck_y, ck_x, stat_post, stat_pre, stream), "laga_res_fwd")


def res_workspace_bytes(dims: LagaResDims) -> int:
    return int(load().laga_res_workspace_bytes(ctypes.byref(dims)))


def res_bwd(dims: LagaResDims, dx_out, dh, kept_y, kept_x, stat_post, stat_pre, gate, alpha,
            gamma_post, gamma_pre, dx, dy, dgate, dalpha, dgamma_post, dgamma_pre, ws, ws_bytes,
            stream=0):
    """laga_res_bwd with raw device addresses (ints; 0 for what is off)."""
    _check(load().laga_res_bwd(ctypes.byref(dims), dx_out, dh, kept_y, kept_x, stat_post, stat_pre,
                               gate, alpha, gamma_post, gamma_pre, dx, dy, dgate, dalpha,
                               dgamma_post, dgamma_pre, ws, ws_bytes, stream), "laga_res_bwd")


def ckpt_row_bytes(d: int) -> int:
    """Bytes of one checkpoint row of d channels (0: not a valid width)."""
    return int(load().laga_ckpt_row_bytes(d))


def ckpt_pack(rows, d, dtype, x, ck, stream=0):
    """laga_ckpt_pack with raw device addresses (ints); dtype "bf16" or "fp32"."""
    _check(load().laga_ckpt_pack(rows, d, DTYPES[dtype], x, ck, stream), "laga_ckpt_pack")


def ckpt_pack_rows(rows, d, dtype, x, end, ck, stream=0):
    """laga_ckpt_pack_rows with raw device addresses (ints)."""
    _check(load().laga_ckpt_pack_rows(rows, d, DTYPES[dtype], x, end, ck, stream),
           "laga_ckpt_pack_rows")


def ckpt_unpack(rows, d, dtype, ck, x, stream=0):
    """laga_ckpt_unpack with raw device addresses (ints)."""
    _check(load().laga_ckpt_unpack(rows, d, DTYPES[dtype], ck, x, stream), "laga_ckpt_unpack")


def ckpt_dw_workspace_bytes(rows, d, n, dy_dtype) -> int:
    return int(load().laga_ckpt_dw_workspace_bytes(rows, d, n, DTYPES[dy_dtype]))


def ckpt_dw(rows, d, n, dy_dtype, ck, dy, gamma, dw, ws, ws_bytes, stream=0):
    """laga_ckpt_dw with raw device addresses (ints; gamma 0: no row gain)."""
    _check(load().laga_ckpt_dw(rows, d, n, DTYPES[dy_dtype], ck, dy, gamma, dw, ws, ws_bytes,
                               stream), "laga_ckpt_dw")


def make_route_dims(tokens, experts, top_k, *, groups=1, top_groups=1, score="sigmoid",
                    renormalise=True, scale=1.0, first=0, local=None, align=128,
                    io_dtype="fp32") -> LagaRouteDims:
    return LagaRouteDims(tokens, experts, top_k, groups, top_groups, SCORES[score],
                         int(renormalise), scale, first, experts if local is None else local,
                         align, DTYPES[io_dtype])


def route_rows(dims: LagaRouteDims) -> int:
    """Rows that the pairs can need (0: none, or invalid dims)."""
    return int(load().laga_route_rows(ctypes.byref(dims)))


def route_workspace_bytes(dims: LagaRouteDims) -> int:
    return int(load().laga_route_workspace_bytes(ctypes.byref(dims)))


def route_fwd(dims: LagaRouteDims, logits, bias, expert, weight, row, pair, start, ws, ws_bytes,
              stream=0):
    """laga_route_fwd with raw device addresses (ints; bias 0: none)."""
    _check(load().laga_route_fwd(ctypes.byref(dims), logits, bias, expert, weight, row, pair,
                                 start, ws, ws_bytes, stream), "laga_route_fwd")


def route_bwd(dims: LagaRouteDims, logits, expert, dweight, dlogits, stream=0):
    """laga_route_bwd with raw device addresses (ints)."""
    _check(load().laga_route_bwd(ctypes.byref(dims), logits, expert, dweight, dlogits, stream),
           "laga_route_bwd")


def weight_pack(experts, k, n, dtype, w, fwd, bwd, stream=0):
    """laga_weight_pack with raw device addresses (ints; bwd 0: not written)."""
    _check(load().laga_weight_pack(experts, k, n, DTYPES[dtype], w, fwd, bwd, stream),
           "laga_weight_pack")


def mm8_workspace_bytes(rows, k, n, experts, out_dtype) -> int:
    return int(load().laga_mm8_workspace_bytes(rows, k, n, experts, DTYPES[out_dtype]))


def mm8(rows, k, n, experts, out_dtype, a, b, start, pair, y, ws, ws_bytes, stream=0):
    """laga_mm8 with raw device addresses (ints; experts 0: one matrix b; pair 0: none)."""
    _check(load().laga_mm8(rows, k, n, experts, DTYPES[out_dtype], a, b, start, pair, y, ws,
                           ws_bytes, stream), "laga_mm8")


def experts_dw_workspace_bytes(rows, d, n, experts, dy_dtype) -> int:
    return int(load().laga_experts_dw_workspace_bytes(rows, d, n, experts, DTYPES[dy_dtype]))


def experts_dw(rows, d, n, experts, dy_dtype, ck, dy, gamma, start, dw, ws, ws_bytes, stream=0):
    """laga_experts_dw with raw device addresses (ints; gamma 0: no row gain)."""
    _check(load().laga_experts_dw(rows, d, n, experts, DTYPES[dy_dtype], ck, dy, gamma, start, dw,
                                  ws, ws_bytes, stream), "laga_experts_dw")


def spread8(rows, tokens, top_k, d, ck, pair, end, out, stream=0):
    """laga_spread8 with raw device addresses (ints)."""
    _check(load().laga_spread8(rows, tokens, top_k, d, ck, pair, end, out, stream),
           "laga_spread8")


def combine_fwd(tokens, top_k, rows, d, dtype, y, weight, row, out, stream=0):
    """laga_combine_fwd with raw device addresses (ints; weight 0: ones)."""
    _check(load().laga_combine_fwd(tokens, top_k, rows, d, DTYPES[dtype], y, weight, row, out,
                                   stream), "laga_combine_fwd")


def combine_bwd(tokens, top_k, rows, d, dtype, dout, y, weight, row, pair, end, dy, dweight,
                stream=0):
    """laga_combine_bwd with raw device addresses (ints; y and dweight 0: no dweight)."""
    _check(load().laga_combine_bwd(tokens, top_k, rows, d, DTYPES[dtype], dout, y, weight, row,
                                   pair, end, dy, dweight, stream), "laga_combine_bwd")


def swiglu_fwd(rows, f, dtype, gu, end, ck, stream=0):
    """laga_swiglu_fwd with raw device addresses (ints; end 0: all rows)."""
    _check(load().laga_swiglu_fwd(rows, f, DTYPES[dtype], gu, end, ck, stream), "laga_swiglu_fwd")


def swiglu_bwd(rows, f, dtype, gu, da, end, dgu, stream=0):
    """laga_swiglu_bwd with raw device addresses (ints; end 0: all rows)."""
    _check(load().laga_swiglu_bwd(rows, f, DTYPES[dtype], gu, da, end, dgu, stream),
           "laga_swiglu_bwd")
