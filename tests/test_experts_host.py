"""Host-side checks of routing, the 8-bit products and the experts' rows:
sizes and refusals, all before any CUDA call."""

import ctypes

import pytest
import torch

from oracle import residual as ores


@pytest.fixture(scope="module")
def lib():
    from sequence_latent_norm_gb300.build import build_library
    build_library()
    import sequence_latent_norm_gb300 as pkg
    return pkg._lib


no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake pointers are only safe without a GPU")


def _addr(n):
    return [0x10000 * (i + 1) for i in range(n)]


def test_rows_of_a_batch(lib):
    for T, k, E, align, want in [(0, 2, 8, 128, 0), (1, 2, 8, 1, 2), (1, 2, 8, 128, 256),
                                 (100, 8, 32, 1, 800), (100, 8, 32, 128, (800 + 32 * 127) // 128 * 128)]:
        assert lib.route_rows(lib.make_route_dims(T, E, k, align=align)) == want
    # a shard gets no more of a token's pairs than it has experts
    assert lib.route_rows(lib.make_route_dims(100, 32, 8, first=3, local=2, align=1)) == 200
    top = lib.make_route_dims(2 ** 26, 256, 32, align=1)
    assert lib.route_rows(top) == 0                    # 2^31 pairs
    assert lib.route_rows(lib.make_route_dims(2 ** 26 - 8, 256, 31, align=1)) == (2 ** 26 - 8) * 31
    assert lib.route_workspace_bytes(lib.make_route_dims(1, 256, 8)) == 0
    assert lib.route_workspace_bytes(lib.make_route_dims(16384, 256, 8)) > 0


BAD_DIMS = [("tokens", -1), ("experts", 0), ("experts", 1025), ("top_k", 0), ("top_k", 33),
            ("groups", 0), ("groups", 33), ("groups", 7), ("top_groups", 0), ("top_groups", 5),
            ("score", 2), ("score", -1), ("renormalise", 2), ("scale", float("inf")),
            ("scale", float("nan")), ("first", -1), ("first", 64), ("local", 0), ("local", 65),
            ("align", 0), ("align", 64), ("io_dtype", 2), ("top_k", 17)]


def test_bad_dims_have_no_rows(lib):
    for field, v in BAD_DIMS:
        d = lib.make_route_dims(8, 64, 4, groups=4, top_groups=1)
        assert lib.route_rows(d) > 0
        setattr(d, field, v)
        assert lib.route_rows(d) == 0 and lib.route_workspace_bytes(d) == 0, (field, v)


@no_gpu
def test_route_refusals(lib):
    so, p = lib.load(), _addr(8)
    d = lib.make_route_dims(4000, 64, 4, groups=4, top_groups=1)
    nb = lib.route_workspace_bytes(d)

    def fwd(dims, q, n=nb):
        return so.laga_route_fwd(ctypes.byref(dims), *q, n, None)

    def bwd(dims, q):
        return so.laga_route_bwd(ctypes.byref(dims), *q, None)

    assert so.laga_route_fwd(None, *p, nb, None) == lib.LAGA_ERR_ARG
    for field, v in BAD_DIMS:
        bad = lib.make_route_dims(4000, 64, 4, groups=4, top_groups=1)
        setattr(bad, field, v)
        assert fwd(bad, p) == lib.LAGA_ERR_ARG and bwd(bad, p[:4]) == lib.LAGA_ERR_ARG
    for i in range(8):
        q = list(p)
        q[i] = 0
        want = lib.LAGA_ERR_CUDA if i == 1 else (lib.LAGA_ERR_WORKSPACE if i == 7 else lib.LAGA_ERR_ARG)
        assert fwd(d, q) == want, i                     # no bias is fine (no GPU here)
        q[i] = p[i] + 4
        assert fwd(d, q) == lib.LAGA_ERR_ALIGN, i
    assert fwd(d, p, nb - 1) == lib.LAGA_ERR_WORKSPACE
    for i in range(4):
        q = p[:4]
        q[i] = 0
        assert bwd(d, q) == lib.LAGA_ERR_ARG
        q[i] = p[i] + 8
        assert bwd(d, q) == lib.LAGA_ERR_ALIGN
    assert bwd(lib.make_route_dims(0, 64, 4), [0] * 4) == lib.LAGA_OK


@no_gpu
def test_product_refusals(lib):
    so, p = lib.load(), _addr(7)

    def mm8(rows, k, n, e, dt, q, nb=0):
        return so.laga_mm8(rows, k, n, e, dt, *q, nb, None)

    ok = (300, 256, 20000 // 2, 3, 0)
    for i, v in [(0, -1), (0, 2 ** 31 - 1), (1, 0), (1, 16385), (2, 0), (2, 16385), (3, -1),
                 (3, 1025), (4, 2)]:
        a = list(ok)
        a[i] = v
        assert mm8(*a, p[:6]) == lib.LAGA_ERR_ARG, (i, v)
        assert lib.load().laga_mm8_workspace_bytes(*a) == 0
    for i in (0, 1, 2, 4):                             # a, b, start, y; pair may be missing
        q = p[:6]
        q[i] = 0
        assert mm8(*ok, q) == lib.LAGA_ERR_ARG, i
    for i in range(5):
        q = p[:6]
        q[i] += 8
        assert mm8(*ok, q) == lib.LAGA_ERR_ALIGN, i
    # one row: K is split, its partial sums need room
    nb = lib.mm8_workspace_bytes(1, 7168, 256, 0, "bf16")
    assert nb > 0
    q = [p[0], p[1], 0, 0, p[4], p[5]]
    assert mm8(1, 7168, 256, 0, 0, q, nb - 1) == lib.LAGA_ERR_WORKSPACE
    assert mm8(1, 7168, 256, 0, 0, q[:5] + [0], nb) == lib.LAGA_ERR_WORKSPACE
    assert mm8(1, 7168, 256, 0, 0, q, nb) == lib.LAGA_ERR_CUDA
    assert mm8(0, 256, 256, 0, 0, [0] * 6) == lib.LAGA_OK

    for a in [(0, 8, 8, 0), (1025, 8, 8, 0), (1, 0, 8, 0), (1, 8, 16385, 0), (1, 8, 8, 2)]:
        assert so.laga_weight_pack(*a, p[0], p[1], p[2], None) == lib.LAGA_ERR_ARG
    assert so.laga_weight_pack(1, 8, 8, 0, 0, p[1], p[2], None) == lib.LAGA_ERR_ARG
    assert so.laga_weight_pack(1, 8, 8, 0, p[0], p[1], p[2] + 8, None) == lib.LAGA_ERR_ALIGN
    assert so.laga_weight_pack(1, 8, 8, 0, p[0], p[1], 0, None) == lib.LAGA_ERR_CUDA


@no_gpu
def test_weight_gradient_and_row_refusals(lib):
    so, p = lib.load(), _addr(8)
    nb = lib.experts_dw_workspace_bytes(300, 200, 100, 3, "fp32")
    assert nb > 0
    for a in [(-1, 8, 8, 1), (8, 0, 8, 1), (8, 16385, 8, 1), (8, 8, 0, 1), (8, 8, 2 ** 20 + 1, 1),
              (8, 8, 8, 0), (8, 8, 8, 1025), (2 ** 31 - 1, 8, 8, 1)]:
        assert lib.experts_dw_workspace_bytes(*a, "bf16") == 0, a
        assert so.laga_experts_dw(*a, 0, *p[:6], nb, None) == lib.LAGA_ERR_ARG, a

    def dw(q, n=nb):
        return so.laga_experts_dw(300, 200, 100, 3, 1, *q, n, None)

    for i in (0, 1, 3, 4):
        q = p[:6]
        q[i] = 0
        assert dw(q) == lib.LAGA_ERR_ARG, i
    assert dw(p[:5] + [0]) == lib.LAGA_ERR_WORKSPACE and dw(p[:6], nb - 1) == lib.LAGA_ERR_WORKSPACE
    assert dw([p[0] + 8] + p[1:6]) == lib.LAGA_ERR_ALIGN

    for a in [(-1, 8, 2, 64), (8, -1, 2, 64), (8, 8, 0, 64), (8, 8, 33, 64), (8, 8, 2, 0),
              (8, 8, 2, 16385), (8, 2 ** 27, 16, 64)]:
        assert so.laga_spread8(*a, *p[:4], None) == lib.LAGA_ERR_ARG, a
        rows, T, k, d = a
        assert so.laga_combine_fwd(T, k, rows, d, 0, *p[:4], None) == lib.LAGA_ERR_ARG, a
        assert so.laga_combine_bwd(T, k, rows, d, 0, *p[:8], None) == lib.LAGA_ERR_ARG, a
    assert so.laga_spread8(8, 8, 2, 64, p[0], p[1], 0, p[3], None) == lib.LAGA_ERR_ARG
    assert so.laga_combine_fwd(8, 2, 8, 64, 2, *p[:4], None) == lib.LAGA_ERR_ARG
    # dweight needs y
    assert so.laga_combine_bwd(8, 2, 8, 64, 0, p[0], 0, *p[2:8], None) == lib.LAGA_ERR_ARG
    assert so.laga_combine_bwd(8, 2, 8, 64, 0, p[0], 0, *p[2:7], 0, None) == lib.LAGA_ERR_CUDA
    for a in [(-1, 8, 0), (8, 0, 0), (8, 16385, 0), (8, 8, 2)]:
        assert so.laga_swiglu_fwd(*a, p[0], 0, p[1], None) == lib.LAGA_ERR_ARG
        assert so.laga_swiglu_bwd(*a, p[0], p[1], 0, p[2], None) == lib.LAGA_ERR_ARG
    assert so.laga_swiglu_fwd(8, 8, 0, p[0] + 8, 0, p[1], None) == lib.LAGA_ERR_ALIGN


def test_router_refusals(lib):
    from sequence_latent_norm_gb300 import Router
    for kw in [dict(score="tanh"), dict(io_dtype="fp16"), dict(groups=3), dict(groups=64),
               dict(groups=4, top_groups=5), dict(groups=4, top_groups=0), dict(scale=float("nan")),
               dict(align=2), dict(shard=(60, 5)), dict(shard=(-1, 5)), dict(shard=(0, 0)),
               dict(device="cpu")]:
        with pytest.raises(ValueError):
            Router(64, 4, **{"device": "cuda:0", **kw})
    for n, k in [(0, 1), (1025, 1), (64, 0), (64, 33)]:
        with pytest.raises(ValueError):
            Router(n, k, device="cuda:0")
    with pytest.raises(ValueError):
        Router(64, 17, groups=4, top_groups=1, device="cuda:0")
    r = Router(64, 4, device="cuda:0")
    assert r.rows(10) == (40 + 40 * 127) // 128 * 128
    with pytest.raises(ValueError, match="2\\^31"):
        r.rows(2 ** 30)
    with pytest.raises(TypeError):
        r.forward(None)
    with pytest.raises(ValueError, match="64 experts"):
        r.forward(torch.zeros(3, 65))
    with pytest.raises(ValueError, match="CUDA|cuda"):
        r.forward(torch.zeros(3, 64))


def test_what_is_not_in_8_bits_is_refused(lib):
    import sequence_latent_norm_gb300 as laga
    t = torch.zeros(4, 8, dtype=torch.bfloat16)
    for f in (laga.linear8, laga.linear8_dx):
        with pytest.raises(TypeError, match="Weight8"):
            f(t, t)
    with pytest.raises(TypeError, match="Checkpoint8"):
        laga.spread8(t, None)
    with pytest.raises(TypeError):
        laga.pack_weight8(t.half())
    for shape in [(4,), (1, 2, 3, 4)]:
        with pytest.raises(ValueError):
            laga.pack_weight8(torch.zeros(shape))
    for shape in [(8,), (0, 8), (8, 16385), (1025, 8, 8), (0, 8, 8)]:
        with pytest.raises(ValueError):
            laga.Weight8(shape, t)
    for f in (laga.swiglu8, laga.combine):
        with pytest.raises(TypeError):
            f(t.half(), None) if f is laga.combine else f(t.half())
    with pytest.raises(ValueError, match="even"):
        laga.swiglu8(torch.zeros(4, 7))
    with pytest.raises(ValueError, match="sets shard"):
        laga.RoutedExperts(8, 2, shard=(0, 4), device="cuda:0")


def test_blocks_refuse_unknown_options(lib):
    import sequence_latent_norm_gb300 as laga
    from sequence_latent_norm_gb300.block import LagaAttentionBlock, LagaResidualStack
    with pytest.raises(ValueError, match="projections"):
        LagaAttentionBlock(None, 2, projections="fp16")
    e = laga.RoutedExperts(8, 2, device="cuda:0")
    with pytest.raises(ValueError, match="several ranks"):
        LagaResidualStack([LagaAttentionBlock(None, 2, distributed=True), e], 64, device="cuda:0")
    with pytest.raises(ValueError, match="dtype"):
        e.forward(torch.zeros(2, 64), None, None, None)
    h = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="kept_gain"):
        e.forward(h, None, None, None, kept_gain=h)
    with pytest.raises(TypeError, match="Checkpoint8"):
        e.forward(h, None, None, None, kept=h)


def test_row_layout_of_weights(lib):
    assert lib.ckpt_row_bytes(7168) == ores.row_layout(7168)[1]
