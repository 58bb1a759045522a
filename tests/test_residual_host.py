"""Host-side checks of the residual-stream and 8-bit checkpoint entry points:
sizes, layouts and refusals, all before any CUDA call."""

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


def test_checkpoint_row_bytes_match_the_layout(lib):
    for d in (1, 127, 128, 129, 1001, 2048, 2049, 7168, 16384):
        assert lib.ckpt_row_bytes(d) == ores.row_layout(d)[1]
    for d in (0, -1, 16385):
        assert lib.ckpt_row_bytes(d) == 0


def test_workspace_sizes_are_zero_for_invalid_dims(lib):
    ok = lib.make_res_dims(64, 512)
    assert lib.res_workspace_bytes(ok) > 0
    for field, v in [("rows", -1), ("d", 0), ("d", 16385), ("post", 2), ("pre", -1),
                     ("norm_post", 3), ("norm_pre", 2), ("gate", 3), ("ckpt", 2), ("io_dtype", 2),
                     ("eps", 0.0), ("eps", float("inf")), ("eps", float("nan"))]:
        dims = lib.make_res_dims(64, 512)
        setattr(dims, field, v)
        assert lib.res_workspace_bytes(dims) == 0, (field, v)
    dims = lib.make_res_dims(64, 512, post=False, pre=False)
    assert lib.res_workspace_bytes(dims) == 0
    for bad in [(-1, 64, 64), (4, 0, 64), (4, 16385, 64), (4, 64, 0), (4, 64, (1 << 20) + 1)]:
        assert lib.ckpt_dw_workspace_bytes(*bad, "bf16") == 0


no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake pointers are only safe without a GPU")


def _addr(n):
    return [0x10000 * (i + 1) for i in range(n)]


@no_gpu
def test_res_fwd_refusals(lib):
    so, d = lib.load(), lib.make_res_dims(8, 256, gate="full", ckpt=True)
    p = _addr(12)

    def call(dims, ptrs):
        return so.laga_res_fwd(ctypes.byref(dims), *ptrs, None)

    assert so.laga_res_fwd(None, *p, None) == lib.LAGA_ERR_ARG
    for i in range(12):
        q = list(p)
        q[i] = 0
        assert call(d, q) == lib.LAGA_ERR_ARG, i
        q[i] = p[i] + 8
        assert call(d, q) == lib.LAGA_ERR_ALIGN, i
    assert call(d, p) == lib.LAGA_ERR_CUDA           # no GPU here
    # what is off is ignored: y, gate, alpha, gamma_post, x_out, ck_y, stat_post
    pre = lib.make_res_dims(8, 256, post=False)
    q = [p[0], 0, 0, 0, 0, p[5], 0, p[7], 0, 0, 0, p[11]]
    assert call(pre, q) == lib.LAGA_ERR_CUDA
    assert call(lib.make_res_dims(0, 256), [0] * 12) == lib.LAGA_OK
    assert call(lib.make_res_dims(8, 256, post=False, pre=False), p) == lib.LAGA_ERR_ARG


@no_gpu
def test_res_bwd_refusals(lib):
    so, d = lib.load(), lib.make_res_dims(8, 256, gate="full", ckpt=True)
    p, nb = _addr(17), lib.res_workspace_bytes(lib.make_res_dims(8, 256))

    def call(dims, ptrs, n=nb):
        return so.laga_res_bwd(ctypes.byref(dims), *ptrs, n, None)

    for i in range(1, 17):
        q = list(p)
        q[i] = 0
        assert call(d, q) == (lib.LAGA_ERR_WORKSPACE if i == 16 else lib.LAGA_ERR_ARG), i
        q[i] = p[i] + 4
        assert call(d, q) == lib.LAGA_ERR_ALIGN, i
    assert call(d, p, nb - 1) == lib.LAGA_ERR_WORKSPACE
    assert call(d, p) == lib.LAGA_ERR_CUDA
    assert call(d, [0] + p[1:]) == lib.LAGA_ERR_CUDA     # x' may have no other use ...
    post = lib.make_res_dims(8, 256, pre=False, gate="full")
    assert call(post, [0] + p[1:]) == lib.LAGA_ERR_ARG   # ... unless it is the only output


@no_gpu
def test_checkpoint_refusals(lib):
    so, p = lib.load(), _addr(5)
    for f in (so.laga_ckpt_pack, so.laga_ckpt_unpack):
        assert f(4, 64, 0, p[0], p[1], None) == lib.LAGA_ERR_CUDA
        assert f(0, 64, 0, None, None, None) == lib.LAGA_OK
        for bad in [(-1, 64, 0), (4, 0, 0), (4, 16385, 0), (4, 64, 2)]:
            assert f(*bad, p[0], p[1], None) == lib.LAGA_ERR_ARG
        assert f(4, 64, 0, None, p[1], None) == lib.LAGA_ERR_ARG
        assert f(4, 64, 0, p[0], None, None) == lib.LAGA_ERR_ARG
        assert f(4, 64, 0, p[0] + 1, p[1], None) == lib.LAGA_ERR_ALIGN
        assert f(4, 64, 0, p[0], p[1] + 8, None) == lib.LAGA_ERR_ALIGN
    nb = lib.ckpt_dw_workspace_bytes(300, 256, 65, "fp32")

    def dw(sizes, ck, dy, g, out, ws, n):
        return so.laga_ckpt_dw(*sizes, ck, dy, g, out, ws, n, None)

    ok = (300, 256, 65, 1)
    assert dw(ok, p[0], p[1], p[2], p[3], p[4], nb) == lib.LAGA_ERR_CUDA
    assert dw(ok, p[0], p[1], None, p[3], p[4], nb) == lib.LAGA_ERR_CUDA
    assert dw(ok, None, p[1], None, p[3], p[4], nb) == lib.LAGA_ERR_ARG
    assert dw(ok, p[0], None, None, p[3], p[4], nb) == lib.LAGA_ERR_ARG
    assert dw(ok, p[0], p[1], None, None, p[4], nb) == lib.LAGA_ERR_ARG
    assert dw(ok, p[0], p[1] + 8, None, p[3], p[4], nb) == lib.LAGA_ERR_ALIGN
    assert dw(ok, p[0], p[1], p[2] + 4, p[3], p[4], nb) == lib.LAGA_ERR_ALIGN
    if nb:
        assert dw(ok, p[0], p[1], None, p[3], p[4], nb - 1) == lib.LAGA_ERR_WORKSPACE
        assert dw(ok, p[0], p[1], None, p[3], None, nb) == lib.LAGA_ERR_WORKSPACE
    for bad in [(-1, 64, 64, 0), (4, 0, 64, 0), (4, 64, 0, 0), (4, 64, (1 << 20) + 1, 0),
                (4, 64, 64, 2)]:
        assert dw(bad, p[0], p[1], None, p[3], p[4], 1 << 40) == lib.LAGA_ERR_ARG


def test_python_refusals(lib):
    import sequence_latent_norm_gb300 as laga
    for kw in (dict(norm_post="batch"), dict(norm_pre="none"), dict(gate="row"),
               dict(io_dtype="fp16"), dict(post=False, pre=False), dict(eps=0.0),
               dict(eps=float("nan"))):
        with pytest.raises(ValueError):
            laga.ResidualNorm(64, device="cuda:0", **kw)
    for d in (0, 16385):
        with pytest.raises(ValueError):
            laga.ResidualNorm(d, device="cuda:0")
    with pytest.raises(ValueError, match="CUDA device"):
        laga.ResidualNorm(64, device="cpu")
    op = laga.ResidualNorm(64, device="cuda:0")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected cuda:0"):
        op.forward(x, x)                                    # not on the GPU
    with pytest.raises(ValueError, match="dtype"):
        op.forward(x.float(), x)
    with pytest.raises(ValueError, match="shape"):
        op.forward(torch.zeros(4, 65, dtype=torch.bfloat16), x)
    with pytest.raises(TypeError):
        op.forward(None, x)
    with pytest.raises(TypeError):
        laga.pack8(x.half())
    with pytest.raises(ValueError, match="CUDA device"):
        laga.pack8(x)
    with pytest.raises(ValueError):
        laga.Checkpoint8(torch.zeros(4, 144, dtype=torch.uint8), 64)       # not on the GPU
    with pytest.raises(ValueError):
        laga.Checkpoint8(torch.zeros(4, 143, dtype=torch.uint8), 64)
    with pytest.raises(ValueError):
        laga.Checkpoint8(torch.zeros(4, 144, dtype=torch.uint8), 0)


def test_block_refuses_a_kept_that_is_not_h():
    import sequence_latent_norm_gb300 as laga
    from sequence_latent_norm_gb300.block import LagaAttentionBlock
    h = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    b = LagaAttentionBlock(None, 2)
    with pytest.raises(ValueError, match="kept_gain"):
        b.forward(h, *[None] * 7, kept_gain=torch.ones(64))
    with pytest.raises(TypeError, match="Checkpoint8"):
        b.forward(h, *[None] * 7, kept=h)
    for rows, d in ((3, 64), (4, 128)):
        ck = laga.Checkpoint8.__new__(laga.Checkpoint8)
        ck.data, ck.d, ck.shape = torch.zeros(rows, 144, dtype=torch.uint8), d, (rows, d)
        with pytest.raises(ValueError, match="expected 4 of 64"):
            b.forward(h, *[None] * 7, kept=ck)
