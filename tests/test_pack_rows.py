"""Packing of experts' rows: the rows in use alone.  Buffers of rows hold the most
that a batch can need, and what lies behind the last row in use is neither written
nor read."""

import pytest
import torch

DEV = "cuda:0"


@pytest.fixture(scope="module")
def lib():
    from sequence_latent_norm_gb300.build import build_library
    build_library()
    import sequence_latent_norm_gb300 as pkg
    return pkg._lib


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only safe without a GPU")
def test_refusals(lib):
    so, p = lib.load(), [0x10000 * (i + 1) for i in range(3)]

    def pack(rows, d, dt, x, end, ck):
        return so.laga_ckpt_pack_rows(rows, d, dt, x, end, ck, None)

    for a in [(-1, 8, 0), (4, 0, 0), (4, 16385, 0), (4, 8, 2)]:
        assert pack(*a, *p) == lib.LAGA_ERR_ARG, a
    for i in range(3):
        q = list(p)
        q[i] = 0
        assert pack(4, 8, 0, *q) == lib.LAGA_ERR_ARG, i
    assert pack(4, 8, 0, p[0] + 8, p[1], p[2]) == lib.LAGA_ERR_ALIGN
    assert pack(4, 8, 0, p[0], p[1] + 4, p[2]) == lib.LAGA_ERR_CUDA      # of 4 bytes: start's last
    assert pack(0, 8, 0, 0, 0, 0) == lib.LAGA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dt,name", [(torch.bfloat16, "bf16"), (torch.float32, "fp32")])
@pytest.mark.parametrize("d", [1, 129, 256, 7168])
@pytest.mark.parametrize("rows,used", [(37, 0), (37, 1), (300, 128), (300, 299), (300, 300), (9, 50),
                                       (9, -3)])
def test_rows_behind_the_last_one_keep_their_bytes(lib, rows, used, d, dt, name):
    import sequence_latent_norm_gb300 as laga
    x = torch.randn(rows, d, generator=torch.Generator().manual_seed(rows + d)).to(dt).to(DEV)
    want = laga.pack8(x).data
    n = min(max(used, 0), rows)
    x[n:] = float("nan")
    ck = torch.full_like(want, 0x5a)
    end = torch.tensor([7, used], dtype=torch.int32, device=DEV)
    lib.ckpt_pack_rows(rows, d, name, x.data_ptr(), end.data_ptr() + 4, ck.data_ptr(),
                       torch.cuda.current_stream().cuda_stream)
    lib.sync_check()
    assert torch.equal(ck[:n], want[:n]) and (ck[n:] == 0x5a).all()


@pytest.mark.gpu
@pytest.mark.parametrize("align", [1, 128])
def test_pack8_by_routes(lib, align):
    import sequence_latent_norm_gb300 as laga
    r = laga.Router(16, 2, align=align, device=DEV).forward(torch.randn(50, 16, device=DEV))
    used = int(r.start[-1])
    x = torch.randn(r.rows, 384, device=DEV)
    ck = laga.pack8(x, routes=r)
    assert ck.shape == (r.rows, 384) and torch.equal(ck.data[:used], laga.pack8(x).data[:used])
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    other = laga.pack8(x, side, routes=r)
    side.synchronize()
    assert torch.equal(ck.data[:used], other.data[:used])
    with pytest.raises(ValueError, match="rows"):
        laga.pack8(x[:-1].contiguous(), routes=r)
    # none in use, and no tokens
    off = laga.Router(16, 2, align=align, device=DEV).forward(
        torch.full((50, 16), -float("inf"), device=DEV))
    assert laga.pack8(x, routes=off).shape == x.shape
    none = laga.Router(16, 2, align=align, device=DEV).forward(torch.zeros(0, 16, device=DEV))
    assert laga.pack8(x[:0], routes=none).rows == 0
    lib.sync_check()


@pytest.mark.gpu
def test_the_block_packs_the_rows_in_use(lib, monkeypatch):
    """Both gradients that the backward pass packs are experts' rows."""
    import sequence_latent_norm_gb300 as laga
    from sequence_latent_norm_gb300 import experts
    seen = []

    def spy(x, stream=None, **kw):
        seen.append((x.shape[0], kw.get("routes")))
        return laga.pack8(x, stream, **kw)

    monkeypatch.setattr(experts, "pack8", spy)
    g = torch.Generator().manual_seed(1)
    h = torch.randn(40, 256, generator=g).bfloat16().to(DEV)
    w = [torch.randn(*s, generator=g).mul_(0.05).to(DEV) for s in ((256, 8), (8, 256, 256), (8, 128, 256))]
    block = laga.RoutedExperts(8, 2, device=DEV)
    block.forward(h, w[0], w[1].bfloat16(), w[2].bfloat16())
    block.backward(torch.randn(40, 256, generator=g).bfloat16().to(DEV))
    lib.sync_check()
    rows = block.router.rows(40)
    assert [n for n, _ in seen] == [40, rows, rows]
    assert seen[0][1] is None and all(r is not None for _, r in seen[1:])
