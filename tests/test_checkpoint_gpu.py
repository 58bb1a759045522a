"""8-bit checkpoints on the GPU: packing bit for bit against the fp64 oracle,
and the weight gradient taken from the codes.

The weight gradient multiplies values that are exact in bf16 with dy (exact
too) and adds rows of them in fp32: n products in a chain add at most n u of
the sum of their magnitudes, u = 2^-24 for a rounded addition and 2^-23 for
one that truncates, as the tensor cores' may; the checks allow (n + 64) 2^-23,
and the row gain's own rounding fits in the 64."""

import numpy as np
import pytest
import torch

from laga_inputs import as_f64
from oracle import residual as ores

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda:0"


def _laga():
    import sequence_latent_norm_gb300 as laga
    return laga


def _sync():
    _laga()._lib.sync_check()


def _same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (2, 127), (5, 128), (4, 129), (33, 200),
                                    (257, 1001), (6, 2048), (9, 7168), (1, 16384), (2, 16383),
                                    (2000, 512)])
def test_pack_and_unpack_bit_for_bit(rows, d, dtype):
    g = torch.Generator().manual_seed(rows * 7 + d)
    x = torch.randn(rows, d, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g))
    x = x.to(DT[dtype])
    ck = _laga().pack8(x.to(DEV))
    _sync()
    want = ores.pack(as_f64(x))
    assert _same(ck.data.cpu().numpy(), want)
    v = ores.unpack(want, d)
    for out in (torch.bfloat16, torch.float32):
        assert _same(as_f64(ck.unpack(out)), v)
    assert ck.shape == (rows, d) and ck.nbytes == want.size


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pack_borders(dtype):
    """Zeros, the scale's borders and clamps, ties, and groups that hold an
    infinity or a NaN, each next to ordinary groups."""
    d = 384
    x = torch.zeros(10, d)
    x[0, 3] = 448.0
    x[1, 3] = 450.0
    x[2, 3] = 2.0 ** -130
    x[3, 3] = 3.0e38
    x[4, 130] = float("inf")
    x[5, 3] = float("nan")
    x[6, :5] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11, -0.0])
    x[7, 383] = -float("inf")
    x[8] = torch.linspace(-480, 480, d)
    x[4, :128] = 1.5
    x = x.to(DT[dtype])
    ck = _laga().pack8(x.to(DEV))
    want = ores.pack(as_f64(x))
    assert _same(ck.data.cpu().numpy(), want)
    v = as_f64(ck.unpack(torch.float32))
    assert _same(v, ores.unpack(want, d))
    assert np.isnan(v[4, 128:256]).all() and (v[4, :128] == 1.5).all() and (v[4, 256:] == 0).all()


def test_every_code_under_every_scale():
    """All finite codes under every scale byte, and NaN groups, decode to their
    values, in unpack and in the weight gradient (a row of dy that is one 1)."""
    laga = _laga()
    codes = np.array([b for b in range(256) if b & 0x7f != 0x7f], np.uint8)
    d = 256                                        # two groups: the codes, padded by zeros
    scales = np.concatenate([np.arange(127 + ores.E_MIN, 127 + ores.E_MAX + 1), [255]])
    buf = np.zeros((len(scales), ores.row_layout(d)[1]), np.uint8)
    buf[:, :len(codes)] = codes
    buf[:, 256:258] = scales[:, None]
    ck = laga.Checkpoint8(torch.from_numpy(buf).to(DEV), d)
    want = ores.unpack(buf, d)
    assert _same(as_f64(ck.unpack(torch.float32)), want)
    assert _same(as_f64(ck.unpack(torch.bfloat16)), want)
    for r in (0, 50, 110, 117, 124, 125, 180, len(scales) - 2):
        one = laga.Checkpoint8(ck.data[r:r + 1].contiguous(), d)
        dw = laga.weight_grad8(one, torch.ones(1, 8, dtype=torch.bfloat16, device=DEV))
        assert _same(as_f64(dw), np.repeat(want[r][:, None], 8, axis=1)), r


def _dw_case(rows, d, n, dtype, gain, seed=0):
    g = torch.Generator().manual_seed(seed + rows + 3 * d + 5 * n)
    buf = ores.pack(torch.randn(rows, d, generator=g).double().numpy() if rows else np.zeros((0, d)))
    dy = torch.randn(rows, n, generator=g).to(DT[dtype])
    gamma = 1 + 0.1 * torch.randn(d, generator=g) if gain else None
    return buf, dy, gamma


def _dw_check(rows, d, n, dtype, gain, seed=0):
    laga = _laga()
    buf, dy, gamma = _dw_case(rows, d, n, dtype, gain, seed)
    ck = laga.Checkpoint8(torch.from_numpy(buf).to(DEV), d)
    got = laga.weight_grad8(ck, dy.to(DEV), None if gamma is None else gamma.to(DEV))
    _sync()
    assert got.shape == (d, n) and got.dtype == torch.float32
    dw, size = ores.weight_grad(buf, d, as_f64(dy), None if gamma is None else as_f64(gamma))
    off = np.abs(as_f64(got) - dw)
    bound = (rows + 64) * 2.0 ** -23 * size
    worst = float(np.max(off / np.maximum(bound, 1e-300))) if size.any() else 0.0
    assert (off <= bound).all(), f"{rows}x{d}x{n} {dtype}: {worst:.2f} of its bound"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,d,n", [
    (1, 1, 1), (1, 128, 8), (2, 7, 3), (15, 129, 17), (63, 128, 64), (64, 256, 192), (65, 300, 193),
    (127, 512, 255), (128, 384, 256), (129, 512, 257), (333, 384, 200), (200, 640, 576),
    (1000, 1001, 100), (300, 2048, 513), (70, 7168, 40), (40, 100, 2000), (5000, 130, 72)])
def test_weight_grad(rows, d, n, dtype):
    _dw_check(rows, d, n, dtype, gain=False)
    _dw_check(rows, d, n, dtype, gain=True, seed=1)


def test_weight_grad_of_no_rows_is_zero():
    laga = _laga()
    ck = laga.Checkpoint8(torch.empty(0, laga._lib.ckpt_row_bytes(200), dtype=torch.uint8,
                                      device=DEV), 200)
    for dt in DT.values():
        dw = laga.weight_grad8(ck, torch.empty(0, 24, dtype=dt, device=DEV))
        _sync()
        assert dw.shape == (200, 24) and (dw == 0).all()


def test_weight_grad_repeats_bit_for_bit():
    laga = _laga()
    buf, dy, gamma = _dw_case(3000, 640, 200, "bf16", True)
    ck, dy, gamma = laga.Checkpoint8(torch.from_numpy(buf).to(DEV), 640), dy.to(DEV), gamma.to(DEV)
    a = laga.weight_grad8(ck, dy, gamma)
    for _ in range(3):
        assert torch.equal(a, laga.weight_grad8(ck, dy, gamma))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_weight_grad_non_finite(dtype):
    """A NaN group poisons its 128 channels, a NaN or infinity in dy its column;
    everything else is as without them."""
    laga = _laga()
    buf, dy, _ = _dw_case(200, 384, 72, dtype, False)
    ref = as_f64(laga.weight_grad8(laga.Checkpoint8(torch.from_numpy(buf).to(DEV), 384), dy.to(DEV)))
    buf[77, 384 + 1] = 255
    dy[199, 40], dy[0, 71] = float("nan"), float("inf")
    got = as_f64(laga.weight_grad8(laga.Checkpoint8(torch.from_numpy(buf).to(DEV), 384),
                                   dy.to(DEV)))
    assert np.isnan(got[128:256]).all() and np.isnan(got[:, 40]).all()
    assert not np.isfinite(got[:, 71]).any()
    rest = np.ones((384, 72), bool)
    rest[128:256] = rest[:, 40] = rest[:, 71] = False
    assert (got[rest] == ref[rest]).all()


def test_refusals_on_the_gpu():
    laga = _laga()
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    ck = laga.pack8(x)
    with pytest.raises(ValueError, match="contiguous"):
        laga.pack8(x[:, ::2])
    with pytest.raises(ValueError, match="rows"):
        laga.weight_grad8(ck, x[:7])
    with pytest.raises(ValueError, match="shape"):
        laga.weight_grad8(ck, x, gamma=torch.ones(63, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        laga.weight_grad8(ck, x.t().contiguous().t())
    with pytest.raises(TypeError):
        laga.weight_grad8(ck, x.half())
    with pytest.raises(ValueError):
        ck.unpack(torch.float16)
    with pytest.raises(ValueError, match="shape"):
        laga.Checkpoint8(ck.data[:, :128].contiguous(), 64)


@pytest.mark.parametrize("n", [512, 1536])
def test_weight_grad_step_by_step_at_full_size(n):
    """Several tiles for each pair of CTAs, as a 16384-token step has them.
    Column j of dy picks the tokens of one 128-token step, whose values are a
    number that tells neighbouring steps apart: every element is the exact
    sum of its step, whichever tiles, chains and fragments it went through."""
    laga = _laga()
    T, d = 16384, 7168
    step = torch.arange(T, device=DEV) // 128
    ck = laga.pack8((1 + (step % 8) / 8.0)[:, None].expand(T, d).contiguous())
    col = torch.arange(n, device=DEV)
    dy = ((col % 128)[None, :] == step[:, None]).to(torch.bfloat16)
    want = (128 * (1 + (col % 8) / 8.0)).expand(d, n)
    for _ in range(3):
        assert torch.equal(laga.weight_grad8(ck, dy), want)


@pytest.mark.parametrize("rows,d,n,dtype", [(16384, 7168, 1536, "bf16"), (16384, 7168, 576, "fp32"),
                                            (4096, 6000, 1000, "bf16"), (1000, 16384, 1026, "bf16"),
                                            (9000, 5001, 1530, "fp32")])
def test_weight_grad_at_full_size(rows, d, n, dtype):
    """Against the product in 64 bits on the GPU, with the bound of the small
    sizes; every run gives the same bits."""
    laga = _laga()
    g = torch.Generator(device=DEV).manual_seed(n)
    ck = laga.pack8(torch.randn(rows, d, generator=g, device=DEV))
    dy = torch.randn(rows, n, generator=g, device=DEV).to(DT[dtype])
    gamma = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    got = laga.weight_grad8(ck, dy, gamma)
    for _ in range(3):
        assert torch.equal(got, laga.weight_grad8(ck, dy, gamma))
    v = ck.unpack(torch.float32).double() * gamma.double()
    ref, size = v.t() @ dy.double(), v.abs().t() @ dy.double().abs()
    assert ((got.double() - ref).abs() <= (rows + 64) * 2.0 ** -23 * size).all()
    _sync()
