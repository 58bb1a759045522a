"""The weight gradient from 8-bit checkpoints before any CUDA call: sizes at
the top of their accepted range, and what is not a checkpoint."""

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from sequence_latent_norm_gb300.build import build_library
    build_library()
    import sequence_latent_norm_gb300 as pkg
    return pkg._lib


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("d", [1, 128, 7168, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_workspace_of_the_most_rows(lib, d, dtype):
    """A step is 128 rows: counts within the last one of 2^31 need as much as
    those in front of them, and an fp32 dy its three pieces."""
    n = 8
    sizes = [lib.ckpt_dw_workspace_bytes(rows, d, n, dtype)
             for rows in (2 ** 30, TOP - 200, TOP - 128, TOP - 127, TOP - 126, TOP - 1, TOP)]
    assert sizes[0] > 0 and sizes == sorted(sizes), sizes
    if dtype == "fp32":
        assert sizes[-1] >= 3 * TOP * n * 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only safe without a GPU")
def test_the_most_rows_need_their_workspace(lib):
    so, p = lib.load(), [0x10000 * (i + 1) for i in range(4)]
    for rows in (TOP - 127, TOP - 126, TOP):
        nb = lib.ckpt_dw_workspace_bytes(rows, 128, 8, "bf16")
        for ws, n in ((None, 0), (p[3], nb - 1)):
            assert so.laga_ckpt_dw(rows, 128, 8, 0, p[0], p[1], None, p[2], ws, n, None) == \
                lib.LAGA_ERR_WORKSPACE


def test_what_is_not_a_checkpoint_is_refused(lib):
    import sequence_latent_norm_gb300 as laga
    dy = torch.zeros(4, 8, dtype=torch.bfloat16)
    for ck in (None, dy, torch.zeros(4, 144, dtype=torch.uint8)):
        with pytest.raises(TypeError, match="Checkpoint8"):
            laga.weight_grad8(ck, dy)
