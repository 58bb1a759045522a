"""How exact the weight gradient from 8-bit checkpoints is over 16384 tokens.

All values and gradients are positive, so that every loss of the tensor
cores' accumulation points the same way and adds up.  What a sum may lose,
relative to itself:

* An MMA adds 16 products to an accumulator and cuts off what does not fit
  below its last place: less than one unit where the products are aligned and
  one where they are added, 2 * 2^-23 of the accumulator as it is by then.
* bf16 dy: a chain is 8 steps of 128 tokens, 64 MMAs.  The accumulator grows
  evenly, to within a tenth (an MMA's 16 products are a mean of 16 draws), so
  the 64 cuts are of (64 + 1) / 2 whole accumulators.
* fp32 dy: a chain is 2 steps, 8 MMAs for each of the three pieces, smallest
  first.  The two small pieces (2^-8 of dy and less) meet an accumulator of
  nearly 0 in the first step and of 1/2 in the second; the largest piece takes
  it from 0 to 1/2 and from 1/2 to 1: 16 * 0 + 8 / 4 + 16 / 2 + 8 * 3 / 4 = 16
  whole accumulators, and a tenth.
* The chains are added in fp32, rounded to nearest: 2^-24 of a sum that grows
  evenly, 16 chains or 64 (half of them, and one whole for what the work split
  adds and for the dy pieces beyond 24 bits).
"""

import numpy as np
import pytest
import torch

from laga_inputs import as_f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T, D = 16384, 7168
ULP = 2.0 ** -23
CUTS = {"bf16": 1.1 * 65 / 2, "fp32": 1.1 * 16}
CHAINS = {"bf16": T / 1024, "fp32": T / 256}
BOUND = {k: 2 * ULP * CUTS[k] + ULP / 2 * (CHAINS[k] / 2 + 1) for k in CUTS}


def _operands(n, dtype):
    g = torch.Generator(device=DEV).manual_seed(n)
    import sequence_latent_norm_gb300 as laga
    ck = laga.pack8(1 + torch.rand(T, D, generator=g, device=DEV))
    dy = 1 + torch.rand(T, n, generator=g, device=DEV)
    return laga, ck, dy.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _loss(got, v, dy):
    """The largest loss of an element, relative to its exact sum."""
    ref = v.t() @ dy.double()
    return float(((ref - got.double()).abs() / ref).max())


@pytest.mark.parametrize("n,dtype", [(1536, "bf16"), (576, "fp32"), (576, "bf16")])
def test_long_sums_lose_no_more_than_their_chains(n, dtype):
    laga, ck, dy = _operands(n, dtype)
    got = laga.weight_grad8(ck, dy)
    laga._lib.sync_check()
    loss = _loss(got, ck.unpack(torch.float32).double(), dy)
    print(f"weight gradient {n} {dtype}: loses {loss:.2e}, bound {BOUND[dtype]:.2e}")
    assert loss <= BOUND[dtype]


def test_the_bound_would_see_a_dropped_piece():
    """dy without what its third bf16 piece holds, in the exact sum."""
    _, ck, dy = _operands(576, "fp32")
    two = (dy.view(torch.int32) & ~0xff).view(torch.float32)     # 16 significand bits
    v = ck.unpack(torch.float32).double()[:, :256]
    full = v.t() @ dy.double()
    assert float(((full - v.t() @ two.double()) / full).min()) > BOUND["fp32"]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_bound_would_see_one_long_chain(dtype):
    """Sums whose accumulator is cut to fp32, once for an MMA's 16 products,
    from the first token to the last, and as the kernel's chains cut it."""
    _, ck, dy = _operands(64, dtype)
    v, dy = as_f64(ck.unpack(torch.float32)[:, :8]), as_f64(dy)
    if dtype == "bf16":
        pieces = [dy]
    else:
        parts = torch.from_numpy(dy).float()
        top = (parts.view(torch.int32) & ~0xffff).view(torch.float32)
        mid = ((parts - top).view(torch.int32) & ~0xffff).view(torch.float32)
        pieces = [as_f64(parts - top - mid), as_f64(mid), as_f64(top)]
    sums = [np.einsum("skc,skn->scn", v.reshape(-1, 16, 8), p.reshape(-1, 16, 64)) for p in pieces]

    def cut(a):      # to 24 significand bits, towards zero
        m, e = np.frexp(a)
        return np.ldexp(np.trunc(m * 2.0 ** 24) * 2.0 ** -24, e)

    def run(steps_a_chain):
        total, acc = np.zeros((8, 64), np.float32), np.zeros((8, 64))
        for step in range(T // 128):
            for s in sums:
                for k in range(step * 8, step * 8 + 8):
                    acc = cut(acc + s[k])
            if (step + 1) % steps_a_chain == 0:
                total, acc = total + acc.astype(np.float32), np.zeros((8, 64))
        return total

    ref = v.T @ dy
    chain = {"bf16": 8, "fp32": 2}[dtype]
    assert np.abs((run(chain) - ref) / ref).max() <= BOUND[dtype]
    assert ((ref - run(T // 128)) / ref).min() > BOUND[dtype]
