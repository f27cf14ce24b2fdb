"""Attention over a paged cache in 8 bits at the ends of what scores can be, and of what tables can be."""

import numpy as np
import pytest
import torch

from linear_attention_ssm_step_gb300 import kda
from paged_cases import ints
from paged_fp8_cases import Attention, cache, f64

pytestmark = pytest.mark.gpu

CHUNKS = ([130, 1, 77], [500, 129, 77])   # the kernel for chunks
FEW = ([1, 1, 3], [300, 90, 1000])        # the kernel for few rows


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,shape,power", [(128, FEW, 100), (64, FEW, 100), (80, FEW, 100), (80, CHUNKS, 100),
                                           (128, FEW, 17), (128, CHUNKS, 17), (64, CHUNKS, 17)])
def test_scores_of_any_size(dev, D, shape, power, sign):
    """All scores far below, or far above, zero, the first key's the largest by a seventh or more: it takes all the weight.
    Its value comes out whole (four bits of fraction at most, and the weights' quotient is good to 2^-10), and lse is its
    score, which the fp32 sum, the scaling and the logarithm move by (D + 8) 2^-23 + 2^-20 of it at most. The kernel for
    chunks takes scores below 2^23 in magnitude (power 17: 2^22.8)."""
    a = Attention(*shape, 4, 2, D, 16, seed=90)
    a.q[:] = 0
    a.q[:, :, 1] = 2.0 ** min(power, 60)
    a.k[:], a.ks[:] = 0, 2.0 ** max(power - 60, 0)
    a.k[..., 1] = 0xFE if sign < 0 else 0x78  # -448, 256
    first = 0xF8 if sign < 0 else 0x7E        # -256, 448
    for r in range(3):
        a.k[int(a.table[r, 0]), 0, :, 1] = first
    out, lse = a.run(dev, kda)
    score = a.scale * 2.0 ** power * (-256 if sign < 0 else 448)
    off = np.abs(f64(lse) / score - 1).max()
    assert off <= (D + 8) * 2.0 ** -23 + 2.0 ** -20
    _, v = a.values()
    for r in range(3):
        want = np.repeat(v[int(a.table[r, 0]), 0], 2, axis=0)
        assert np.array_equal(f64(out)[a.cu[r]:a.cu[r + 1]], np.broadcast_to(want, (a.new[r], 4, D)))


@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64, 80])
def test_scores_below_all_numbers(dev, D, shape):
    """Queries, key scales and a scale so small that their product is below fp32's smallest number: every seen key has the
    same weight, and the masked ones none."""
    a = Attention(*shape, 4, 2, D, 16, window=60, seed=91, scale=1e-30).poison()
    a.q *= 2.0 ** -60
    a.ks[torch.isfinite(a.ks)] = 2.0 ** -40
    a.check(*a.run(dev, kda))


def test_a_table_too_wide_for_the_kernel_of_few_rows(dev):
    """One token of 512 heads over 128, and a table of 1.2 billion tokens: two items of few rows (a token each at most, of
    9.6 million units) for 128 heads would pass 32 bits, one item of chunks does not. The call gives what the kernel for chunks does (which the second call takes, its rows padded to 40: one
    unit of keys, so that no bit depends on how the work is shared out)."""
    H, D, page, width, kv = 128, 64, 4096, 300000, 100
    gen = torch.Generator().manual_seed(92)
    sides = [x.to(dev) for x in (*cache(2, page, H, D, "thd", gen), *cache(2, page, H, D, "thd", gen))]
    kc, ks, vc, vs = sides
    q = torch.randn((40, 4 * H, D), generator=gen).to(torch.bfloat16).to(dev)
    table = torch.full((1, width), -1, dtype=torch.int32, device=dev)
    table[0, 0] = 1
    got = []
    for rows, columns in ((1, width), (40, 1)):
        lse = torch.zeros((rows, 4 * H), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention_fp8(q[:rows], kc, vc, ks, vs, table[:, :columns], ints([0, 1], dev), ints([kv], dev),
                                          lse=lse)
        got.append((out[0], lse[0]))
    assert torch.equal(got[0][1], got[1][1]) and torch.equal(got[0][0], got[1][0])
