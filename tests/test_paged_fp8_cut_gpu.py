"""The append to a cache in 8 bits where rows of a block are not stored in the middle of it: the others are still taken
together, whichever part of the grid has them. Bounds: paged_fp8_cases.py."""

import numpy as np
import pytest
import torch

from linear_attention_ssm_step_gb300 import kda
from test_paged_fp8_gpu import Append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


CASES = [
    # lengths, starts, Hq, Hkv, D, rot, page, order, share of the rows that are not stored
    ([64], [0], 2, 2, 128, 64, 16, "thd", 0.2),
    ([40, 7, 100, 16, 1], [3, 12, 0, 16, 9], 4, 2, 64, 64, 32, "htd", 0.5),
    ([90], [5], 3, 1, 80, 16, 20, "odd", 0.3),            # pages that end in a short block, an element at a time
    ([700, 300], [11, 0], 2, 1, 128, 0, 64, "thd", 0.1),  # a CTA looks for runs in two rows
    ([1800], [1], 2, 9, 64, 32, 16, "thd", 0.8),          # in four
    ([3000, 2000], [7, 30], 2, 2, 64, 64, 32, "thd", 0.3),
    ([8800], [4], 1, 1, 128, 64, 64, "padded", 0.5),      # in sixteen
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_blocks_with_rows_that_are_not_stored(dev, case):
    lengths, starts, Hq, Hkv, D, rot, page, order, share = CASES[case]
    a = Append(lengths, starts, Hq, Hkv, D, rot, False, page, order, seed=70 + case)
    rng = np.random.default_rng(case)
    limit = a.kc.shape[0] * a.page
    kinds = rng.integers(0, 3, len(a.pos))
    for t in np.flatnonzero(rng.random(len(a.pos)) < share):
        if kinds[t] == 0:
            a.pos[t] = -1
        else:
            a.slots[t] = -1 if kinds[t] == 1 else limit + int(rng.integers(0, 100))
    ref = a.oracle()
    assert ref[4] == kda.KDA_ERR_PAGES
    got = a.run(dev)
    a.check(*got, ref)
    again = a.run(dev)
    assert all(torch.equal(x, y) for x, y in zip([got[0], *got[1]], [again[0], *again[1]]))


def test_a_block_of_its_first_and_last_row_alone(dev):
    """Rows 0 and 15 of a block, each in turn the larger one, with the fourteen between them left out: one scale for both,
    and the tokens between keep their codes."""
    for large in (0, 15):
        a = Append([16], [0], 2, 2, 128, 0, False, 16, "thd", seed=80)
        a.k[large] *= 64
        a.v[large] *= 64
        a.slots[1:15] = -1
        ref = a.oracle()
        out, sides, bits = a.run(dev)
        a.check(out, sides, bits, ref)
        page = int(a.slots[0]) // 16
        assert torch.equal(sides[1][page, 1:15].cpu(), a.vc[page, 1:15])
