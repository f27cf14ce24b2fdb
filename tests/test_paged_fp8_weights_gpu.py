"""Attention over a paged cache in 8 bits: weights far below their row's largest, of which there are many. What they give
together is a dimension of the output that nothing else reaches, so that its error is theirs."""

import numpy as np
import pytest
import torch

from linear_attention_ssm_step_gb300 import kda
from paged_fp8_cases import Attention, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def sink(new, n, below, D, seed):
    """A first key that takes most of the weight, and n others whose weights scatter around 2^-below of it, by half a power
    of two either way. The first key's value is 1 in dimension 5, the others' in dimension 3."""
    a = Attention(new, [n + x for x in new], 4, 1, D, 64, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    a.q[:] = 0
    a.q[:, :, :2] = 1.0
    for t, s in ((a.k, a.ks), (a.v, a.vs)):
        t[:], s[:] = 0, 1.0
    codes = torch.randint(0, 0x39, a.k.shape[:3], generator=gen) | torch.randint(0, 2, a.k.shape[:3], generator=gen) << 7
    a.k[..., 1] = codes.to(torch.uint8)  # numbers from -1 to 1, many of them small
    a.ks[:] = float(np.log(2)) / 2 / a.scale
    a.v[..., 3] = 0x38  # 1
    for r in range(len(new)):
        page = int(a.table[r, 0])
        a.k[page, :16, 0, 1] = 0
        a.k[page, 0, 0, 0] = 0x50   # 8
        a.ks[page, 0, 0] = below * float(np.log(2)) / 8 / a.scale
        a.v[page, 0, 0, 3] = 0
        a.v[page, 0, 0, 5] = 0x38
    return a


@pytest.mark.parametrize("below", [19.5, 23.5, 24.5, 28.0])
@pytest.mark.parametrize("D,new", [(128, [1]), (64, [1]), (128, [2, 1]), (128, [8, 8]), (128, [60]), (64, [40, 50])])
def test_many_weights_far_below_the_largest(dev, D, new, below):
    """Relative to what the small weights give: each is rounded to fp16, by 2^-11 of itself or by half a step of fp16's
    subnormals, 2^-25, where the row's largest is 2^10 or more in the kernel for few rows and 2^6 in the one for chunks
    (2^-35 and 2^-31 of it; the smallest of them is 2^-(below + 1/2) of it). A score's error e moves a weight, and the sum of
    all, by e. Sums over n keys: (n + 64) 2^-23. The output is rounded to bf16, by 2^-8 at most."""
    n = 20000
    a = sink(new, n, below, D, seed=60)
    out, lse = a.run(dev, kda)
    o, z, A, S, count, _ = a.oracle()
    few = -(-sum(new) // len(new)) * 4 <= 32
    e = ((D + 8) * 2.0 ** -23 + 2.0 ** -22) * np.max(S)
    rel = 2.0 ** -11 + 2.0 ** (below + 0.5 - (35 if few else 31)) + 2 * e + 2.0 ** -21 + (n + 64) * 2.0 ** -23 + 2.0 ** -8
    want = o[..., 3]
    assert want.min() > 0.5 * n * 2.0 ** -below / (1 + n * 2.0 ** -below)
    err = np.abs(f64(out)[..., 3] / want - 1)
    assert err.max() <= rel, f"{err.max():.2e}, bound {rel:.2e}"
    a.check(out, lse)
