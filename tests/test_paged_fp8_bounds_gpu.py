"""Attention over a paged cache in 8 bits within bounds made for each row and kernel.

With A, S, n and e as paged_cases.py has them:
  * on the CUDA cores everything is fp32: 2 e A, 2^-21 A of the exponentials, (n + 64) 2^-23 A of the sums, 2^-8 |o| of the
    output's rounding; lse as there.
  * on the tensor cores, besides:
      - a query number below 2^-9 of its head's largest is off by less than 2^-17 of that: a score by 2^-17 scale max |q|
        times the sum of |k_jc| over those numbers alone, of the keys that the row sees;
      - y = f s + log2 vs, its reference and their difference round three times at up to M = S log2 e + max |log2 vs| + 16
        (the largest weight, and a row's distance to it below which nothing counts): 3 ln 2 2^-24 M < 2^-22 M of a weight;
      - a weight is rounded to fp16: 2^-11 A, or half a step of its subnormals, 2^-25, where the row's largest weight times
        value scale vs* is 2^10 at the least for few rows, 2^6 for chunks: 2^-35 or 2^-31 of that largest. Times a code, 448
        at most, over the sum of the weights, at least that of the largest: 448 vs* 2^-35, and 224 vs* is below the
        largest |v| of its block, so 2^-34 (2^-30) max |v| a key;
      - lse = m ln 2 + ln l, both of M at most, the logarithm good to 2^-22 of itself: 2^-21 M.
"""

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


class Close(Attention):
    def on_tensor_cores(self):
        return self.D in (64, 128) and self.page >= 16 and self.page & (self.page - 1) == 0 and \
            all(x % 16 == 0 for t in (self.k, self.v) for x in t.stride()[:3])

    def split(self):
        """[rows, heads]: what the split of the queries moves a score by."""
        q, (k, _) = f64(self.q), self.values()
        top = np.abs(q).max(-1, keepdims=True)
        small = (np.abs(q) < 2.0 ** -9 * top).astype(float)
        off = np.zeros(q.shape[:2])
        g = self.Hq // self.Hkv
        for r, n in enumerate(self.new):
            j = np.arange(max(self.kv[r], 0))
            keys = np.abs(k[self.table[r, j // self.page], j % self.page])  # [kv, Hkv, D]
            for t in range(n):
                pos = self.kv[r] - n + t
                lo = max(0, pos - self.window + 1) if self.window else 0
                seen = keys[lo:pos + 1]
                if len(seen):
                    row = self.cu[r] + t
                    for h in range(self.Hq):
                        off[row, h] = (seen[:, h // g] @ small[row, h]).max()
        return 2.0 ** -17 * self.scale * top[..., 0] * off

    def bounds(self, ref):
        out, lse, A, S, count, _ = ref
        _, v = self.values()
        e = ((self.D + 8) * 2.0 ** -23 + 2.0 ** -22) * S
        sums = ((count + 64) * 2.0 ** -23)[:, None]
        safe = np.where(np.isfinite(lse), np.abs(lse), 0.0)
        ztol = sums + 2.0 ** -20 + 2.0 ** -22 * safe
        rel = 2.0 ** -21 + sums
        small = 0.0
        if self.on_tensor_cores():
            vs = f64(self.vs)
            M = S / np.log(2) + np.abs(np.log2(vs[np.isfinite(vs)])).max() + 16
            e = e + self.split() + 2.0 ** -22 * M
            ztol = ztol + 2.0 ** -21 * M
            rel = rel + 2.0 ** -11
            few = -(-self.q.shape[0] // len(self.kv)) * (self.Hq // self.Hkv) <= 32
            small = (count * 2.0 ** (-34 if few else -30) * np.abs(v).max(initial=0.0))[:, None, None]
        return (rel + 2 * e)[:, :, None] * A + 2.0 ** -8 * np.abs(out) + small + 1e-30, ztol + e


CASES = [
    # new, kv, Hq, Hkv, D, page, window, order
    ([1] * 6, [1, 128, 129, 1000, 40, 3000], 8, 2, 128, 64, 0, "thd"),
    ([4, 4, 1], [300, 90, 2000], 6, 2, 64, 16, 0, "htd"),
    ([8, 3], [700, 1100], 4, 1, 128, 32, 200, "thd"),
    ([130, 1, 77], [500, 129, 77], 4, 2, 128, 64, 0, "thd"),
    ([60, 90], [900, 400], 8, 1, 64, 16, 100, "padded"),
    ([5, 200], [2, 190], 4, 2, 128, 16, 0, "thd"),   # rows that see none
    ([20, 1], [60, 777], 4, 2, 96, 24, 0, "thd"),    # the CUDA cores
    ([6, 1], [50, 900], 2, 1, 80, 20, 9, "odd"),
    ([4], [170], 2, 2, 256, 1, 0, "thd"),
    ([3, 40], [40, 400], 6, 1, 5, 16, 0, "thd"),
    ([3, 40], [40, 400], 4, 2, 128, 24, 0, "thd"),
]


@pytest.mark.parametrize("q_spread", [0.0, 1.5, 4.0])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_within_bounds_of_its_rows(dev, case, q_spread):
    new, kv, Hq, Hkv, D, page, window, order = CASES[case]
    a = Close(new, kv, Hq, Hkv, D, page, window, order, seed=200 + case, q_spread=q_spread).poison()
    a.check(*a.run(dev, kda))


@pytest.mark.parametrize("case", [0, 1, 3, 4, 6])
def test_scales_far_apart_within_bounds_of_its_rows(dev, case):
    new, kv, Hq, Hkv, D, page, window, order = CASES[case]
    a = Close(new, kv, Hq, Hkv, D, page, window, order, seed=300 + case)
    gen = torch.Generator().manual_seed(301)
    a.vs *= 2.0 ** torch.randint(-30, 31, a.vs.shape, generator=gen).float()
    a.ks[::3] = 2.0 ** -40
    a.check(*a.run(dev, kda))
