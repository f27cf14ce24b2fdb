"""Inputs and bounds shared by the paged-attention tests.

Bounds (derived, element-wise):
  * rope: the result is rounded to bf16 once, 2^-8 of it (8 significant bits:
    half an ulp is up to 2^-8 of the value). Before that, fp32: the phase enters with
    2^-25 of a turn at most (its upper 32 bits as fp32), pi 2^-24 radians; sine
    and cosine are good to 2 ulps, the scale and the two products and their
    difference round once each: together below 2^-20 mscale (|x| + |y|).
    bf16 subnormals (below 2^-126) are not drawn.
  * attention: with w_j the weights, A = sum w_j |v_j| and S the largest scale
    sum_c |q_c k_c| of the row's keys, n the keys seen:
      - a weight is rounded to bf16 before it meets v, its sum is not: 2^-8 A;
      - a score carries its fp32 sum's error, (D + 8) 2^-23 S allowing a
        truncating adder, and 2^-22 S for the scaling, the difference to the
        maximum and the exponential's argument; a weight and the sum of the
        weights each move by that much, relatively: 2 e A;
      - exp itself, 2^-21 A with its sum, and the fp32 accumulation over n keys
        (truncating, blocks joined): (n + 64) 2^-23 A;
      - out is rounded to bf16 once: 2^-8 |o|.
    lse: the score's error e, the sum's (n + 64) 2^-23, exp and log 2^-20, its
    rounding 2^-22 |lse|.
"""

import numpy as np
import torch

import oracle


def rope_bound(ref, x, partner, mscale):
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * abs(mscale) * (np.abs(x) + np.abs(partner)) + 1e-30


def attention_bounds(out, lse, A, S, count, D):
    e = ((D + 8) * 2.0 ** -23 + 2.0 ** -22) * S
    sums = ((count + 64) * 2.0 ** -23)[:, None]
    rel = 2.0 ** -8 + 2 * e + 2.0 ** -21 + sums
    tol = rel[:, :, None] * A + 2.0 ** -8 * np.abs(out) + 1e-30
    safe = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return tol, e + sums + 2.0 ** -20 + 2.0 ** -22 * safe


def ints(x, device):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


def cache(pages, page, heads, dim, order, gen):
    """bf16 (k, v), each viewed [pages, page, heads, dim], stored in one of the layouts:
    "thd" tokens before heads, "htd" heads before tokens, "pair" keys and values of a page side by
    side, "padded" rows with gaps, "odd" rows off a 16-byte boundary."""
    def rand(*shape):
        return torch.randn(shape, generator=gen).to(torch.bfloat16)
    if order == "thd":
        return rand(pages, page, heads, dim), rand(pages, page, heads, dim)
    if order == "htd":
        return rand(pages, heads, page, dim).transpose(1, 2), rand(pages, heads, page, dim).transpose(1, 2)
    if order == "pair":
        both = rand(pages, 2, page, heads, dim)
        return both[:, 0], both[:, 1]
    if order == "padded":
        return rand(pages, page, heads, dim + 16)[..., :dim], rand(pages, page + 2, heads, dim)[:, :page]
    if order == "odd":
        return rand(pages, page, heads, dim + 3)[..., 1:dim + 1], rand(pages, page, heads, dim + 1)[..., :dim]
    raise ValueError(order)


def to_device(t, dev):
    """The same values on the device with the same strides."""
    base = t if t._base is None else t._base
    flat = base.flatten() if base.is_contiguous() else base.contiguous().flatten()
    return flat.to(dev).as_strided(t.shape, t.stride(), t.storage_offset())


class Attention:
    """One attention problem on the CPU: ragged requests over scattered pages."""

    def __init__(self, new, kv, Hq, Hkv, D, page, window=0, order="thd", seed=0, scale=None, extra_width=0,
                 fused_q=False):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.Hq, self.Hkv, self.D, self.page = list(new), list(kv), Hq, Hkv, D, page
        self.window, self.scale = window, D ** -0.5 if scale is None else scale
        R = len(new)
        used = [-(-x // page) if x > 0 else 0 for x in kv]
        pages = sum(used) + 3
        perm = torch.randperm(pages, generator=gen).tolist()
        self.k, self.v = cache(pages, page, Hkv, D, order, gen)
        self.table = np.full((R, max([1] + used) + extra_width), -7, dtype=np.int64)
        for r, u in enumerate(used):
            self.table[r, :u] = [perm.pop() for _ in range(u)]
        self.unused = perm
        T = sum(new)
        if fused_q:
            self.q = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(torch.bfloat16)[:, :Hq]
        else:
            self.q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
        self.cu = np.concatenate([[0], np.cumsum(new)])

    def f64(self, t):
        return t.double().numpy()

    def poison(self):
        """NaN in everything no row may read: the rest of each last page, and pages no request owns."""
        for t in (self.k, self.v):
            for p in self.unused:
                t[p] = float("nan")
            for r, x in enumerate(self.kv):
                if x > 0 and x % self.page:
                    t[int(self.table[r, x // self.page]), x % self.page:] = float("nan")
        return self

    def oracle(self):
        k, v = np.nan_to_num(self.f64(self.k)), np.nan_to_num(self.f64(self.v))
        return oracle.paged_attention(self.f64(self.q), k, v, self.table, self.cu, self.kv, self.scale, self.window)

    def run(self, dev, kda, workspace=None, error_word=None, out=None, lse=None, **kw):
        args = (to_device(self.q, dev), to_device(self.k, dev), to_device(self.v, dev), ints(self.table, dev),
                ints(self.cu, dev), ints(self.kv, dev))
        T = self.q.shape[0]
        if out is None:
            out = torch.full((T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.full((T, self.Hq), 7.0, dtype=torch.float32, device=dev)
        kda.kda_paged_attention(*args, out=out, lse=lse, scale=self.scale, window=self.window, workspace=workspace,
                                error_word=error_word, **kw)
        return out, lse

    def check(self, out, lse, ref=None):
        o, z, A, S, count, _ = self.oracle() if ref is None else ref
        tol, ztol = attention_bounds(o, z, A, S, count, self.D)
        got, gz = out.double().cpu().numpy(), lse.double().cpu().numpy()
        seen = ~np.isnan(z)
        err = np.abs(got - o)[seen] / tol[seen]
        assert np.isfinite(got[seen]).all(), "out has a value that is not finite"
        assert err.size == 0 or err.max() <= 1.0, f"out: {err.max():.3f} x its bound"
        empty = np.isneginf(z)
        assert (got[empty] == 0).all() and np.isneginf(gz[empty]).all()
        full = seen & ~empty
        zerr = np.abs(gz - np.where(full, z, 0))[full] / ztol[full]
        assert zerr.size == 0 or zerr.max() <= 1.0, f"lse: {zerr.max():.3f} x its bound"
        assert (got[~seen] == 7).all() and (gz[~seen] == 7).all(), "a row no request covers was written"
