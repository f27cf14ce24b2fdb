"""Inputs and bounds shared by the tests of the paged cache held in 8 bits.

Bounds (derived, element-wise):
  * a code is its number over the scale rounded to the nearest: half a step, which is 2^(E - 4) in the binade
    [2^E, 2^(E + 1)), 2^-10 among the subnormals (E4M3 has 3 bits of fraction). Values enter without any arithmetic but
    the exact scaling, so their codes are equal to the oracle's. Keys carry the fp32 turn before that, off by
    KEY_ERROR * mscale (|x| + |y|): a sine or cosine off by 2^-20.5 in the fast form, its angle by 2^-25 of a turn and a
    rounding (pi 2^-24 + pi 2^-24, together below 2^-21), then three roundings of the products and their sum, 2^-22:
    below 2^-19.
  * a scale may differ by a step of 2 only where the largest key is within KEY_ERROR of a border.
  * attention: as paged_cases.py derives for the 16-bit cache (A, S, n, e as there), over the exact values code * scale,
    with two changes:
      - a weight times its key's value scale is rounded to fp16, not bf16, before it meets v: 2^-11 A. They are kept so
        that the largest of a row is 2^6 or more, and fp16's subnormals round by 2^-25: 2^-31 of that largest for each
        key seen, times |code| <= 448, and a scale s has a code of 224 or more in its block, so |v| >= 224 s in it:
        2^-30 max |v| each, 2^-29 with room. For few rows the fp16 number goes on as three E4M3 numbers, each 2^5 below
        the one before, the last off by half its subnormals' step: 2^-20 where the largest of a row is 2^4 or more, so
        2^-24 instead of 2^-31, 2^-22 max |v| each with room;
      - on the tensor cores a query number below 2^-9 of its head's largest is off by 2^-17 of that: a score by
        2^-17 scale max_c |q_c| max_j sum_c |k_jc|. Added to e.
"""

import numpy as np
import torch

import oracle
from paged_cases import ints, to_device

KEY_ERROR = 2.0 ** -19
TOKENS = 16


def half_step(x):
    """Half the distance of E4M3 numbers around |x|."""
    x = np.maximum(np.abs(x), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(x)) - 4)


def in_order(t, order, pad):
    """The same [pages, tokens, heads, ...] values in another layout: "thd", "htd" heads before tokens, "padded" rows
    with gaps."""
    if order == "htd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if order in ("padded", "odd"):
        shape = list(t.shape)
        shape[-1] += pad
        base = torch.zeros(shape, dtype=t.dtype)
        base[..., :t.shape[-1]] = t
        return base[..., :t.shape[-1]]
    return t


def cache(pages, page, heads, dim, order, gen, spread=0.5):
    """(codes, scales) of one side, blocks of different sizes, quantised by their largest value."""
    blocks = -(-page // TOKENS)
    x = torch.randn((pages, page, heads, dim), generator=gen).double().numpy()
    size = np.exp(spread * torch.randn((pages, blocks, heads), generator=gen).double().numpy())
    block = np.arange(page) // TOKENS
    x = x * size[:, block][..., None]
    top = np.stack([np.abs(x[:, block == b]).max(axis=(1, 3)) for b in range(blocks)], axis=1)
    scale = 2.0 ** np.ceil(np.log2(top / 448.0))
    codes = oracle.e4m3_encode(x / scale[:, block][..., None])
    pad = {"padded": 16, "odd": 3}.get(order, 0)
    codes = in_order(torch.from_numpy(np.ascontiguousarray(codes)), order, pad)
    scale = torch.from_numpy(scale).float()
    if order == "odd":  # scales between others
        wide = torch.zeros(pages, blocks, heads, 2)
        wide[..., 1] = scale
        scale = wide[..., 1]
    elif order == "htd":
        scale = scale.transpose(1, 2).contiguous().transpose(1, 2)
    return codes, scale


def f64(t):
    return t.double().cpu().numpy()


class Attention:
    """One attention problem on the CPU: ragged requests over scattered pages of a cache in 8 bits."""

    def __init__(self, new, kv, Hq, Hkv, D, page, window=0, order="thd", seed=0, scale=None, q_spread=0.0):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.Hq, self.Hkv, self.D, self.page = list(new), list(kv), Hq, Hkv, D, page
        self.window, self.scale = window, D ** -0.5 if scale is None else scale
        used = [-(-x // page) if x > 0 else 0 for x in kv]
        pages = sum(used) + 3
        perm = torch.randperm(pages, generator=gen).tolist()
        self.k, self.ks = cache(pages, page, Hkv, D, order, gen)
        self.v, self.vs = cache(pages, page, Hkv, D, order, gen, spread=1.0)
        self.table = np.full((len(new), max([1] + used)), -7, dtype=np.int64)
        for r, u in enumerate(used):
            self.table[r, :u] = [perm.pop() for _ in range(u)]
        self.unused = perm
        T = sum(new)
        q = torch.randn((T, Hq, D), generator=gen)
        self.q = (q * torch.exp(q_spread * torch.randn((T, Hq, D), generator=gen))).to(torch.bfloat16)
        self.cu = np.concatenate([[0], np.cumsum(new)])

    def poison(self):
        """NaN codes in everything no row may read, and scales that are not numbers where no block is read."""
        for t, s in ((self.k, self.ks), (self.v, self.vs)):
            for p in self.unused:
                t[p], s[p] = 0x7F, float("nan")
            for r, x in enumerate(self.kv):
                if x > 0 and x % self.page:
                    p, at = int(self.table[r, x // self.page]), x % self.page
                    t[p, at:] = 0xFF
                    s[p, -(-at // TOKENS):] = float("nan")
        return self

    def values(self):
        return tuple(np.nan_to_num(oracle.dequantized(c.numpy(), s.numpy())) for c, s in ((self.k, self.ks), (self.v, self.vs)))

    def oracle(self):
        k, v = self.values()
        return oracle.paged_attention(f64(self.q), k, v, self.table, self.cu, self.kv, self.scale, self.window)

    def run(self, dev, kda, workspace=None, error_word=None, out=None, lse=None, **kw):
        T = self.q.shape[0]
        if out is None:
            out = torch.full((T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device=dev)
        if lse is None:
            lse = torch.full((T, self.Hq), 7.0, dtype=torch.float32, device=dev)
        kda.kda_paged_attention_fp8(*(to_device(t, dev) for t in (self.q, self.k, self.v, self.ks, self.vs)),
                                    ints(self.table, dev), ints(self.cu, dev), ints(self.kv, dev), out=out, lse=lse,
                                    scale=self.scale, window=self.window, workspace=workspace, error_word=error_word, **kw)
        return out, lse

    def bounds(self, ref):
        out, lse, A, S, count, _ = ref
        k, v = self.values()
        e = ((self.D + 8) * 2.0 ** -23 + 2.0 ** -22) * S
        e = e + 2.0 ** -17 * self.scale * np.abs(f64(self.q)).max(-1) * np.abs(k).sum(-1).max(initial=0.0)
        sums = ((count + 64) * 2.0 ** -23)[:, None]
        rel = 2.0 ** -11 + 2 * e + 2.0 ** -21 + sums
        few = -(-self.q.shape[0] // len(self.kv)) * (self.Hq // self.Hkv) <= 32
        small = (count * 2.0 ** (-22 if few else -29) * np.abs(v).max(initial=0.0))[:, None, None]
        tol = rel[:, :, None] * A + 2.0 ** -8 * np.abs(out) + small + 1e-30
        safe = np.where(np.isfinite(lse), np.abs(lse), 0.0)
        return tol, e + sums + 2.0 ** -20 + 2.0 ** -22 * safe

    def check(self, out, lse, ref=None):
        ref = self.oracle() if ref is None else ref
        o, z = ref[:2]
        tol, ztol = self.bounds(ref)
        got, gz = f64(out), f64(lse)
        seen = ~np.isnan(z)
        assert np.isfinite(got[seen]).all(), "out has a value that is not finite"
        err = np.abs(got - o)[seen] / tol[seen]
        assert err.size == 0 or err.max() <= 1.0, f"out: {err.max():.3f} x its bound"
        empty = np.isneginf(z)
        assert (got[empty] == 0).all() and np.isneginf(gz[empty]).all()
        full = seen & ~empty
        zerr = np.abs(gz - np.where(full, z, 0))[full] / ztol[full]
        assert zerr.size == 0 or zerr.max() <= 1.0, f"lse: {zerr.max():.3f} x its bound"
        assert (got[~seen] == 7).all() and (gz[~seen] == 7).all(), "a row no request covers was written"
