"""The paged cache held in 8 bits on the GPU against the fp64 oracle: the append,
reading back, attention, and a step of all of them. Bounds and their derivation:
paged_fp8_cases.py. Codes and scales that no arithmetic precedes must be equal."""

import numpy as np
import pytest
import torch

import oracle
from linear_attention_ssm_step_gb300 import kda
from paged_cases import ints, rope_bound, to_device
from paged_fp8_cases import KEY_ERROR, TOKENS, Attention, cache, f64, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda:0")


def err_word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------- append

def partner_sizes(x, rot, interleaved):
    """|x| + |its pair's other number|, for the bound of a turn."""
    y = np.abs(x)
    out = y.copy()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[..., a] = out[..., b] = y[..., a] + y[..., b]
    return out


class Append:
    """Rows of requests at consecutive slots from `starts` on (tokens into pages of their own), one call."""

    def __init__(self, lengths, starts, Hq, Hkv, D, rot, interleaved, page, order, seed, mscale=1.0, fused=False,
                 size=1.0):
        gen = torch.Generator().manual_seed(seed)
        T = sum(lengths)
        self.rot, self.interleaved, self.mscale, self.page = rot, interleaved, mscale, page
        rows = torch.randn((T, Hq + 2 * Hkv, D), generator=gen) * torch.exp(torch.randn((T, 1, 1), generator=gen)) * size
        if fused:
            rows = rows.to(torch.bfloat16)
            self.q, self.k, self.v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = (x.to(torch.bfloat16).contiguous() for x in rows.split((Hq, Hkv, Hkv), dim=1))
        pages = sum(-(-(n + s % page) // page) for n, s in zip(lengths, starts)) + 2
        perm = torch.randperm(pages, generator=gen).numpy()
        slots, pos, at = [], [], 0
        for n, s in zip(lengths, starts):
            i = s % page + np.arange(n)
            slots.append(perm[at + i // page] * page + i % page)
            pos.append(s + np.arange(n))
            at += -(-(n + s % page) // page)
        self.slots, self.pos = np.concatenate(slots), np.concatenate(pos)
        self.kc, self.ks = cache(pages, page, Hkv, D, order, gen)
        self.vc, self.vs = cache(pages, page, Hkv, D, order, gen)
        self.freqs = kda.rope_freqs(rot, 10000.0, device="cpu") if rot else torch.zeros(0, dtype=torch.int64)

    def oracle(self):
        turns = [int(x) % (1 << 64) for x in self.freqs.tolist()]
        return oracle.rope_append_fp8(f64(self.q), f64(self.k), f64(self.v), self.pos, self.slots, turns, self.kc.numpy(),
                                      self.vc.numpy(), f64(self.ks), f64(self.vs), self.interleaved, self.mscale)

    def run(self, dev, q_out=None):
        put = lambda t: to_device(t, dev)  # noqa: E731
        q, sides = put(self.q), [put(t) for t in (self.kc, self.vc, self.ks, self.vs)]
        err = err_word(dev)
        out = q if q_out == "in place" else torch.full(tuple(self.q.shape), 7.0, dtype=torch.bfloat16, device=dev)
        got = kda.kda_rope_append_fp8(q, put(self.k), put(self.v), ints(self.pos, dev), ints(self.slots, dev),
                                      self.freqs.to(dev), *sides, q_out=out, interleaved=self.interleaved,
                                      mscale=self.mscale, error_word=err)
        assert got is out
        return out, sides, int(err.item())

    def check(self, out, sides, bits, ref=None):
        qo, keys, values, written, err = self.oracle() if ref is None else ref
        assert bits == err
        q = f64(self.q)
        other = partner_sizes(q, self.rot, self.interleaved) - np.abs(q)
        tol = rope_bound(qo, q, other, self.mscale)
        assert (np.abs(f64(out) - qo)[written] <= tol[written]).all()
        # values: every code and scale
        codes, scales, _, kind = values
        assert np.array_equal(f64(sides[3]), scales)
        assert np.array_equal(sides[1].cpu().numpy(), codes)
        # keys: within the rounding of a code and the error of the turn
        codes, scales, exact, kind = keys
        got, got_scale = sides[0].cpu().numpy(), f64(sides[2])
        assert np.array_equal(got[kind == 0], codes[kind == 0]), "a code that no row touches was written"
        turn = np.zeros(exact.shape)
        k = partner_sizes(f64(self.k), self.rot, self.interleaved)
        for t, slot in enumerate(self.slots):
            if kind[slot // self.page, slot % self.page].any() if 0 <= slot < kind.shape[0] * self.page else False:
                turn[slot // self.page, slot % self.page] = KEY_ERROR * self.mscale * k[t]
        ratio = got_scale / scales
        assert np.isin(ratio, (0.5, 1.0, 2.0)).all()
        assert (ratio != 1.0).mean() <= 1e-3
        s = got_scale[:, np.arange(self.page) // TOKENS][..., None]
        touched = kind > 0
        off = np.abs(oracle.e4m3_decode(got) * s - exact)
        tol = half_step((np.abs(exact) + turn) / s) * s + turn
        assert (off[touched] <= tol[touched]).all(), f"{(off / tol)[touched].max():.3f} x its bound"


CASES = [
    # lengths, starts, Hq, Hkv, D, rot, interleaved, page, order
    ([1], [0], 4, 2, 128, 128, False, 16, "thd"),
    ([1, 1, 1, 1, 1], [0, 1, 15, 16, 77], 8, 2, 128, 128, False, 64, "thd"),
    ([40, 3, 1, 17, 33], [0, 14, 31, 5, 100], 4, 4, 128, 64, True, 32, "htd"),
    ([100], [7], 2, 1, 64, 64, False, 16, "thd"),
    ([37, 2], [3, 9], 3, 3, 64, 16, True, 48, "htd"),
    ([33], [12], 5, 1, 128, 32, False, 128, "padded"),
    ([50, 1], [11, 8], 4, 2, 64, 62, False, 16, "thd"),   # half a head's pairs on no boundary: one by one
    ([21, 4], [2, 30], 2, 2, 96, 96, True, 24, "thd"),    # pages that end in a short block
    ([19], [1], 3, 1, 80, 0, False, 20, "odd"),
    ([9, 30], [6, 0], 2, 2, 256, 256, False, 16, "thd"),
    ([31], [2], 1, 1, 1, 0, False, 16, "thd"),
    ([26], [3], 2, 1, 128, 128, False, 16, "odd"),
    ([20], [5], 2, 12, 64, 64, False, 1, "thd"),          # pages of one token: a scale each
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_equals_oracle(dev, case):
    lengths, starts, Hq, Hkv, D, rot, inter, page, order = CASES[case]
    a = Append(lengths, starts, Hq, Hkv, D, rot, inter, page, order, seed=case, mscale=1.0 if case % 2 else 1.3,
               fused=case % 3 == 0)
    a.check(*a.run(dev, "in place" if case % 4 == 0 else None))


@pytest.mark.parametrize("size", [1e-14, 1e-9, 3e4, 1e14, 1e20])
def test_append_at_the_ends_of_the_scales(dev, size):
    """Numbers so small that they vanish, and so large that they saturate."""
    a = Append([40], [3], 2, 2, 128, 128, False, 16, "thd", seed=5, size=size)
    out, sides, bits = a.run(dev)
    ref = a.oracle()
    assert np.array_equal(f64(sides[3]), ref[2][1]) and np.array_equal(sides[1].cpu().numpy(), ref[2][0])
    assert f64(sides[2]).min() >= 2.0 ** -40 and f64(sides[2]).max() <= 2.0 ** 40
    assert bits == 0


def test_append_skips_what_it_is_told_to(dev):
    """Negative positions, slots of -1 and outside the cache, in the middle of runs that they cut."""
    a = Append([64], [0], 2, 2, 128, 64, False, 16, "thd", seed=6)
    limit = a.kc.shape[0] * a.page
    a.pos[5], a.slots[20], a.slots[37], a.slots[40] = -1, -1, limit, -2
    # a block whose run is cut has two runs in one call: keep one of each
    for t in list(range(6, 16)) + list(range(21, 32)) + list(range(38, 48)):
        a.slots[t] = -1
    ref = a.oracle()
    assert ref[4] == kda.KDA_ERR_PAGES
    out, sides, bits = a.run(dev)
    a.check(out, sides, bits, ref)
    assert (f64(out)[5] == 7).all()


def test_append_of_numbers_that_are_not_finite(dev):
    a = Append([20, 3], [0, 4], 2, 2, 128, 0, False, 32, "thd", seed=7)
    a.k[3, 0, 5] = float("nan")
    a.k[4, 1, 5] = float("inf")
    a.v[3, 0, 7] = float("-inf")
    a.v[21, 1, :] = float("nan")
    out, sides, bits = a.run(dev)
    _, keys, values, _, _ = a.oracle()
    for codes, scales, ref in ((sides[0], sides[2], keys), (sides[1], sides[3], values)):
        got, want = codes.cpu().numpy(), ref[0]
        nan = (want & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan)
        assert np.array_equal(got[~nan], want[~nan])
        assert np.array_equal(f64(scales), ref[1])


def test_append_token_by_token(dev):
    """A block filled by single calls: the scale grows, never shrinks, begins anew with the block, and every code stays
    within a rounding a growth of its number."""
    gen = torch.Generator().manual_seed(8)
    n, H, D, page = 48, 2, 128, 32
    v = (torch.randn((n, H, D), generator=gen) * torch.exp(2 * torch.randn((n, 1, 1), generator=gen))).to(torch.bfloat16)
    vd = v.to(dev)
    sides = [torch.randint(0, 255, (2, page, H, D), dtype=torch.uint8, device=dev) for _ in range(2)]
    sides += [torch.full((2, 2, H), float("nan"), device=dev) for _ in range(2)]
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    for t in range(n):
        kda.kda_rope_append_fp8(vd[t:t + 1], vd[t:t + 1], vd[t:t + 1], ints([t], dev), ints([t], dev), none, *sides)
    assert torch.equal(sides[0].view(-1, H, D)[:n], sides[1].view(-1, H, D)[:n])
    assert torch.equal(sides[2].view(-1, H)[:3], sides[3].view(-1, H)[:3])
    got = oracle.dequantized(sides[1].cpu().numpy(), f64(sides[3])).reshape(-1, H, D)[:n]
    exact = f64(v)
    for b in range(3):
        rows = slice(16 * b, 16 * b + 16)
        for h in range(H):
            need = [2.0 ** oracle.scale_exponent(np.abs(exact[t, h]).max()) for t in range(16 * b, 16 * b + 16)]
            assert float(sides[3].view(-1, H)[b, h]) == max(need)
            grown = np.maximum.accumulate(need)
            for i, t in enumerate(range(16 * b, 16 * b + 16)):
                x = exact[t, h]
                steps = sorted(set(grown[i:]))
                tol = sum(half_step(np.abs(x) * (1 + 2.0 ** -3) / s) * s for s in steps)
                assert (np.abs(got[rows][i, h] - x) <= tol).all()


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("Hkv,D,page,order", [(2, 128, 64, "thd"), (4, 64, 16, "htd"), (1, 80, 20, "odd"),
                                              (3, 16, 48, "padded"), (2, 256, 1, "thd"), (1, 1, 24, "thd")])
def test_read_equals_oracle(dev, Hkv, D, page, order):
    kv = [1, 200, 0, 37, 64, page]
    a = Attention(kv, kv, Hkv, Hkv, D, page, order=order, seed=D).poison()
    T = sum(kv) + 5
    err = err_word(dev)
    out = kda.PagedRead(*(torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2)))
    got = kda.kda_paged_read_fp8(*(to_device(t, dev) for t in (a.k, a.v, a.ks, a.vs)), ints(a.table, dev),
                                 ints(a.cu, dev), ints(a.kv, dev), T, out=out, error_word=err)
    k, v, bits = oracle.paged_read_fp8(a.k.numpy(), a.v.numpy(), f64(a.ks), f64(a.vs), a.table, a.cu, a.kv, T)
    assert int(err.item()) == bits == 0
    for g, r in zip(got, (k, v)):
        g = f64(g)
        assert (g[-5:] == 7).all()
        assert np.array_equal(g[:-5], r[:-5])


def test_read_of_the_last_tokens_and_of_bad_lengths_and_pages(dev):
    a = Attention([4, 30, 5, 2, 8], [90, 12, 40, 33, 64], 2, 2, 64, 16, seed=3)
    a.kv[3] = 10 ** 6          # longer than the table: no tokens
    a.table[4, 3] = -1         # tokens 48..63 of the last request
    a.cu = np.array([0, 4, 34, 34, 41, 49])  # the fourth has 7 rows
    T = 49
    err = err_word(dev)
    strided = torch.full((2, T, 3, 70), 7.0, dtype=torch.bfloat16, device=dev)
    out = kda.PagedRead(strided[0, :, 1:, 3:67], strided[1, :, :2, :64])
    kda.kda_paged_read_fp8(*(to_device(t, dev) for t in (a.k, a.v, a.ks, a.vs)), ints(a.table, dev), ints(a.cu, dev),
                           ints(a.kv, dev), T, out=out, error_word=err)
    k, v, bits = oracle.paged_read_fp8(a.k.numpy(), a.v.numpy(), f64(a.ks), f64(a.vs), a.table, a.cu, a.kv, T)
    assert int(err.item()) == bits == kda.KDA_ERR_LENGTHS | kda.KDA_ERR_PAGES
    assert np.array_equal(f64(out.k), k) and np.array_equal(f64(out.v), v)
    assert (strided[0, :, 0] == 7).all() and (strided[1, :, 2] == 7).all()
    # bounds out of order: that request is skipped, and said to be
    cu = np.array([0, 4, 50, 34, 41, 49])
    err.zero_()
    kda.kda_paged_read_fp8(*(to_device(t, dev) for t in (a.k, a.v, a.ks, a.vs)), ints(a.table, dev), ints(cu, dev),
                           ints(a.kv, dev), T, out=out, error_word=err)
    assert int(err.item()) & kda.KDA_ERR_SEQLENS


# ---------------------------------------------------------------- attention

SHAPES = [
    # new, kv, Hq, Hkv, D, page, window, order
    ([1], [1], 4, 1, 128, 16, 0, "thd"),
    ([1, 1, 1], [5, 300, 128], 8, 2, 128, 64, 0, "thd"),
    ([1, 4, 0, 9], [700, 4, 0, 333], 6, 2, 64, 16, 0, "htd"),
    ([300], [300], 4, 1, 128, 128, 0, "thd"),
    ([130, 1, 77], [500, 129, 77], 4, 2, 64, 32, 0, "padded"),
    ([5, 200], [2, 190], 4, 2, 128, 16, 0, "thd"),       # fewer keys than rows: rows that see none
    ([3, 90], [400, 1000], 3, 1, 128, 64, 100, "htd"),   # a window
    ([17, 33], [1500, 700], 8, 1, 64, 64, 1, "thd"),     # a row sees itself alone
    ([20, 1], [60, 77], 4, 2, 96, 24, 0, "thd"),         # the CUDA cores: other sizes
    ([6, 1], [50, 90], 2, 1, 80, 20, 9, "odd"),
    ([4], [70], 2, 2, 256, 1, 0, "thd"),
    ([3], [40], 6, 1, 5, 16, 0, "thd"),
    ([2], [260], 128, 1, 64, 64, 0, "thd"),              # 128 heads share a key
    ([1] * 9, [64 * i + 1 for i in range(9)], 2, 1, 128, 64, 0, "thd"),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention_equals_oracle(dev, case):
    new, kv, Hq, Hkv, D, page, window, order = SHAPES[case]
    a = Attention(new, kv, Hq, Hkv, D, page, window, order, seed=case).poison()
    err = err_word(dev)
    out, lse = a.run(dev, kda, error_word=err)
    a.check(out, lse)
    assert int(err.item()) == 0
    without, _ = a.run(dev, kda)
    assert torch.equal(out, without)


FEW = [
    # decode and verify steps: new, kv, heads that share a key (times Hkv), Hkv, page, window, order
    ([1], [77], 4, 2, 16, 0, "thd"),
    ([1] * 5, [1, 128, 129, 1000, 0], 1, 3, 64, 0, "thd"),
    ([1] * 3, [3000, 5, 640], 2, 1, 128, 0, "htd"),
    ([1] * 40, [17 * i % 700 for i in range(40)], 4, 2, 32, 0, "thd"),
    ([1, 0, 1, 1], [9000, 0, 400, 4096], 8, 1, 64, 0, "thd"),      # cut between many CTAs
    ([8, 8, 8], [1200, 8, 130], 3, 2, 32, 0, "htd"),
    ([4, 4], [2, 300], 3, 2, 16, 0, "thd"),                        # rows that see no key
    ([2, 2, 2], [500, 900, 40], 16, 1, 64, 100, "padded"),         # a window
    ([1, 1], [700, 300], 32, 1, 64, 1, "thd"),                     # a row sees itself alone
    ([1, 30, 1, 1, 2, 1, 1, 1], [200, 700, 64, 1, 333, 90, 128, 127], 6, 2, 64, 0, "thd"),  # ragged
    ([1] * 200, [5 + i for i in range(200)], 7, 1, 16, 0, "thd"),
]


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_attention_of_few_rows_equals_oracle(dev, case, D):
    new, kv, g, Hkv, page, window, order = FEW[case]
    a = Attention(new, kv, g * Hkv, Hkv, D, page, window, order, seed=100 + case, q_spread=0.5).poison()
    err = err_word(dev)
    work = kda.paged_attention_workspace(D, dev)
    out, lse = a.run(dev, kda, workspace=work, error_word=err)
    a.check(out, lse)
    assert int(err.item()) == 0
    again, lse2 = a.run(dev, kda, workspace=work)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
