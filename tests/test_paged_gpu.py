"""The page plan, rotary append and paged attention on the GPU against the
fp64 oracle, at the sizes and masks where they can go wrong. Bounds and their
derivation: paged_cases.py. Whole numbers must be equal."""

import numpy as np
import pytest
import torch

import oracle
from linear_attention_ssm_step_gb300 import kda
from paged_cases import Attention, cache, ints, rope_bound, to_device

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


# ---------------------------------------------------------------- plan

def plan_inputs(new, cached, page, seed, spare=5, width=None):
    rng = np.random.default_rng(seed)
    new, cached = np.asarray(new), np.asarray(cached)
    have = [-(-max(int(c), 0) // page) for c in cached]
    total = [-(-max(int(c) + int(n), 0) // page) for c, n in zip(cached, new)]
    pages = sum(max(h, t) for h, t in zip(have, total)) + spare
    perm = rng.permutation(pages)
    w = max([1] + total + have) if width is None else width
    table = np.full((len(new), w), -1, dtype=np.int64)
    at = 0
    for r, h in enumerate(have):
        h = min(h, w)
        table[r, :h] = perm[at:at + h]
        at += h
    return new, cached, table, perm[at:], pages


def check_plan(dev, new, cached, table, free, pages, page, num_tokens, free_count=None, stride=None):
    fc = len(free) if free_count is None else free_count
    ref = oracle.paged_plan(cached, new, table, free, fc, page, pages, num_tokens)
    t_d = ints(table, dev)
    if stride is not None:
        wide = torch.full((len(new), stride), -9, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = t_d
        t_d = wide[:, :table.shape[1]]
    err = err_word(dev)
    free_d = ints(free, dev)
    got = kda.kda_paged_plan(ints(cached, dev), ints(new, dev), t_d, free_d, ints([fc], dev), page, pages, num_tokens,
                             error_word=err)
    for name, g, r in zip(("table",) + got._fields, (t_d,) + tuple(got), ref[:6]):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(r).reshape(-1)), name
    assert int(err.item()) == ref[6]
    if stride is not None:
        assert (wide[:, table.shape[1]:] == -9).all()
    return ref


@pytest.mark.parametrize("page", [1, 16, 24, 64])
@pytest.mark.parametrize("R,most", [(1, 1), (1, 700), (5, 40), (300, 3), (700, 9)])
def test_plan_equals_oracle(dev, R, most, page):
    rng = np.random.default_rng(R * 100 + most + page)
    new, cached = rng.integers(0, most + 1, R), rng.integers(0, 200, R)
    cached[::3] = page * rng.integers(0, 4, len(cached[::3]))  # full last pages, and none
    p = plan_inputs(new, cached, page, seed=R)
    check_plan(dev, *p[:4], p[4], page, int(new.sum()))
    check_plan(dev, *p[:4], p[4], page, int(new.sum()) + 37, stride=p[2].shape[1] + 3)  # padded rows and table


def test_plan_of_the_largest_batch(dev):
    rng = np.random.default_rng(1)
    R = kda.KDA_MAX_REQUESTS
    p = plan_inputs(rng.integers(0, 4, R), rng.integers(0, 90, R), 16, seed=2)
    check_plan(dev, *p[:4], p[4], 16, int(p[0].sum()))


def test_plan_admission(dev):
    """Free pages that run out, rows that run out, broken lengths, page numbers outside the pool."""
    new, cached, table, free, pages = plan_inputs([40, 3, 500, 1, 0, 7], [10, 16, 0, 15, 64, 300], 16, seed=3)
    T = int(new.sum())
    for fc in (0, 1, 2, 3, 4, 20, len(free), len(free) + 50, -4):
        check_plan(dev, new, cached, table, free, pages, 16, T, free_count=fc)
    for rows in (0, 1, 40, 43, 542, 543, 550):
        check_plan(dev, new, cached, table, free, pages, 16, rows)
    bad_new, bad_cached = new.copy(), cached.copy()
    bad_new[1], bad_cached[3], bad_new[5] = -2, -1, 2 ** 31 - 10
    ref = check_plan(dev, bad_new, bad_cached, table, free, pages, 16, T)
    assert ref[6] & kda.KDA_ERR_LENGTHS
    wild = table.copy()
    wild[0, 0] = pages  # the open page of request 0
    assert check_plan(dev, new, cached, wild, free, pages, 16, T)[6] == kda.KDA_ERR_PAGES
    wild_free = free.copy()
    wild_free[-2] = -3
    assert check_plan(dev, new, cached, table, wild_free, pages, 16, T)[6] == kda.KDA_ERR_PAGES


def test_plan_without_requests(dev):
    check_plan(dev, np.zeros(0, int), np.zeros(0, int), np.zeros((0, 3), int), np.arange(4), 4, 16, 5)


# ---------------------------------------------------------------- rope and append

def rope_case(dev, T, Hq, Hkv, D, rot, interleaved, page, order, fused, mscale, in_place, seed, poke=True):
    gen = torch.Generator().manual_seed(seed)
    if fused:
        row = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(torch.bfloat16)
        q, k, v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn((T, h, D), generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pages = -(-T // page) + 2
    kc, vc = cache(pages, page, Hkv, D, order, gen)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 1 << 20, T)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1  # the last position there is
    slots = rng.permutation(pages * page)[:T]
    if poke and T > 6:
        pos[2], slots[3], slots[4], slots[5] = -1, -1, pages * page, -2
    freqs = kda.rope_freqs(rot, 10000.0, device=dev) if rot else torch.zeros(0, dtype=torch.int64, device=dev)
    turns = [int(x) % (1 << 64) for x in freqs.cpu().tolist()]
    f = lambda t: t.double().numpy()  # noqa: E731
    qo, ko, vo, written, bits = oracle.rope_append(f(q), f(k), f(v), pos, slots, turns, f(kc), f(vc), interleaved, mscale)
    qd, kd, vd, kcd, vcd = (to_device(t, dev) for t in (q, k, v, kc, vc))
    err = err_word(dev)
    out = qd if in_place else torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    kda.kda_rope_append(qd, kd, vd, ints(pos, dev), ints(slots, dev), freqs, kcd, vcd, q_out=out,
                        interleaved=interleaved, mscale=mscale, error_word=err)
    assert int(err.item()) == bits
    half = rot // 2

    def partner(x):
        y = np.zeros_like(x)
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2] = x[..., 1:rot:2], x[..., 0:rot:2]
        else:
            y[..., :half], y[..., half:rot] = x[..., half:rot], x[..., :half]
        return y

    got = out.double().cpu().numpy()
    qn = f(q)
    bound = rope_bound(qo, qn, partner(qn), mscale)
    assert (np.abs(got - qo)[written] <= bound[written]).all()
    assert np.array_equal(got[..., rot:][written], qn[..., rot:][written]), "values past rotary_dim pass unchanged"
    assert np.array_equal(got[~written], qn[~written] if in_place else np.full_like(qn[~written], 7.0))
    gk, gv = kcd.double().cpu().numpy(), vcd.double().cpu().numpy()
    assert np.array_equal(gv, vo), "values are copied, other slots untouched"
    kn = f(k)
    kb = np.zeros_like(gk)
    for t in range(T):
        if pos[t] >= 0 and 0 <= slots[t] < pages * page:
            kb[slots[t] // page, slots[t] % page] = rope_bound(ko[slots[t] // page, slots[t] % page], kn[t],
                                                               partner(kn)[t], mscale)
            kb[slots[t] // page, slots[t] % page, :, rot:] = 0
    assert (np.abs(gk - ko) <= kb).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,order,fused", [
    (1, 1, 1, 64, 64, 16, "thd", False),
    (9, 32, 8, 128, 128, 64, "thd", True),
    (33, 12, 12, 64, 32, 16, "htd", True),
    (17, 8, 2, 128, 96, 16, "pair", False),
    (17, 6, 3, 128, 16, 32, "padded", False),
    (21, 5, 1, 128, 64, 7, "odd", False),      # rows off 16 bytes: single accesses
    (19, 3, 3, 80, 40, 16, "thd", True),       # a turned part of five runs of 8
    (19, 3, 1, 33, 14, 5, "thd", False),       # an odd head_dim
    (9, 2, 1, 256, 256, 16, "thd", False),
    (9, 2, 1, 128, 0, 16, "thd", False),       # nothing turned
    (300, 40, 8, 128, 128, 64, "thd", False),
])
def test_rope_append(dev, T, Hq, Hkv, D, rot, interleaved, page, order, fused):
    rope_case(dev, T, Hq, Hkv, D, rot, interleaved, page, order, fused, 1.0, False, seed=T + D)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 64), (48, 12)])
def test_rope_in_place_and_scaled(dev, D, rot, interleaved):
    rope_case(dev, 15, 4, 2, D, rot, interleaved, 16, "thd", True, 1.25, True, seed=5)


# ---------------------------------------------------------------- attention

def run_and_check(dev, a, **kw):
    err = err_word(dev)
    out, lse = a.run(dev, kda, error_word=err, **kw)
    a.check(out, lse)
    assert int(err.item()) == 0
    return out, lse


SHAPES = [  # Hq, Hkv, D, page, order
    (8, 1, 128, 64, "thd"),
    (32, 8, 128, 16, "htd"),
    (4, 4, 64, 16, "thd"),
    (12, 4, 128, 32, "pair"),
    (10, 2, 64, 128, "padded"),
    (24, 2, 128, 256, "thd"),
    (64, 1, 64, 64, "thd"),
    (6, 2, 128, 16, "odd"),    # CUDA cores: rows off 16 bytes
    (6, 3, 80, 16, "thd"),     # CUDA cores: head_dim
    (4, 2, 128, 24, "thd"),    # CUDA cores: page size
    (3, 1, 33, 5, "thd"),      # CUDA cores: all odd
    (2, 1, 256, 16, "thd"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("new,kv", [
    ([1], [1]),                                    # the first token there is
    ([1, 1, 1, 1, 1, 1], [1, 15, 16, 17, 129, 700]),  # decode across page and tile ends
    ([8, 8, 3], [8, 137, 400]),                    # verify
    ([130, 1, 0, 77], [130, 260, 40, 333]),        # chunks, a decode token and an idle request
], ids=["one", "decode", "verify", "mixed"])
def test_attention(dev, shape, new, kv):
    Hq, Hkv, D, page, order = shape
    a = Attention(new, kv, Hq, Hkv, D, page, order=order, seed=sum(kv) + D).poison()
    run_and_check(dev, a)


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 16), (64, 4, 4, 64), (48, 4, 2, 8)])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 300, 100000])
def test_attention_window(dev, D, Hq, Hkv, page, window):
    a = Attention([1, 200, 8, 1], [513, 431, 300, 40], Hq, Hkv, D, page, window=window, seed=window).poison()
    # pages before every row's window may have been given away
    for r, (n, L) in enumerate(zip(a.new, a.kv)):
        a.table[r, :max(0, L - n - window + 1) // page] = -1
    run_and_check(dev, a)


@pytest.mark.parametrize("D,page", [(128, 16), (64, 32), (40, 16)])
def test_attention_empty_rows(dev, D, page):
    """kv_len below the new tokens: the first rows stand before the first key."""
    a = Attention([5, 300, 1, 40], [3, 20, 0, 0], 8, 2, D, page, seed=4).poison()
    out, lse = run_and_check(dev, a)
    assert torch.isneginf(lse[:2]).all() and (out[-40:] == 0).all()


@pytest.mark.parametrize("D", [128, 64, 72])
def test_attention_bad_requests_are_skipped_and_reported(dev, D):
    a = Attention([4, 3, 6, 2], [40, 3, 90, 20], 4, 2, D, 16, seed=6)
    a.cu = np.array([0, 4, 7, 99, 15])       # request 2 ends past the rows, request 3's bounds go backwards
    a.kv[1] = 10 ** 6                        # over its block table
    ref = a.oracle()
    err = err_word(dev)
    out, lse = a.run(dev, kda, error_word=err)
    a.check(out, lse, ref=ref)
    assert int(err.item()) == ref[5] == kda.KDA_ERR_SEQLENS | kda.KDA_ERR_LENGTHS
    b = Attention([4, 3], [40, 60], 4, 2, D, 16, seed=7)
    b.table[0, 1] = b.k.shape[0]
    b.table[1, 0] = -5
    ref = b.oracle()
    err = err_word(dev)
    out, lse = b.run(dev, kda, error_word=err)
    b.check(out, lse, ref=ref)
    assert int(err.item()) == ref[5] == kda.KDA_ERR_PAGES


@pytest.mark.parametrize("D", [128, 64, 96])
def test_attention_strided_rows_and_scale(dev, D):
    a = Attention([3, 90], [77, 150], 6, 2, D, 16, seed=8, scale=0.37, extra_width=3, fused_q=True)
    wide = torch.full((93, 9, D + 8), 7.0, dtype=torch.bfloat16, device=dev)
    run_and_check(dev, a, out=wide[:, 1:7, :D])
    assert (wide[:, 0] == 7).all() and (wide[:, 7:] == 7).all() and (wide[..., D:] == 7).all()


@pytest.mark.parametrize("D", [128, 64, 32])
def test_attention_large_scores(dev, D):
    """Scores that span hundreds: the running maximum moves far, in both directions."""
    a = Attention([70, 1], [500, 400], 4, 2, D, 16, seed=9, scale=4.0)
    ramp = torch.linspace(0.2, 6.0, a.page)[None, :, None, None]
    a.k.mul_(ramp.to(torch.bfloat16))
    run_and_check(dev, a)


@pytest.mark.parametrize("D", [128, 64])
def test_attention_many_splits_and_repeats(dev, D):
    """One long request: its keys are split over the whole GPU; the same bits every call, and the
    workspace is left ready."""
    a = Attention([1], [20000], 2, 1, D, 64, seed=10)
    ws = kda.paged_attention_workspace(D, dev)
    out, lse = run_and_check(dev, a, workspace=ws)
    assert (ws[:kda.KDA_ATTENTION_WORKSPACE_ZEROED] == 0).all()
    for _ in range(3):
        o2, l2 = a.run(dev, kda, workspace=ws)
        assert torch.equal(o2.view(torch.int16), out.view(torch.int16)) and torch.equal(l2, lse)


@pytest.mark.parametrize("D", [128, 64, 48])
def test_attention_nan_rows(dev, D):
    """A query, and a key, of NaN: the rows that see one are NaN, value and log-sum; the others are as without it."""
    a = Attention([1, 150, 3], [300, 400, 260], 8, 2, D, 16, seed=12)
    b = Attention([1, 150, 3], [300, 400, 260], 8, 2, D, 16, seed=12)
    b.q[0, 5], b.q[20] = float("nan"), float("nan")
    key = 351  # of request 1: seen by its rows from 351 - 250 on
    b.k[int(b.table[1, key // 16]), key % 16, 1] = float("nan")
    (o, z), (on, zn) = run_and_check(dev, a), b.run(dev, kda)
    bad = torch.zeros((154, 8), dtype=torch.bool, device=dev)
    bad[0, 5], bad[20] = True, True
    bad[1 + 101:151, 4:] = True
    assert torch.isnan(on[bad]).all() and torch.isnan(zn[bad]).all()
    assert torch.equal(on[~bad], o[~bad]) and torch.equal(zn[~bad], z[~bad])


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("R,new,g,kv", [(160, 1, 4, 700), (120, 8, 16, 500), (3, 8, 16, 3000), (2, 3, 16, 5000),
                                        (150, 2, 3, 140), (40, 5, 12, 1100)])
def test_attention_tiles_of_one_request(dev, D, R, new, g, kv):
    """Few and many rows in a tile, held whole by one block or cut between several."""
    rng = np.random.default_rng(R + g)
    lens = rng.integers(max(new, kv // 3), kv + 1, R)
    a = Attention([new] * R, lens.tolist(), 2 * g, 2, D, 32, seed=R + g).poison()
    run_and_check(dev, a)


@pytest.mark.parametrize("D,Hq,Hkv,new,kv", [
    (128, 32, 8, [300, 1, 700], [300, 3000, 1900]),           # chunks: items of two tiles cut in two
    (64, 16, 4, [100, 37, 1, 60] * 6, [1200, 900, 2500, 64] * 6),
    (128, 12, 4, [8] * 32, list(range(1000, 5000, 125))),     # few rows
    (128, 32, 2, [5] * 9, list(range(700, 3400, 300))),       # one tile, many rows
    (64, 8, 1, [2], [30000]),                                 # more parts than a batch of the join
])
def test_attention_same_bits_whatever_the_order_of_arrival(dev, D, Hq, Hkv, new, kv):
    """Parts of cut items are joined by whichever block ends last: with the GPU to itself, and with other work beside
    that makes blocks end in other orders, the same bits."""
    a = Attention(new, kv, Hq, Hkv, D, 16, seed=17)
    ws = kda.paged_attention_workspace(D, dev)
    out, lse = run_and_check(dev, a, workspace=ws)
    args = (to_device(a.q, dev), to_device(a.k, dev), to_device(a.v, dev), ints(a.table, dev), ints(a.cu, dev),
            ints(a.kv, dev))
    outs = [(torch.empty_like(out), torch.empty_like(lse)) for _ in range(24)]
    noise = torch.empty(1 << 26, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, (o, z) in enumerate(outs):
        if i % 3:
            with torch.cuda.stream(side):
                noise.add_(1.0)
        kda.kda_paged_attention(*args, out=o, lse=z, scale=a.scale, workspace=ws)
    torch.cuda.synchronize()
    for o, z in outs:
        assert torch.equal(o, out) and torch.equal(z, lse)
    assert (ws[:kda.KDA_ATTENTION_WORKSPACE_ZEROED] == 0).all()


def test_attention_many_requests(dev):
    rng = np.random.default_rng(11)
    R = 900
    new = rng.integers(0, 3, R)
    kv = new + rng.integers(0, 40, R)
    run_and_check(dev, Attention(new.tolist(), kv.tolist(), 4, 2, 64, 16, seed=12).poison())


@pytest.mark.parametrize("Hq,Hkv,D", [(128, 1, 128), (100, 1, 64), (65, 1, 128), (43, 1, 64)])
def test_attention_many_heads_share(dev, Hq, Hkv, D):
    """Groups that fill a tile of rows, or leave much of it empty."""
    run_and_check(dev, Attention([1, 3, 20], [200, 131, 20], Hq, Hkv, D, 16, seed=Hq).poison())


@pytest.mark.parametrize("D", [128, 64])
def test_attention_rows_off_16_bytes(dev, D):
    """q and out rows that single accesses alone can reach, on the cache of the tensor-core kernel."""
    a = Attention([3, 150, 1], [77, 350, 600], 6, 2, D, 16, seed=15)
    a.q = torch.cat([a.q, a.q[:, :1]], dim=1).reshape(-1)[1:1 + a.q.numel()].view(a.q.shape)
    wide = torch.full((154, 6, D + 3), 7.0, dtype=torch.bfloat16, device=dev)
    run_and_check(dev, a, out=wide[..., 1:D + 1])
    assert (wide[..., 0] == 7).all() and (wide[..., D + 1:] == 7).all()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 2, 2)])
def test_attention_long_chunk(dev, D, Hq, Hkv):
    """Many items of many units: whole ones, ones cut in two, and their order on the line."""
    run_and_check(dev, Attention([600, 1, 257], [1700, 3000, 257], Hq, Hkv, D, 64, seed=16).poison())


def test_attention_without_lse_and_largest_window(dev):
    a = Attention([5, 2], [3, 90], 4, 2, 128, 16, seed=17, window=2 ** 31 - 1)
    out, _ = a.run(dev, kda)
    args = (to_device(a.q, dev), to_device(a.k, dev), to_device(a.v, dev), ints(a.table, dev), ints(a.cu, dev),
            ints(a.kv, dev))
    only = kda.kda_paged_attention(*args, scale=a.scale, window=a.window)
    assert torch.equal(out, only)
    a.check(*a.run(dev, kda))


@pytest.mark.parametrize("D", [128, 64])
def test_attention_wait_that_runs_out(dev, D):
    """Failure detection without a fault: in the build that issues no copy (tests/test_timeout_gpu.py) the bounded waits
    run out, the call reports KDA_ERR_TIMEOUT and returns, and the context stays usable."""
    from linear_attention_ssm_step_gb300 import _build
    wlib = kda.bind_library(_build.build(variant="waittest"))
    a = Attention([1, 40], [300, 90], 4, 2, D, 16, seed=18)
    err = err_word(dev)
    call = kda.prepare_paged_attention(to_device(a.q, dev), to_device(a.k, dev), to_device(a.v, dev), ints(a.table, dev),
                                       ints(a.cu, dev), ints(a.kv, dev), error_word=err)
    assert wlib.kda_paged_attention(*call._args) == kda.KDA_OK
    torch.cuda.synchronize()
    assert int(err.item()) == kda.KDA_ERR_TIMEOUT
    run_and_check(dev, a)


def test_attention_without_work(dev):
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=dev)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device=dev)
    z = torch.zeros(1, dtype=torch.int32, device=dev)
    out = kda.kda_paged_attention(q, c, c.clone(), torch.zeros((1, 1), dtype=torch.int32, device=dev),
                                  torch.zeros(2, dtype=torch.int32, device=dev), z)
    assert out.shape == (0, 4, 64)


def test_attention_graph_and_side_stream(dev):
    a = Attention([1, 8, 40], [300, 90, 260], 8, 2, 128, 16, seed=13)
    ref, _ = a.run(dev, kda)
    args = (to_device(a.q, dev), to_device(a.k, dev), to_device(a.v, dev), ints(a.table, dev), ints(a.cu, dev),
            ints(a.kv, dev))
    ws = kda.paged_attention_workspace(128, dev)
    out = torch.empty_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call = kda.prepare_paged_attention(*args, out=out, scale=a.scale, workspace=ws)
        call()
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gcall = kda.prepare_paged_attention(*args, out=out, scale=a.scale, workspace=ws)
        gcall()
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("D", [128, 64, 96])
def test_pages_past_2_to_the_31_elements(dev, D):
    """Append and attention in the last pages of a cache of more than 2^31 elements: the same bits as in a small one."""
    Hq, Hkv, page = 16, 8, 64
    a = Attention([1, 140, 5], [600, 300, 64], Hq, Hkv, D, page, seed=15)
    T, few = 146, a.k.shape[0]
    many = 2 ** 31 // (page * Hkv * D) + few + 8
    first = many - few  # the small cache's page 0 there
    gen = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn((T, h, D), generator=gen).to(torch.bfloat16).to(dev) for h in (Hq, Hkv, Hkv))
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(a.new, a.kv)])
    owner = np.repeat(np.arange(3), a.new)
    slots = a.table[owner, pos // page] * page + pos % page
    freqs = kda.rope_freqs(D, device=dev)
    got = []
    for base, pages in ((0, few), (first, many)):
        kc, vc = (torch.empty((pages, page, Hkv, D), dtype=torch.bfloat16, device=dev) for _ in range(2))
        kc[base:].copy_(a.k)
        vc[base:].copy_(a.v)
        err = err_word(dev)
        qr = kda.kda_rope_append(q, k, v, ints(pos, dev), ints(slots + base * page, dev), freqs, kc, vc, error_word=err)
        table = np.where(a.table < 0, a.table, a.table + base)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention(qr, kc, vc, ints(table, dev), ints(a.cu, dev), ints(a.kv, dev), lse=lse,
                                      error_word=err)
        assert int(err.item()) == 0
        got.append([x.clone() for x in (qr, out, lse, kc[base:], vc[base:])])
        del kc, vc
    assert not torch.equal(got[0][3], a.k.to(dev)), "the rows were appended"
    for x, y in zip(*got):
        assert torch.equal(x, y) and torch.isfinite(x.float()).all()


def test_the_three_together(dev):
    """A prompt in two chunks, then decode: each token's attention equals attention over the whole
    sequence, laid out plainly."""
    Hq, Hkv, D, page, R = 8, 2, 128, 16, 3
    gen = torch.Generator().manual_seed(14)
    lens = [75, 20, 133]
    steps = [[50, 20, 100], [25, 0, 31], [0, 0, 1], [0, 0, 1]]
    total = [sum(s[r] for s in steps) for r in range(R)]
    assert total == lens
    qkv = [torch.randn((n, Hq + 2 * Hkv, D), generator=gen).to(torch.bfloat16) for n in lens]
    pages = 40
    kc = torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
    vc = kc.clone()
    table = torch.full((R, 12), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=gen).to(torch.int32).to(dev)
    count = ints([pages], dev)
    cached = torch.zeros(R, dtype=torch.int32, device=dev)
    freqs = kda.rope_freqs(64, 10000.0, kda.KDA_ROPE_LINEAR, 2.0, device=dev)
    turns = [int(x) % (1 << 64) for x in freqs.cpu().tolist()]
    err = err_word(dev)
    done, got = [0] * R, [[] for _ in range(R)]
    for new in steps:
        rows = torch.cat([qkv[r][done[r]:done[r] + n] for r, n in enumerate(new)]).to(dev)
        plan = kda.kda_paged_plan(cached, ints(new, dev), table, free, count, page, pages, rows.shape[0], error_word=err)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        qo = kda.kda_rope_append(q, k, v, plan.positions, plan.slots, freqs, kc, vc, error_word=err)
        out = kda.kda_paged_attention(qo, kc, vc, table, plan.cu_new, plan.kv_len, error_word=err).cpu()
        at = 0
        for r, n in enumerate(new):
            got[r].append(out[at:at + n])
            at, done[r] = at + n, done[r] + n
        cached, count = plan.kv_len, plan.free_count
    assert int(err.item()) == 0
    assert int(count.item()) == pages - sum(-(-n // page) for n in lens)
    for r, n in enumerate(lens):
        x = qkv[r].double().numpy()
        pos = np.arange(n)
        bf = lambda y: torch.tensor(y).to(torch.bfloat16).double().numpy()  # noqa: E731
        q = bf(oracle.rope_rotate(x[:, :Hq], pos, turns, False, 1.0))
        k = bf(oracle.rope_rotate(x[:, Hq:Hq + Hkv], pos, turns, False, 1.0))
        o, _, A, S, _, _ = oracle.paged_attention(q, k[None], x[None, :, Hq + Hkv:], np.zeros((1, 1), int), [0, n], [n],
                                                  D ** -0.5, 0)
        g = torch.cat(got[r]).double().numpy()
        # q and k may round to the other bf16 neighbour: one ulp, 2^-7 of a value in [1, 2) mantissa terms at most,
        # of all of the score's terms: 2^-6 S in the scores, twice that in the weights
        assert (np.abs(g - o) <= (2.0 ** -8 + 2.0 ** -5 * S[:, :, None]) * A + 2.0 ** -8 * np.abs(o)).all()


def test_hybrid_layers_in_chunks_equal_one_pass(dev):
    """KDA and attention layers together (hybrid.py): prompts in two chunks and a token each, against all at once.
    The two differ by roundings to bf16: the KDA state between calls, and what follows from it; every layer adds to a
    residual of its own size, so half a percent of the largest output per layer is allowed."""
    from linear_attention_ssm_step_gb300 import hybrid
    lens, steps = [75, 20, 133], [[50, 20, 100], [24, 0, 32], [1, 0, 1]]
    gen = torch.Generator(device=dev).manual_seed(3)
    x = [torch.randn((n, 512), generator=gen, device=dev).to(torch.bfloat16) for n in lens]
    outs = []
    for plan in ([lens], steps):
        model = hybrid.HybridLayers(hidden=512, layers="kka", heads=4, kv_heads=2, requests=3, pages=64, page_size=16,
                                    max_tokens=200, device=dev, seed=5)
        done, got = [0, 0, 0], [[], [], []]
        for new in plan:
            rows = torch.cat([x[r][done[r]:done[r] + n] for r, n in enumerate(new)])
            y = model.step(rows, new)
            at = 0
            for r, n in enumerate(new):
                got[r].append(y[at:at + n])
                at, done[r] = at + n, done[r] + n
        assert int(model.error_word.item()) == 0
        outs.append(torch.cat([torch.cat(g) for g in got]).float())
    assert (outs[0] - outs[1]).abs().max() <= 3 * 0.005 * outs[0].abs().max()


def test_hybrid_layers_leave_a_request_turned_down_as_it_was(dev):
    """A step whose pages run out for one request: its state, cache and length stay, and it goes on later as if that
    step had not been asked of it (the same bits: the later step has the same shapes)."""
    from linear_attention_ssm_step_gb300 import hybrid
    gen = torch.Generator(device=dev).manual_seed(4)
    x = [torch.randn((n, 256), generator=gen, device=dev).to(torch.bfloat16) for n in (31, 34)]
    outs = []
    for asked in (14, 0):
        model = hybrid.HybridLayers(hidden=256, layers="ka", heads=2, kv_heads=1, requests=2, pages=4, page_size=16,
                                    max_tokens=64, device=dev, seed=6)
        model.step(torch.cat([x[0][:30], x[1][:20]]), [30, 20])
        assert int(model.error_word.item()) == 0
        own = model.block_table[1, :2].long()
        state, cache, table = model.memory[0][1].clone(), model.memory[1][own].clone(), model.block_table.clone()
        model.step(torch.cat([x[0][30:], x[1][20:20 + asked]]), [1, asked])  # 34 tokens would take a fifth page
        assert int(model.error_word.item()) == (kda.KDA_ERR_PAGES if asked else 0)
        assert model.cached.tolist() == [31, 20] and int(model.free_count.item()) == 0
        assert torch.equal(model.memory[0][1], state) and torch.equal(model.memory[1][own], cache)
        assert torch.equal(model.block_table, table)
        outs.append(model.step(x[1][20:32], [0, 12]))
        assert model.cached.tolist() == [31, 32]
    assert torch.equal(outs[0], outs[1])
