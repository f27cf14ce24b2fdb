"""The calls on a paged cache in 8 bits at their limits on the GPU: a step of all of them together, streams, graphs,
offsets past 32 bits, shared workspaces, numbers that are not finite, waits that run out, hybrid layers. Bounds:
paged_fp8_cases.py."""

import numpy as np
import pytest
import torch

import oracle
from linear_attention_ssm_step_gb300 import kda
from paged_cases import Attention as Attention16
from paged_cases import ints, to_device
from paged_fp8_cases import TOKENS, Attention, cache, f64, half_step

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


def err_word(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def on_device(a, dev):
    return tuple(to_device(t, dev) for t in (a.q, a.k, a.v, a.ks, a.vs)) + (ints(a.table, dev), ints(a.cu, dev), ints(a.kv, dev))


# ---------------------------------------------------------------- together

def test_a_prompt_in_chunks_then_decode(dev):
    """Plan, append and attention step after step: each step's attention is that over the cache as it stands, the cache
    as the oracle's append leaves it from the GPU's own codes before the step, and what is read back are its values."""
    Hq, Hkv, D, page, R = 8, 2, 128, 16, 3
    gen = torch.Generator().manual_seed(14)
    steps = [[50, 20, 100], [25, 0, 31], [0, 0, 1], [3, 1, 2], [1, 1, 1]]
    lens = [sum(s[r] for s in steps) for r in range(R)]
    qkv = [(torch.randn((n, Hq + 2 * Hkv, D), generator=gen) * torch.exp(torch.randn((n, 1, 1), generator=gen))).to(torch.bfloat16)
           for n in lens]
    pages = 40
    sides = kda.paged_fp8_cache(pages, page, Hkv, D, dev)
    for x, value in zip(sides, (0x7F, 0x7F, float("nan"), float("nan"))):
        x.fill_(value)
    table = torch.full((R, 12), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=gen).to(torch.int32).to(dev)
    count, cached = ints([pages], dev), torch.zeros(R, dtype=torch.int32, device=dev)
    freqs = kda.rope_freqs(64, 10000.0, device=dev)
    turns = [int(x) % (1 << 64) for x in freqs.cpu().tolist()]
    err = err_word(dev)
    work = kda.paged_attention_workspace(D, dev)
    done = [0] * R
    for new in steps:
        rows = torch.cat([qkv[r][done[r]:done[r] + n] for r, n in enumerate(new)]).to(dev)
        plan = kda.kda_paged_plan(cached, ints(new, dev), table, free, count, page, pages, rows.shape[0], error_word=err)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        before = [x.cpu().numpy() for x in sides]
        qo = kda.kda_rope_append_fp8(q, k, v, plan.positions, plan.slots, freqs, *sides, error_word=err)
        lse = torch.empty((rows.shape[0], Hq), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention_fp8(qo, *sides, table, plan.cu_new, plan.kv_len, lse=lse, workspace=work, error_word=err)
        _, keys, values, _, bits = oracle.rope_append_fp8(f64(q), f64(k), f64(v), plan.positions.tolist(), plan.slots.tolist(),
                                                          turns, before[0], before[1], before[2], before[3], False, 1.0)
        assert bits == 0
        assert np.array_equal(sides[1].cpu().numpy(), values[0])
        assert np.array_equal(f64(sides[3]), values[1], equal_nan=True)
        assert np.array_equal(f64(sides[2]), keys[1], equal_nan=True)
        assert (sides[0].cpu().numpy() != keys[0]).mean() <= 1e-4  # ties of the turn
        a = Attention.__new__(Attention)
        a.Hq, a.Hkv, a.D, a.page, a.window, a.scale = Hq, Hkv, D, page, 0, D ** -0.5
        a.q, a.k, a.v, a.ks, a.vs = (x.cpu() for x in (qo, *sides))
        a.table, a.cu, a.kv, a.new = table.cpu().numpy(), plan.cu_new.cpu().numpy(), plan.kv_len.cpu().numpy(), new
        a.check(out, lse)
        read = kda.kda_paged_read_fp8(*sides, table, plan.cu_new, plan.kv_len, rows.shape[0], error_word=err)
        kk, vv = a.values()
        at = plan.slots.cpu().numpy()
        for g, x in zip(read, (kk, vv)):
            assert np.array_equal(f64(g), x.reshape(-1, Hkv, D)[at])
        for r, n in enumerate(new):
            done[r] += n
        cached, count = plan.kv_len, plan.free_count
    assert int(err.item()) == 0


# ---------------------------------------------------------------- streams, graphs, workspaces

@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64])
def test_captured_and_replayed_on_new_contents(dev, D, shape):
    """One graph of append, attention and read, replayed after every input has changed: the bits of eager calls."""
    Hq, Hkv, page = 8, 2, 32
    cases = [Attention(*shape, Hq, Hkv, D, page, seed=s) for s in (40, 41)]
    gen = torch.Generator().manual_seed(42)
    T = cases[0].q.shape[0]
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(*shape)])
    owner = np.repeat(np.arange(3), shape[0])
    freqs = kda.rope_freqs(D, device=dev)
    inputs = []
    for a in cases:
        k, v = (torch.randn((T, Hkv, D), generator=gen).to(torch.bfloat16).to(dev) for _ in range(2))
        slots = ints(a.table[owner, pos // page] * page + pos % page, dev)
        inputs.append([k, v, slots, ints(pos, dev), *on_device(a, dev)])

    def step(k, v, slots, at, q, kc, vc, ks, vs, table, cu, kv, work):
        qo = kda.kda_rope_append_fp8(q, k, v, at, slots, freqs, kc, vc, ks, vs)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention_fp8(qo, kc, vc, ks, vs, table, cu, kv, lse=lse, workspace=work)
        read = kda.kda_paged_read_fp8(kc, vc, ks, vs, table, cu, kv, T)
        return qo, out, lse, *read, kc, vc, ks, vs

    work = kda.paged_attention_workspace(D, dev)
    eager = [step(*[x.clone() for x in i], work) for i in inputs]
    held = [x.clone() for x in inputs[0]]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        step(*held, work)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held, work)
    for i in (1, 0, 1):
        for x, y in zip(held, inputs[i]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, eager[i]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("shape", [CHUNKS, FEW])
def test_calls_on_another_stream_allocate_there(dev, shape):
    """stream= without outputs or a workspace, while the current stream writes into memory that it has given back."""
    a = Attention(*shape, 8, 2, 128, 16, seed=21)
    args = on_device(a, dev)
    T, Hq, D = a.q.shape
    none = torch.zeros(0, dtype=torch.int64, device=dev)
    at = ints(np.arange(T), dev), ints(np.full(T, -1), dev)
    rows = args[0][:, :2]
    ref = (kda.kda_paged_attention_fp8(*args), kda.kda_rope_append_fp8(args[0], rows, rows, *at, none, *args[1:5]),
           *kda.kda_paged_read_fp8(*args[1:], T))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        big = torch.full((kda.paged_attention_workspace_bytes(D),), 7, dtype=torch.uint8, device=dev)
        small = [torch.full((T * Hq * D,), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(6)]
        torch.cuda._sleep(20_000_000)
        for t in [big] + small:
            t.fill_(9)
        del big, small, t
        got = (kda.kda_paged_attention_fp8(*args, stream=side),
               kda.kda_rope_append_fp8(args[0], rows, rows, *at, none, *args[1:5], stream=side),
               *kda.kda_paged_read_fp8(*args[1:], T, stream=side))
        torch.cuda.synchronize()
        for x, y in zip(got, ref):
            assert torch.equal(x, y)


def test_one_workspace_for_both_caches(dev):
    """The calls on 16 and on 8 bits take turns with a workspace, for chunks and few rows, and leave it ready."""
    work = kda.paged_attention_workspace(128, dev)
    for seed in range(2):
        for shape in (FEW, CHUNKS):
            a = Attention(*shape, 8, 2, 128, 64, seed=seed)
            b = Attention16(*shape, 8, 2, 128, 64, seed=seed)
            a.check(*a.run(dev, kda, workspace=work))
            b.check(*b.run(dev, kda, workspace=work))
    assert (work[:kda.KDA_ATTENTION_WORKSPACE_ZEROED] == 0).all()


@pytest.mark.parametrize("D,Hq,Hkv,new,kv", [(128, 4, 1, [1], [30000]), (64, 8, 2, [1, 2], [9000, 12345]),
                                             (128, 4, 1, [300], [4000]), (64, 4, 2, [90, 200], [3000, 700])])
def test_attention_same_bits_whatever_the_order_of_arrival(dev, D, Hq, Hkv, new, kv):
    """Items cut between many CTAs, while another stream disturbs their order."""
    a = Attention(new, kv, Hq, Hkv, D, 64, seed=11)
    work = kda.paged_attention_workspace(D, dev)
    args = on_device(a, dev)
    ref = a.run(dev, kda, workspace=work)
    a.check(*ref)
    side, noise = torch.cuda.Stream(), torch.zeros(1 << 24, device=dev)
    outs = []
    for i in range(8):
        if i % 2:
            with torch.cuda.stream(side):
                noise.add_(1.0)
        outs.append(kda.kda_paged_attention_fp8(*args, scale=a.scale, workspace=work))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref[0]) for x in outs)


# ---------------------------------------------------------------- sizes

@pytest.mark.parametrize("new,kv", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64, 96])
def test_pages_past_2_to_the_31_elements(dev, D, new, kv):
    """Append, attention and read in the last pages of a cache of more than 2^31 codes: the same bits as in a small one."""
    Hq, Hkv, page = 16, 8, 64
    a = Attention(new, kv, Hq, Hkv, D, page, seed=15)
    T, few = sum(new), a.k.shape[0]
    many = 2 ** 31 // (page * Hkv * D) + few + 8
    first = many - few
    gen = torch.Generator().manual_seed(16)
    q, k, v = (torch.randn((T, h, D), generator=gen).to(torch.bfloat16).to(dev) for h in (Hq, Hkv, Hkv))
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)])
    owner = np.repeat(np.arange(3), new)
    slots = a.table[owner, pos // page] * page + pos % page
    freqs = kda.rope_freqs(D, device=dev)
    got = []
    for base, pages in ((0, few), (first, many)):
        sides = kda.paged_fp8_cache(pages, page, Hkv, D, dev)
        for x, y in zip(sides, (a.k, a.v, a.ks, a.vs)):
            x[base:].copy_(y)
        err = err_word(dev)
        qr = kda.kda_rope_append_fp8(q, k, v, ints(pos, dev), ints(slots + base * page, dev), freqs, *sides, error_word=err)
        table = ints(np.where(a.table < 0, a.table, a.table + base), dev)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention_fp8(qr, *sides, table, ints(a.cu, dev), ints(a.kv, dev), lse=lse, error_word=err)
        read = kda.kda_paged_read_fp8(*sides, table, ints(a.cu, dev), ints(a.kv, dev), T, error_word=err)
        assert int(err.item()) == 0
        got.append([x.clone() for x in (qr, out, lse, *read, *(s[base:] for s in sides))])
        del sides
    assert not torch.equal(got[0][5], a.k.to(dev)), "the rows were appended"
    for x, y in zip(*got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("R,few", [(383, True), (800, True), (kda.KDA_MAX_REQUESTS, True), (383, False), (800, False)])
def test_attention_of_many_requests(dev, R, few):
    """Requests in several blocks of the sum over their lengths."""
    new = [1] * R if few else [(40 if i % 8 == 0 else 0) for i in range(R)]
    kv = [n + (7 * i) % 40 for i, n in enumerate(new)]
    a = Attention(new, kv, 4 if few else 8, 2 if few else 1, 64, 16, seed=R)
    a.check(*a.run(dev, kda))


def test_append_of_many_requests(dev):
    """Rows enough for a CTA of the append to look for runs in several rows, single ones and whole blocks in turn."""
    from test_paged_fp8_gpu import Append
    lengths = [(1, 16, 3, 1, 30)[i % 5] for i in range(260)]
    a = Append(lengths, [(5 * i) % 37 for i in range(260)], 4, 2, 64, 64, False, 16, "thd", seed=9)
    assert sum(lengths) > 2048
    a.check(*a.run(dev))
    a = Append([9000], [5], 2, 1, 64, 32, True, 32, "thd", seed=10)
    a.check(*a.run(dev, "in place"))


# ---------------------------------------------------------------- numbers

@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (80, 16)])
def test_queries_and_codes_that_are_not_finite(dev, D, page, shape):
    """A query with an infinite or NaN number gives NaN in its row and head alone; a NaN code of a key NaN in the rows of
    its head that see it; a NaN code of a value NaN in its dimension of those rows."""
    a = Attention(*shape, 4, 2, D, page, seed=31)
    ref, ref_lse = a.run(dev, kda)
    last = a.q.shape[0] - 1                    # a row of the third request
    a.q[last, 1, 3] = float("inf")
    a.q[0, 2, 5] = float("nan")
    out, lse = a.run(dev, kda)
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device=dev)
    bad[last, 1] = bad[0, 2] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], ref[~bad]) and torch.equal(lse[~bad], ref_lse[~bad])
    a = Attention(*shape, 4, 2, D, page, seed=31)
    a.k[int(a.table[0, 0]), 2, 1, 4] = 0xFF    # key 2 of the first request, heads 2 and 3
    a.v[int(a.table[2, 0]), 5, 0, 7] = 0x7F    # value 5 of the third request, heads 0 and 1
    out, lse = a.run(dev, kda)
    rows = slice(int(a.cu[0]), int(a.cu[1]))
    assert out[rows, 2:].isnan().all() and lse[rows, 2:].isnan().all()
    assert torch.equal(out[rows, :2], ref[rows, :2])
    rows = slice(int(a.cu[2]), int(a.cu[3]))
    assert torch.equal(lse[rows], ref_lse[rows]) and torch.equal(out[rows, 2:], ref[rows, 2:])
    seen = [t for t in range(rows.start, rows.stop) if a.kv[2] - a.new[2] + t - rows.start >= 5]
    assert out[seen, :2, 7].isnan().all()
    keep = [c for c in range(D) if c != 7]
    assert torch.equal(out[rows, :2][:, :, keep], ref[rows, :2][:, :, keep])


@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64, 80])
def test_scales_far_apart(dev, D, shape):
    """Value blocks whose scales differ by 2^60, key blocks of 2^-40 and large ones; queries of 2^-60 and 2^60."""
    a = Attention(*shape, 4, 2, D, 32, seed=33)
    gen = torch.Generator().manual_seed(34)
    a.vs *= 2.0 ** torch.randint(-30, 31, a.vs.shape, generator=gen).float()
    a.ks[::3] = 2.0 ** -40
    a.check(*a.run(dev, kda))
    a = Attention(*shape, 4, 2, D, 32, seed=35)
    a.q[:, 0] *= 2.0 ** -60
    a.ks *= 2.0 ** -30
    a.q[:, 1] *= 2.0 ** 30
    a.check(*a.run(dev, kda))


@pytest.mark.parametrize("new", [[1], [2, 1], [60]])
def test_one_key_far_above_many_others(dev, new):
    """A first key that takes most of the weight, and 20000 others with 2^-19 of it each, whose values all point the same
    way: together they are 4 % of the output, which must not vanish."""
    D, Hkv = 128, 1
    a = Attention(new, [20000 + n for n in new], 4, Hkv, D, 64, seed=36)
    a.q[:] = 0
    a.q[:, :, 0] = 1.0
    for t, s in ((a.k, a.ks), (a.v, a.vs)):
        t[:], s[:] = 0, 1.0
    a.v[..., 3] = 0x38  # 1
    for r in range(len(new)):
        page = int(a.table[r, 0])
        a.k[page, 0, 0, 0] = 0x50   # 8
        a.ks[page, 0, 0] = 19 * float(np.log(2)) / 8 / a.scale
        a.v[page, 0, 0, 3] = 0
        a.v[page, 0, 0, 5] = 0x38
    out, lse = a.run(dev, kda)
    a.check(out, lse)
    o = a.oracle()[0]
    assert abs(o[0, 0, 3] - 20000 * 2.0 ** -19 / (1 + 20000 * 2.0 ** -19)) < 1e-3
    assert np.abs(f64(out)[..., 3] - o[..., 3]).max() <= 2.0 ** -6 * o[0, 0, 3]


def test_attention_over_a_cache_read_back_in_16_bits(dev):
    """The cache read back is what the attention attends over: kda_paged_attention on it gives the same within the bounds
    of both (the 16-bit call rounds its weights to bf16)."""
    a = Attention([3, 60], [300, 200], 4, 2, 128, 16, seed=37)
    out, lse = a.run(dev, kda)
    k, v = (torch.from_numpy(x).to(torch.bfloat16).to(dev) for x in a.values())
    z = torch.empty_like(lse)
    o = kda.kda_paged_attention(to_device(a.q, dev), k, v, *(ints(x, dev) for x in (a.table, a.cu, a.kv)), lse=z, scale=a.scale)
    ref = a.oracle()
    tol, ztol = a.bounds(ref)
    assert (np.abs(f64(out) - f64(o)) <= 2 * tol + 2.0 ** -8 * ref[2]).all()
    assert (np.abs(f64(lse) - f64(z)) <= 2 * ztol).all()


# ---------------------------------------------------------------- requests that are wrong

@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64, 80])
def test_bad_requests_are_skipped_and_reported(dev, D, shape):
    a = Attention(*shape, 4, 2, D, 16, seed=38)
    a.kv[1] = 10 ** 6
    a.table[2, 1] = a.k.shape[0]
    ref = a.oracle()
    err = err_word(dev)
    out, lse = a.run(dev, kda, error_word=err)
    a.check(out, lse, ref)
    assert int(err.item()) == ref[5] == kda.KDA_ERR_LENGTHS | kda.KDA_ERR_PAGES
    a = Attention(*shape, 4, 2, D, 16, seed=39)
    a.cu = a.cu.copy()
    a.cu[2] = -1  # neither the second request nor the third
    ref = a.oracle()
    err.zero_()
    out, lse = a.run(dev, kda, error_word=err)
    a.check(out, lse, ref)
    assert int(err.item()) == ref[5] == kda.KDA_ERR_SEQLENS


@pytest.mark.parametrize("few", [True, False])
def test_ranges_that_hold_too_many_rows(dev, few):
    """cu_new that jumps back gives the same rows to many requests: nothing is done, and the workspace is left ready."""
    T, R, page, pages = (64, 64, 16, 8) if few else (4096, 64, 64, 70)
    q = torch.zeros((T, 4, 128), dtype=torch.bfloat16, device=dev)
    sides = kda.paged_fp8_cache(pages, page, 1, 128, dev)
    table = torch.zeros((R, pages), dtype=torch.int32, device=dev)
    cu = ints([0, T] * (R // 2) + [0], dev)
    kv = ints([T] * R, dev)
    work = kda.paged_attention_workspace(128, dev)
    out = torch.full((T, 4, 128), 7.0, dtype=torch.bfloat16, device=dev)
    err = err_word(dev)
    kda.kda_paged_attention_fp8(q, *sides, table, cu, kv, out=out, workspace=work, error_word=err)
    assert int(err.item()) == kda.KDA_ERR_SEQLENS and (out == 7).all()
    a = Attention(*FEW, 8, 2, 128, 16, seed=3)
    a.check(*a.run(dev, kda, workspace=work))


@pytest.mark.parametrize("shape", [CHUNKS, FEW])
@pytest.mark.parametrize("D", [128, 64])
def test_attention_wait_that_runs_out(dev, D, shape):
    """Failure detection without a fault: in the build that issues no copy (tests/test_timeout_gpu.py) the bounded waits
    run out, the call reports KDA_ERR_TIMEOUT and returns, and the context stays usable."""
    from linear_attention_ssm_step_gb300 import _build
    wlib = kda.bind_library(_build.build(variant="waittest"))
    a = Attention(*shape, 4, 2, D, 16, seed=18)
    err = err_word(dev)
    call = kda.prepare_paged_attention_fp8(*on_device(a, dev), error_word=err)
    assert wlib.kda_paged_attention_fp8(*call._args) == kda.KDA_OK
    torch.cuda.synchronize()
    assert int(err.item()) == kda.KDA_ERR_TIMEOUT
    a.check(*a.run(dev, kda))


def test_calls_without_work(dev):
    sides = kda.paged_fp8_cache(2, 16, 2, 64, dev)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=dev)
    zero, none = ints([0], dev), torch.zeros(0, dtype=torch.int32, device=dev)
    table = torch.zeros((1, 1), dtype=torch.int32, device=dev)
    assert kda.kda_paged_attention_fp8(q, *sides, table, ints([0, 0], dev), zero).shape == (0, 4, 64)
    assert kda.kda_paged_read_fp8(*sides, table, ints([0, 0], dev), zero, 0).k.shape == (0, 2, 64)
    freqs = torch.zeros(0, dtype=torch.int64, device=dev)
    assert kda.kda_rope_append_fp8(q, q[:, :2], q[:, :2], none, none, freqs, *sides).shape == (0, 4, 64)
    empty = kda.paged_fp8_cache(0, 16, 2, 64, dev)  # no pages: rows get zeros
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device=dev)
    err = err_word(dev)
    out = kda.kda_paged_attention_fp8(q, *empty, table, ints([0, 3], dev), ints([3], dev), error_word=err)
    assert (out == 0).all() and int(err.item()) == kda.KDA_ERR_PAGES


# ---------------------------------------------------------------- hybrid layers

def test_hybrid_layers_on_a_cache_in_8_bits(dev):
    """KDA and attention layers with keys and values in 8 bits: the first step's cache is the 16-bit one's, rounded; the
    outputs differ from those on 16 bits by no more than a code's rounding makes of them (2^-4 of a value at most, spread
    over the keys and a residual: a twentieth of the largest output is allowed)."""
    from linear_attention_ssm_step_gb300 import hybrid
    gen = torch.Generator(device=dev).manual_seed(3)
    steps = [[50, 20, 100], [24, 0, 32], [1, 1, 1]]
    x = [torch.randn((sum(n), 512), generator=gen, device=dev).to(torch.bfloat16) for n in steps]
    outs, caches = [], []
    for bits in (16, 8):
        model = hybrid.HybridLayers(hidden=512, layers="kaka", heads=4, kv_heads=2, requests=3, pages=64, page_size=16,
                                    max_tokens=200, device=dev, seed=5, cache_bits=bits)
        y = [model.step(x[0], steps[0])]
        caches.append(model.cached_rows(1))
        y += [model.step(rows, n) for rows, n in zip(x[1:], steps[1:])]
        assert int(model.error_word.item()) == 0
        assert model.cached_rows(3).k.shape == (229, 2, 128)
        outs.append(torch.cat(y).float())
    for a, b in zip(*caches):  # the same numbers went in: the KDA layer before is the same
        a, b = a.double(), b.double()
        top = torch.cat([s.abs().amax(dim=(0, 2), keepdim=True).expand_as(s) for r in a.split([50, 20, 100])
                         for s in r.split(TOKENS)])
        assert ((a - b).abs() <= 2.0 ** -4 * a.abs() + 2.0 ** -10 * top / 220 + 2.0 ** -8 * a.abs()).all()
    assert (outs[0] - outs[1]).abs().max() <= 0.05 * outs[0].abs().max()
    with pytest.raises(ValueError):
        hybrid.HybridLayers(cache_bits=4, device=dev)
