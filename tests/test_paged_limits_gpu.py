"""The paged-attention calls on the GPU at their limits: many requests, rows and
bounds that go wrong, values that are not finite, other streams. Bounds and
their derivation: paged_cases.py."""

import numpy as np
import pytest
import torch

import paged_sequences as ps
from linear_attention_ssm_step_gb300 import kda
from paged_cases import Attention, ints, rope_bound, to_device

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


def on_device(a, dev):
    """The tensors of an attention problem, in the order of the call's arguments."""
    return (to_device(a.q, dev), to_device(a.k, dev), to_device(a.v, dev), ints(a.table, dev), ints(a.cu, dev),
            ints(a.kv, dev))


# ---------------------------------------------------------------- many requests

@pytest.mark.parametrize("R", [383, 384, 385, 767, 768, 769, 1536, 4096])
def test_attention_requests_in_blocks_of_the_sum(dev, R):
    """Above 384 requests each CTA sums them in blocks, twice: once for the whole and once to find its share. Ragged
    lengths, so that the warps of a CTA reach the second sum at different times, and many calls, with other work
    beside them: every call's rows are right and the same bits."""
    rng = np.random.default_rng(R)
    new = rng.integers(0, 3, R)
    kv = new + rng.integers(0, 30, R)
    for r, extra in ((0, 900), (R // 2, 2500), (R - 1, 400)):
        kv[r] += extra
    new[R // 3] += 300
    kv[R // 3] += 700
    a = Attention(new.tolist(), kv.tolist(), 4, 2, 64, 16, seed=R).poison()
    ws = kda.paged_attention_workspace(64, dev)
    err = err_word(dev)
    out, lse = a.run(dev, kda, workspace=ws, error_word=err)
    a.check(out, lse)
    args = on_device(a, dev)
    outs = [(torch.empty_like(out), torch.empty_like(lse)) for _ in range(40)]
    noise = torch.empty(1 << 25, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, (o, z) in enumerate(outs):
        if i % 3:
            with torch.cuda.stream(side):
                noise.add_(1.0)
        kda.kda_paged_attention(*args, out=o, lse=z, scale=a.scale, workspace=ws, error_word=err)
    torch.cuda.synchronize()
    for o, z in outs:
        assert torch.equal(o, out) and torch.equal(z, lse)
    assert int(err.item()) == 0 and (ws[:kda.KDA_ATTENTION_WORKSPACE_ZEROED] == 0).all()


# ---------------------------------------------------------------- bounds and rows

@pytest.mark.parametrize("D", [128, 64])
def test_attention_ranges_that_hold_too_many_rows(dev, D):
    """cu_new that jumps back gives the same rows to many requests: 2048 requests of 65536 rows over 65536 keys have
    more units than 32 bits count. The call ends, reports the bounds, and leaves its workspace ready."""
    T, R, Hq, page, pages = 65536, 4096, 64 * 64 // D, 256, 300
    heads = Hq  # 32 or 64 key-value heads
    units = 0
    for i in range(0, T, 256):  # the items of a request, 256 rows each: keys up to the last row's, four units of lead
        units += 4 + (i + 256) // 128
    assert R // 2 * units * heads > 2 ** 31
    gen = torch.Generator(device=dev).manual_seed(1)
    q = torch.randn((T, Hq, D), generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)
    k = torch.zeros((pages, page, heads, D), dtype=torch.bfloat16, device=dev)
    table = torch.arange(T // page, dtype=torch.int32, device=dev).expand(R, -1).contiguous()
    cu = torch.tensor([0, T] * (R // 2) + [0], dtype=torch.int32, device=dev)
    kv = torch.full((R,), T, dtype=torch.int32, device=dev)
    ws = kda.paged_attention_workspace(D, dev)
    err = err_word(dev)
    kda.kda_paged_attention(q, k, k.clone(), table, cu, kv, workspace=ws, error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == kda.KDA_ERR_SEQLENS
    a = Attention([3, 90], [40, 300], 4, 2, D, 16, seed=3)
    err.zero_()
    a.check(*a.run(dev, kda, workspace=ws, error_word=err))
    assert int(err.item()) == 0


@pytest.mark.parametrize("requests", [0, 3])
def test_plan_of_the_most_rows(dev, requests):
    """num_tokens of 2^31 - 1: the rows past the requests' get -1 up to the last one, and nothing is written beside
    the arrays (a row number that wrapped would be a store in front of them)."""
    T, page, pages, guard = 2 ** 31 - 1, 16, 40, 1 << 18
    words = torch.full((2, guard + T + guard + 1), 7, dtype=torch.int32, device=dev)
    positions, slots = words[0, guard:guard + T], words[1, guard:guard + T]
    new, cached = [5, 0, 30][:requests], [20, 3, 16][:requests]
    table = torch.full((requests, 4), -1, dtype=torch.int32, device=dev)
    for r, row in enumerate([[1, 2], [3], [4]][:requests]):
        table[r, :len(row)] = ints(row, dev)
    def new_ints(n):
        return torch.empty(n, dtype=torch.int32, device=dev)

    out = kda.PagedPlan(new_ints(requests + 1), new_ints(requests), positions, slots, new_ints(1))
    err = err_word(dev)
    kda.kda_paged_plan(ints(cached, dev), ints(new, dev), table, ints(np.arange(10, 20), dev), ints([10], dev), page,
                       pages, T, out=out, error_word=err)
    assert int(err.item()) == 0
    n = sum(new)
    if requests:
        assert positions[:n].tolist() == list(range(20, 25)) + list(range(16, 46))
        assert slots[:5].tolist() == list(range(2 * page + 4, 2 * page + 9))
        assert slots[5:21].tolist() == list(range(19 * page, 20 * page))
        assert slots[21:n].tolist() == list(range(18 * page, 18 * page + 14))
    for x in (positions, slots):
        for at in range(n, T, 1 << 27):
            assert (x[at:min(at + (1 << 27), T)] == -1).all()
    for side in (words[:, :guard], words[:, guard + T:]):
        assert (side == 7).all()


# ---------------------------------------------------------------- streams

def test_calls_on_another_stream_allocate_there(dev):
    """stream= without outputs or a workspace: what the call allocates belongs to that stream. The current stream is
    kept busy with writes into memory that it gave back to its pool, which a call on the other stream must not get,
    and a zeroing of the workspace that waited for them would come after the kernel."""
    a = Attention([1, 3], [3000, 5000], 8, 2, 128, 16, seed=21)
    args = on_device(a, dev)
    ref, _ = a.run(dev, kda)
    a.check(*a.run(dev, kda))
    T, Hq, D = a.q.shape
    freqs = kda.rope_freqs(D, device=dev)
    pos, slots = ints(np.arange(T), dev), ints(np.full(T, -1), dev)
    turned = kda.kda_rope_append(args[0], args[0][:, :2], args[0][:, :2], pos, slots, freqs, args[1], args[2])
    plan_in = (ints([5, 0], dev), ints([3, 1], dev), ints([[1, 2], [3, 4]], dev), ints(np.arange(8), dev), ints([8], dev))
    planned = kda.kda_paged_plan(*plan_in, 4, 16, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bytes_ = kda.paged_attention_workspace_bytes(D)
    for _ in range(5):
        big = torch.full((bytes_,), 7, dtype=torch.uint8, device=dev)
        small = [torch.full((T * Hq * D,), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(4)]
        few = [torch.full((n,), 7, dtype=torch.int32, device=dev) for n in (3, 2, 4, 4, 1) * 2]
        torch.cuda._sleep(20_000_000)  # about 10 ms, then the writes
        for t in [big] + small + few:
            t.fill_(9)
        del big, small, few, t
        out = kda.kda_paged_attention(*args, scale=a.scale, stream=side)
        q_out = kda.kda_rope_append(args[0], args[0][:, :2], args[0][:, :2], pos, slots, freqs, args[1], args[2],
                                    stream=side)
        plan = kda.kda_paged_plan(*plan_in, 4, 16, 4, stream=side)
        call = kda.prepare_paged_attention(*args, scale=a.scale, stream=side)
        prepared = call()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(prepared, ref) and torch.equal(q_out, turned)
        assert all(torch.equal(x, y) for x, y in zip(plan, planned))


def test_memory_of_a_call_on_another_stream_is_not_reused_early(dev):
    """An unprepared call drops its workspace when it returns, while its kernel has yet to run: the next allocations on
    the current stream must not get that memory."""
    a = Attention([1, 3], [3000, 5000], 8, 2, 128, 16, seed=22)
    args = on_device(a, dev)
    ref, _ = a.run(dev, kda)
    side = torch.cuda.Stream()
    bytes_ = kda.paged_attention_workspace_bytes(a.D)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = kda.kda_paged_attention(*args, scale=a.scale, stream=side)
        over = [torch.full((bytes_,), 9, dtype=torch.uint8, device=dev) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and len(over) == 3


# ---------------------------------------------------------------- workspace

@pytest.mark.parametrize("D", [128, 64, 96])
def test_workspace_needs_zeros_in_its_first_part_alone(dev, D, monkeypatch):
    """Cut items (two chunks), many parts (one token over a long cache): what lies past the zeroed part is not read
    before it is written, and the helper clears that part alone (its cost is one small fill, whatever the head size)."""
    zeroed = kda.KDA_ATTENTION_WORKSPACE_ZEROED
    a = Attention([300, 1, 8], [700, 20000, 900], 8, 2, D, 16, seed=23).poison()
    ws = kda.paged_attention_workspace(D, dev)
    assert (ws[:zeroed] == 0).all()
    ws[zeroed:].fill_(0xff)  # NaN as fp32
    err = err_word(dev)
    a.check(*a.run(dev, kda, workspace=ws, error_word=err))
    assert int(err.item()) == 0 and (ws[:zeroed] == 0).all()
    monkeypatch.setattr(kda, "_empty", lambda n, dtype, device, stream: torch.full((n,), 0xff, dtype=dtype, device=device))
    fresh = kda.paged_attention_workspace(D, dev)
    assert (fresh[:zeroed] == 0).all() and (fresh[zeroed:] == 0xff).all()


# ---------------------------------------------------------------- numbers that are not finite

NOT_FINITE = [(128, 16), (64, 16), (96, 16), (33, 5)]  # tensor cores, tensor cores, CUDA cores wide and narrow


def key_at(a, r, key):
    return int(a.table[r, key // a.page]), key % a.page


@pytest.mark.parametrize("D,page", NOT_FINITE)
def test_attention_key_of_minus_infinity(dev, D, page):
    """One key with -inf in it: where its score is -inf it has weight 0, the same bits as a key whose score is so low
    that its weight is 0 in fp32; where it is +inf, or -inf times 0, the row is NaN. Rows that do not see it are as
    without it."""
    rows = ([1, 150, 3], [300, 400, 260], 8, 2, D, page)
    key, low = 351, -2.0 ** 13  # of request 1, head 1; 2^13 D^-0.5 >= 512 below the others
    a, b = Attention(*rows, seed=24), Attention(*rows, seed=24)
    for x in (a, b):
        x.q[..., 0] = 1.0
        x.q[30, :, 0], x.q[140, :, 0] = 0.0, -1.0
    b.q[140, :, 0] = 1.0
    at, off = key_at(a, 1, key)
    a.k[at, off, 1, 0], b.k[at, off, 1, 0] = float("-inf"), low
    (o, z), (ob, zb) = a.run(dev, kda), b.run(dev, kda)
    b.check(ob, zb)
    bad = torch.zeros((154, 8), dtype=torch.bool, device=dev)
    bad[140, 4:] = True  # row 30 stands before the key, row 140 behind it
    same = ~bad
    same[140] = False
    assert torch.equal(o[same], ob[same]) and torch.equal(z[same], zb[same])
    assert torch.isnan(o[bad]).all() and torch.isnan(z[bad]).all()
    assert torch.isfinite(o[140, :4].float()).all() and torch.isfinite(z[140, :4]).all()
    a.q[140, :, 0] = 0.0
    o, z = a.run(dev, kda)
    assert torch.isnan(o[bad]).all() and torch.isnan(z[bad]).all()
    assert torch.equal(o[same], ob[same]) and torch.equal(z[same], zb[same])


@pytest.mark.parametrize("D,page", NOT_FINITE)
@pytest.mark.parametrize("new,kv,window", [
    ([1, 5, 1], [1, 5, 0], 0),         # one unit of keys, whole
    ([2], [20000], 0),                 # many parts of few rows
    ([300, 7, 9], [700, 500, 4], 0),   # parts of many rows; rows that see no key
    ([40, 1], [300, 200], 1),          # a row's own key alone
    ([60] * 3, [2000, 1500, 1800], 100),
])
def test_attention_scores_of_minus_infinity_alone(dev, D, page, new, kv, window):
    """Every key that a row sees has a score of -inf: out is 0 / 0, NaN, and lse -inf, from keys of -inf and from
    queries of +inf alike; a row that sees no key keeps its zeros."""
    for infinite in ("k", "q"):
        a = Attention(new, kv, 8, 2, D, page, window=window, seed=25)
        a.q[..., 0], a.k[..., 0] = (1.0, float("-inf")) if infinite == "k" else (float("inf"), -1.0)
        err = err_word(dev)
        o, z = a.run(dev, kda, error_word=err)
        pos = torch.tensor(np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)]), device=dev)
        assert int(err.item()) == 0 and torch.isneginf(z).all()
        assert torch.isnan(o[pos >= 0]).all() and (o[pos < 0] == 0).all()


@pytest.mark.parametrize("D,page", NOT_FINITE)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_attention_value_that_is_not_finite(dev, D, page, value):
    """It stays in its dimension of the rows of its request and head."""
    rows = ([1, 150, 3], [300, 400, 260], 8, 2, D, page)
    a, b = Attention(*rows, seed=26), Attention(*rows, seed=26)
    at, off = key_at(a, 1, 260)
    a.v[at, off, 1, 3] = value
    (o, z), (ob, zb) = a.run(dev, kda), b.run(dev, kda)
    b.check(ob, zb)
    assert torch.equal(z, zb)
    assert not torch.isfinite(o[1 + 10:151, 4:, 3].float()).any()  # row 10 of the request stands at key 260
    o[1:151, 4:, 3] = ob[1:151, 4:, 3]
    assert torch.equal(o, ob)


@pytest.mark.parametrize("D,page", NOT_FINITE)
def test_attention_query_of_infinity(dev, D, page):
    """Scores of both signs: +inf among them, so NaN, in that row and head alone."""
    rows = ([1, 150, 3], [300, 400, 260], 8, 2, D, page)
    a, b = Attention(*rows, seed=27), Attention(*rows, seed=27)
    a.q[0, 5, 2], a.q[20, 1, 2] = float("inf"), float("-inf")
    (o, z), (ob, zb) = a.run(dev, kda), b.run(dev, kda)
    b.check(ob, zb)
    for r, h in ((0, 5), (20, 1)):
        assert torch.isnan(o[r, h]).all() and torch.isnan(z[r, h])
        o[r, h], z[r, h] = ob[r, h], zb[r, h]
    assert torch.equal(o, ob) and torch.equal(z, zb)


# ---------------------------------------------------------------- hybrid layers

def test_hybrid_layers_turn_down_a_negative_length(dev):
    """-n tokens for a request of n cached ones: turned down, so its state, cache and length stay, and it goes on as
    if that step had asked nothing of it (the same bits: the later step has the same shapes)."""
    from linear_attention_ssm_step_gb300 import hybrid
    gen = torch.Generator(device=dev).manual_seed(7)
    x = [torch.randn((n, 256), generator=gen, device=dev).to(torch.bfloat16) for n in (31, 32)]
    outs = []
    for asked in (-20, 0):
        model = hybrid.HybridLayers(hidden=256, layers="ka", heads=2, kv_heads=1, requests=2, pages=8, page_size=16,
                                    max_tokens=64, device=dev, seed=6)
        model.step(torch.cat([x[0][:30], x[1][:20]]), [30, 20])
        own = model.block_table[1, :2].long()
        state, cache = model.memory[0][1].clone(), model.memory[1][own].clone()
        model.step(x[0][30:], [1, asked])
        assert int(model.error_word.item()) == (kda.KDA_ERR_LENGTHS if asked else 0)
        assert model.cached.tolist() == [31, 20]
        assert torch.equal(model.memory[0][1], state) and torch.equal(model.memory[1][own], cache)
        outs.append(model.step(x[1][20:], [0, 12]))
        assert model.cached.tolist() == [31, 32]
    assert torch.equal(outs[0], outs[1])


# ---------------------------------------------------------------- rows beside one another

@pytest.mark.parametrize("D", [128, 64, 96])
@pytest.mark.parametrize("by_heads", [False, True])
def test_outputs_beside_their_queries(dev, D, by_heads):
    """q and the outputs in the rows (or in the heads) of one buffer: the bits of outputs of their own, and q as it was."""
    a = Attention([1, 150, 5], [300, 400, 260], 8, 2, D, 16, seed=28).poison()
    args = on_device(a, dev)
    ref, lse = a.run(dev, kda)
    a.check(ref, lse)
    T, H = 156, 8
    both = torch.full((T, H, 2, D) if by_heads else (T, 2, H, D), 7.0, dtype=torch.bfloat16, device=dev)
    q, out = (both[:, :, 0], both[:, :, 1]) if by_heads else (both[:, 0], both[:, 1])
    q.copy_(args[0])
    kda.kda_paged_attention(q, *args[1:], out=out, scale=a.scale)
    assert torch.equal(out, ref) and torch.equal(q, args[0])
    freqs, pos, slots = kda.rope_freqs(D, device=dev), ints(np.arange(T), dev), ints(np.full(T, -1), dev)
    k = args[0][:, :2].clone()
    want = kda.kda_rope_append(args[0], k, k, pos, slots, freqs, args[1], args[2])
    kda.kda_rope_append(q, k, k, pos, slots, freqs, args[1], args[2], q_out=out)
    assert torch.equal(out, want) and torch.equal(q, args[0])


# ---------------------------------------------------------------- the three together

@pytest.mark.parametrize("D,page", [(128, 16), (64, 32), (96, 8)])
def test_every_token_of_the_three_together(dev, D, page):
    """Prompts in two chunks, then decode. Each position's key and value are where the block table says, turned (within
    the append's own bound) and as they were; and each row's attention is that of the whole sequence over the numbers
    that the GPU holds, within the attention's own bound (which test_paged_limits_host.py shows to be below what a
    token lost or misplaced changes)."""
    Hq, Hkv, pages = 8, 2, 48
    qkv = ps.sequences(Hq, Hkv, D, seed=14)
    gen = torch.Generator().manual_seed(15)
    kc = torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
    vc = kc.clone()
    table = torch.full((3, 200 // page), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=gen).to(torch.int32).to(dev)
    count, cached = ints([pages], dev), torch.zeros(3, dtype=torch.int32, device=dev)
    freqs = kda.rope_freqs(D // 2, 10000.0, kda.KDA_ROPE_LINEAR, 2.0, device=dev)
    turns = [int(x) % (1 << 64) for x in freqs.cpu().tolist()]
    err = err_word(dev)
    done, got = [0, 0, 0], [[[], [], []] for _ in range(3)]
    for new in ps.STEPS:
        rows = torch.cat([qkv[r][done[r]:done[r] + n] for r, n in enumerate(new)]).to(dev)
        plan = kda.kda_paged_plan(cached, ints(new, dev), table, free, count, page, pages, rows.shape[0], error_word=err)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        qo = kda.kda_rope_append(q, k, v, plan.positions, plan.slots, freqs, kc, vc, error_word=err)
        lse = torch.empty((rows.shape[0], Hq), dtype=torch.float32, device=dev)
        out = kda.kda_paged_attention(qo, kc, vc, table, plan.cu_new, plan.kv_len, lse=lse, error_word=err)
        at = 0
        for r, n in enumerate(new):
            for x, y in zip(got[r], (qo, out, lse)):
                x.append(y[at:at + n].double().cpu())
            at, done[r] = at + n, done[r] + n
        cached, count = plan.kv_len, plan.free_count
    assert int(err.item()) == 0 and done == ps.LENGTHS
    half = D // 4

    def partner(x):
        y = np.zeros_like(x)
        y[..., :half], y[..., half:2 * half] = x[..., half:2 * half], x[..., :half]
        return y

    for r, n in enumerate(ps.LENGTHS):
        q, out, lse = (torch.cat(x).numpy() for x in got[r])
        at = torch.arange(n, device=dev)
        where = table[r][at // page].long(), at % page
        k, v = kc[where].double().cpu().numpy(), vc[where].double().cpu().numpy()
        x = qkv[r].double().numpy()
        assert np.array_equal(v, x[:, Hq + Hkv:])
        q_ref, k_ref = ps.turned(qkv[r], Hq, Hkv, turns)
        for g, ref, start in ((q, q_ref, x[:, :Hq]), (k, k_ref, x[:, Hq:Hq + Hkv])):
            assert (np.abs(g - ref) <= rope_bound(ref, start, partner(start), 1.0)).all()
        o, z, tol, ztol = ps.attend(q, k, v)
        assert (np.abs(out - o) <= tol).all() and (np.abs(lse - z) <= ztol).all()


def test_pages_of_rejected_drafts_come_back(dev):
    """Verify steps of eight drafts of which some are rejected, and a request that ends: the caller puts the pages that
    are no longer needed back at the end of the free list, as the header says. No page is lost or owned twice, and the
    attention over what was kept is right."""
    Hq, Hkv, D, page, pages, R = 4, 2, 64, 4, 60, 3
    rng = np.random.default_rng(29)
    gen = torch.Generator().manual_seed(29)
    kc, vc = (torch.full((pages, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2))
    table = torch.full((R, 30), -1, dtype=torch.int32, device=dev)
    free = ints(rng.permutation(pages), dev)
    count, cached = ints([pages], dev), ints([0] * R, dev)
    freqs, err = torch.zeros(0, dtype=torch.int64, device=dev), err_word(dev)  # nothing turned: the keys as they are
    kept = [torch.zeros((0, 2, Hkv, D), dtype=torch.bfloat16) for _ in range(R)]  # keys and values of the kept tokens

    def give_back(r, tokens, count):
        held, still = -(-int(cached[r]) // page), -(-tokens // page)
        n = int(count.item())
        free[n:n + held - still] = table[r, still:held]
        cached[r] = tokens
        return count + (held - still)

    for step in range(12):
        new = [17, 5, 1] if step == 0 else [8] * R
        rows = torch.randn((sum(new), Hq + 2 * Hkv, D), generator=gen).to(torch.bfloat16)
        q, k, v = (x.to(dev) for x in (rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]))
        plan = kda.kda_paged_plan(cached, ints(new, dev), table, free, count, page, pages, sum(new), error_word=err)
        kda.kda_rope_append(q, k, v, plan.positions, plan.slots, freqs, kc, vc, error_word=err)
        out = kda.kda_paged_attention(q, kc, vc, table, plan.cu_new, plan.kv_len, error_word=err)
        cached, count = plan.kv_len.clone(), plan.free_count.clone()
        at = 0
        for r, n in enumerate(new):
            mine = rows[at:at + n]
            seen = torch.cat([kept[r], torch.stack([mine[:, Hq:Hq + Hkv], mine[:, Hq + Hkv:]], 1)])
            ref = np.zeros((len(seen), Hq, D))
            ref[len(seen) - n:] = mine[:, :Hq].double().numpy()
            o, _, tol, _ = ps.attend(ref, seen[:, 0].double().numpy(), seen[:, 1].double().numpy())
            got = out[at:at + n].double().cpu().numpy()
            assert (np.abs(got - o[-n:]) <= tol[-n:]).all()
            accepted = n if step == 0 else int(rng.integers(1, 9))
            tokens = 0 if step == 6 and r == 1 else len(seen) - n + accepted  # request 1 ends, and its row is used again
            kept[r] = seen[:tokens]
            count = give_back(r, tokens, count)
            at += n
        owned = [int(p) for r in range(R) for p in table[r, :-(-int(cached[r]) // page)]]
        assert sorted(owned + free[:int(count.item())].tolist()) == list(range(pages))
    assert int(err.item()) == 0
