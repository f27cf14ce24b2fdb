"""The paged-attention calls on the host, without a GPU: sizes and strides at
their limits, arguments that share a buffer, what the bounds of the tests tell
apart."""

import ctypes

import numpy as np
import pytest

import paged_sequences as ps
from linear_attention_ssm_step_gb300 import _build, kda
from test_paged_host import INVALID, UNSUPPORTED, fake_attention, fake_plan, fake_rope, no_gpu, put


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load_library()


def status(lib, p):
    """Of a call with these fake addresses. KDA_ELAUNCH: it passed the checks, and found no device."""
    if isinstance(p, kda.KdaPlanParams):
        return lib.kda_paged_plan(ctypes.byref(p), None)
    if isinstance(p, kda.KdaRopeParams):
        return lib.kda_rope_append(ctypes.byref(p), None)
    return lib.kda_paged_attention(ctypes.byref(p), 1 << 45, 1 << 30, None)


# ---------------------------------------------------------------- sizes

@no_gpu
@pytest.mark.parametrize("tensor", ["q", "k", "v", "q_out"])
def test_rope_rows_whose_span_passes_64_bits(lib, tensor):
    """2^31 - 1 rows 2^39 elements apart: the span, 2^70, must not wrap in the check of what overlaps what."""
    p = fake_rope()
    p.num_tokens = 2 ** 31 - 1
    put("q_out_b_stride" if tensor == "q_out" else tensor + ".b_stride", 1 << 39)(p)
    assert status(lib, p) == UNSUPPORTED
    assert f"{tensor} has rows that span" in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("tensor", ["q", "out"])
def test_attention_rows_whose_span_passes_64_bits(lib, tensor):
    p = fake_attention()
    p.num_tokens = 2 ** 31 // 4 - 1
    put("out_b_stride" if tensor == "out" else "q.b_stride", 1 << 39)(p)
    assert status(lib, p) == UNSUPPORTED
    assert f"{tensor} has rows that span" in kda.kda_last_error()


@no_gpu
def test_a_span_that_wraps_to_nothing_hides_no_overlap(lib):
    """2^31 - 1 rows of 2^33 elements (2^64 of them, less two rows): wrapped, an extent that ends before it begins, and
    in which q_out, although it stands there, does not lie."""
    p = fake_rope()
    p.num_tokens = 2 ** 31 - 1
    p.q.b_stride = 1 << 33
    assert status(lib, p) == UNSUPPORTED


@no_gpu
@pytest.mark.parametrize("make", [fake_plan, fake_attention])
def test_table_stride_past_40_bits(lib, make):
    p = make()
    p.table_stride = 1 << 61
    assert status(lib, p) == UNSUPPORTED
    assert "table_stride" in kda.kda_last_error()
    p.num_requests, p.table_stride = 1, 1 << 61  # a stride that is not used
    if isinstance(p, kda.KdaPlanParams):
        assert status(lib, p) == kda.KDA_ELAUNCH


# ---------------------------------------------------------------- rows beside one another

def set_rows(p, name, ptr, b, h):
    if name in ("out", "q_out"):
        setattr(p, name, ptr)
        setattr(p, name + "_b_stride", b)
        setattr(p, name + "_h_stride", h)
    else:
        setattr(p, name, kda.KdaView(ptr, b, 0, h))


FREE = kda.KDA_ELAUNCH  # past the checks: there is no device


@pytest.mark.parametrize("place,want", [
    ("columns", FREE),       # [T, q | out]: columns of one buffer's rows
    ("swapped", FREE),       # [T, out | q]
    ("heads", FREE),         # [T, H, q | out]: columns of its heads
    ("gap", FREE),           # columns with others between
    ("shifted", INVALID),    # out begins in q's last head
    ("wraps", INVALID),      # out ends in the next row's q
    ("other", INVALID),      # a row stride of its own: no common period
])
@no_gpu
@pytest.mark.parametrize("make", [fake_attention, fake_rope])
def test_rows_beside_one_another(lib, make, place, want):
    p = make()
    out = "out" if make is fake_attention else "q_out"
    H, D = p.num_q_heads, p.cache.head_dim
    base, row = 1 << 40, H * D
    q, o, b, h, ob = {"columns": (0, row, 2 * row, D, 2 * row), "swapped": (row, 0, 2 * row, D, 2 * row),
                      "heads": (0, D, 2 * row, 2 * D, 2 * row), "gap": (0, 2 * row, 4 * row, D, 4 * row),
                      "shifted": (0, row - 8, 2 * row, D, 2 * row), "wraps": (0, row + 8, 2 * row, D, 2 * row),
                      "other": (0, row, 2 * row, D, 3 * row)}[place]
    set_rows(p, "q", base + 2 * q, b, h)
    set_rows(p, out, base + 2 * o, ob, h)
    assert status(lib, p) == want
    if want == INVALID:
        assert "overlaps q" in kda.kda_last_error()


@no_gpu
def test_rows_that_share_an_element_are_always_refused(lib):
    """Against the sets of elements themselves, over many layouts (strides that repeat rows, heads across rows, rows
    between rows, odd offsets); and columns that share none are let through often enough to matter."""
    import random
    rng = random.Random(5)
    let_through = 0
    for _ in range(4000):
        p = fake_attention()
        T, Hkv, g, D = rng.choice([1, 2, 5]), rng.choice([1, 2]), rng.choice([1, 2]), rng.choice([1, 3, 8])
        H = Hkv * g
        p.num_tokens, p.num_q_heads, p.cache.num_heads, p.cache.head_dim = T, H, Hkv, D
        period = rng.choice([H * D, 2 * H * D, 2 * H * D + 1, 4 * D])
        lay = []
        for _ in range(2):
            h = rng.choice([D, 2 * D, 2 * D, period, rng.randrange(0, 3 * D + 1)])
            b = rng.choice([period, period, 2 * H * D, rng.randrange(0, 2 * period + 1)])
            lay.append((rng.choice([0, D, H * D, rng.randrange(0, 3 * H * D + 1)]), b, h))
        sets = [{at + t * b + i * h + c for t in range(T) for i in range(H) for c in range(D)} for at, b, h in lay]
        set_rows(p, "q", (1 << 40) + 2 * lay[0][0], *lay[0][1:])
        set_rows(p, "out", (1 << 40) + 2 * lay[1][0], *lay[1][1:])
        got = status(lib, p)
        assert got in (FREE, INVALID)
        apart = not (sets[0] & sets[1])
        assert apart or got == INVALID, (T, H, D, lay)
        if apart and max(min(s) for s in sets) < min(max(s) for s in sets):  # the ranges are not apart
            let_through += got == FREE
    assert let_through > 50


# ---------------------------------------------------------------- what the bounds tell apart

@pytest.mark.parametrize("D", [128, 64, 96])
def test_a_lost_or_misplaced_token_exceeds_the_bounds(D):
    """The sequences of the test of the three calls together: at the decode rows, whose newest key is the row's own,
    leaving that key out, or taking every key and value from the slot before, breaks the attention's bound."""
    Hq, Hkv = 8, 2
    turns = [int(2.0 ** 64 * 10000.0 ** (-4.0 * i / D) / 2 / (2 * np.pi)) for i in range(D // 4)]
    qkv = ps.sequences(Hq, Hkv, D, seed=14)
    for r, pos in ps.DECODE_ROWS:
        q, k = (ps.bf16(x) for x in ps.turned(qkv[r], Hq, Hkv, turns))
        v = qkv[r].double().numpy()[:, Hq + Hkv:]
        out, lse, tol, lse_tol = (x[pos] for x in ps.attend(q, k, v))
        lost = ps.oracle.paged_attention(q[pos:pos + 1], k[None], v[None], np.zeros((1, 1), int), [0, 1], [pos], D ** -0.5, 0)
        kb, vb = (np.concatenate([x[:1], x[:-1]]) for x in (k, v))
        back = ps.oracle.paged_attention(q[pos:pos + 1], kb[None], vb[None], np.zeros((1, 1), int), [0, 1], [pos + 1],
                                         D ** -0.5, 0)
        for wrong in (lost, back):
            # in some head: one in which the newest key has little weight cannot tell by its output
            assert (np.abs(wrong[0][0] - out) > tol).any()
            assert (np.abs(wrong[1][0] - lse) > lse_tol).any()
