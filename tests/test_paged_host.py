"""The paged-attention calls on the host, without a GPU: struct layouts,
constants, refusals before any launch, the frequency table, and the oracle
against closed forms and brute force."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import oracle
from linear_attention_ssm_step_gb300 import _build, kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_paged.h")

# Calls that pass fake host addresses, which validation rejects before any launch.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer checks run only without a GPU")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load_library()


# ---------------------------------------------------------------- header and binding

def test_constants_match_header():
    text = open(HEADER).read()
    for name in ("KDA_ERR_PAGES", "KDA_ERR_LENGTHS", "KDA_MAX_REQUESTS", "KDA_ATTENTION_WORKSPACE_ZEROED",
                 "KDA_ROPE_PLAIN", "KDA_ROPE_LINEAR", "KDA_ROPE_BASE", "KDA_ROPE_PARTS"):
        m = re.search(r"#define\s+" + name + r"\s+(\d+)u?\b", text)
        assert m and int(m.group(1)) == getattr(kda, name), name


def test_struct_layouts_match_header(tmp_path):
    structs = {"kda_pages": kda.KdaPages, "kda_paged_cache": kda.KdaPagedCache, "kda_plan_params": kda.KdaPlanParams,
               "kda_rope_params": kda.KdaRopeParams, "kda_attention_params": kda.KdaAttentionParams}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda_paged.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        key, val = line.rsplit(" ", 1)
        name, _, field = key.partition(".")
        want = getattr(structs[name], field).offset if field else ctypes.sizeof(structs[name])
        assert want == int(val), key


# ---------------------------------------------------------------- refusals

BASE = 1 << 33
MB = 1 << 24


def fake_cache(dim=128, heads=2, page=16, pages=8):
    c = kda.KdaPagedCache()
    c.k = kda.KdaPages(BASE, page * heads * dim, heads * dim, dim)
    c.v = kda.KdaPages(BASE + MB, page * heads * dim, heads * dim, dim)
    c.num_pages, c.page_size, c.num_heads, c.head_dim = pages, page, heads, dim
    return c


def fake_plan():
    p = kda.KdaPlanParams()
    p.num_requests, p.num_tokens, p.page_size, p.num_pages = 3, 40, 16, 20
    for i, f in enumerate(("cached", "new_len", "table", "free_pages", "free_count", "free_count_out", "cu_new",
                           "kv_len", "positions", "slots")):
        setattr(p, f, BASE + i * MB)
    p.table_stride, p.table_width, p.free_capacity = 8, 8, 20
    return p


def fake_rope():
    p = kda.KdaRopeParams()
    p.num_tokens, p.num_q_heads, p.rotary_dim, p.mscale = 5, 4, 128, 1.0
    p.cache = fake_cache()
    p.q = kda.KdaView(BASE + 2 * MB, 512, 0, 128)
    p.k = kda.KdaView(BASE + 3 * MB, 256, 0, 128)
    p.v = kda.KdaView(BASE + 4 * MB, 256, 0, 128)
    p.q_out, p.q_out_b_stride, p.q_out_h_stride = BASE + 5 * MB, 512, 128
    p.positions, p.slots, p.freqs = BASE + 6 * MB, BASE + 7 * MB, BASE + 8 * MB
    return p


def fake_attention():
    p = kda.KdaAttentionParams()
    p.num_requests, p.num_tokens, p.num_q_heads, p.scale = 3, 40, 4, 0.1
    p.cache = fake_cache()
    p.q = kda.KdaView(BASE + 2 * MB, 512, 0, 128)
    p.out, p.out_b_stride, p.out_h_stride = BASE + 3 * MB, 512, 128
    p.cu_new, p.kv_len, p.table = BASE + 4 * MB, BASE + 5 * MB, BASE + 6 * MB
    p.table_stride, p.table_width = 4, 4
    p.lse = BASE + 7 * MB
    return p


def put(path, value):
    def apply(p):
        *head, last = path.split(".")
        for h in head:
            p = getattr(p, h)
        setattr(p, last, value)
    return apply


INVALID, UNSUPPORTED = kda.KDA_EINVAL, kda.KDA_EUNSUPPORTED


@no_gpu
@pytest.mark.parametrize("path,value,status,message", [
    ("num_requests", -1, INVALID, "num_requests"),
    ("num_requests", 4097, UNSUPPORTED, "num_requests"),
    ("num_tokens", -1, INVALID, "num_tokens"),
    ("page_size", 0, INVALID, "page_size"),
    ("num_pages", -1, INVALID, "num_pages"),
    ("num_pages", 1 << 28, UNSUPPORTED, "2^31"),
    ("free_capacity", -1, INVALID, "free_capacity"),
    ("table_width", 0, INVALID, "table_width"),
    ("table_width", 1 << 28, UNSUPPORTED, "2^31 - 256"),
    ("table_stride", 7, INVALID, "table_stride"),
    ("table", None, INVALID, "table is NULL"),
    ("cached", None, INVALID, "cached is NULL"),
    ("new_len", BASE + 2, INVALID, "new_len is not 4-byte aligned"),
    ("free_pages", None, INVALID, "free_pages"),
    ("free_count", None, INVALID, "free_count"),
    ("free_count_out", BASE + 4 * MB, INVALID, "free_count_out overlaps free_count"),
    ("cu_new", None, INVALID, "cu_new"),
    ("kv_len", BASE, INVALID, "kv_len overlaps cached"),
    ("positions", None, INVALID, "positions"),
    ("slots", BASE + 8 * MB + 8, INVALID, "positions overlaps slots"),
    ("error_word", BASE + 9 * MB + 1, INVALID, "error_word"),
])
def test_plan_refusals(lib, path, value, status, message):
    p = fake_plan()
    put(path, value)(p)
    assert lib.kda_paged_plan(ctypes.byref(p), None) == status
    assert message in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("path,value,status,message", [
    ("num_tokens", -1, INVALID, "num_tokens"),
    ("num_q_heads", 0, INVALID, "num_q_heads"),
    ("rotary_dim", 63, INVALID, "rotary_dim"),
    ("rotary_dim", 130, INVALID, "rotary_dim"),
    ("rotary_dim", -2, INVALID, "rotary_dim"),
    ("mscale", float("nan"), INVALID, "mscale"),
    ("q.ptr", None, INVALID, "q is NULL"),
    ("k.ptr", BASE + 3 * MB + 1, INVALID, "k is not 2-byte aligned"),
    ("v.h_stride", -1, INVALID, "v has a negative stride"),
    ("v.b_stride", 1 << 41, UNSUPPORTED, "2^40"),
    ("q_out", None, INVALID, "q_out"),
    ("q_out", BASE + 2 * MB + 128, INVALID, "overlaps"),
    ("q_out", BASE + 100, INVALID, "cache overlaps"),
    ("positions", None, INVALID, "positions"),
    ("slots", None, INVALID, "slots"),
    ("freqs", BASE + 8 * MB + 4, INVALID, "freqs"),
    ("cache.head_dim", 257, UNSUPPORTED, "head_dim"),
    ("cache.num_heads", 0, INVALID, "num_heads"),
    ("cache.page_size", 0, INVALID, "page_size"),
    ("cache.num_pages", -1, INVALID, "num_pages"),
    ("cache.k.ptr", None, INVALID, "cache.k.ptr is NULL"),
    ("cache.v.token_stride", -8, INVALID, "cache.v has a negative stride"),
    ("cache.v.page_stride", 1 << 31, UNSUPPORTED, "2^31"),
])
def test_rope_refusals(lib, path, value, status, message):
    p = fake_rope()
    put(path, value)(p)
    assert lib.kda_rope_append(ctypes.byref(p), None) == status
    assert message in kda.kda_last_error()


@no_gpu
def test_rope_in_place_needs_the_same_strides(lib):
    p = fake_rope()
    p.q_out, p.q_out_b_stride = p.q.ptr, 1024
    assert lib.kda_rope_append(ctypes.byref(p), None) == INVALID
    assert "other strides" in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("path,value,status,message", [
    ("num_requests", -1, INVALID, "num_requests"),
    ("num_requests", 4097, UNSUPPORTED, "num_requests"),
    ("num_tokens", -1, INVALID, "num_tokens"),
    ("num_q_heads", 5, INVALID, "multiple"),
    ("num_q_heads", 2 * 129, UNSUPPORTED, "share"),
    ("window", -1, INVALID, "window"),
    ("scale", 0.0, INVALID, "scale"),
    ("scale", float("inf"), INVALID, "scale"),
    ("q.ptr", None, INVALID, "q is NULL"),
    ("out", None, INVALID, "out is NULL"),
    ("out", BASE + 2 * MB, INVALID, "out overlaps q"),
    ("lse", BASE + 64, INVALID, "lse overlaps cache.k"),
    ("lse", BASE + 7 * MB + 2, INVALID, "lse is not 4-byte aligned"),
    ("cu_new", None, INVALID, "cu_new"),
    ("kv_len", None, INVALID, "kv_len"),
    ("table", None, INVALID, "table"),
    ("table_width", 0, INVALID, "table_width"),
    ("table_stride", 3, INVALID, "table_stride"),
    ("cache.head_dim", 0, UNSUPPORTED, "head_dim"),
    ("cache.v.ptr", None, INVALID, "cache.v.ptr is NULL"),
    ("cache.page_size", 0, INVALID, "page_size"),
])
def test_attention_refusals(lib, path, value, status, message):
    p = fake_attention()
    put(path, value)(p)
    assert lib.kda_paged_attention(ctypes.byref(p), BASE + 9 * MB, 1 << 30, None) == status
    assert message in kda.kda_last_error()


@no_gpu
def test_null_params_and_empty_calls(lib):
    for fn in (lib.kda_paged_plan, lib.kda_rope_append):
        assert fn(None, None) == INVALID
    assert lib.kda_paged_attention(None, None, 0, None) == INVALID
    p = fake_rope()
    p.num_tokens = 0
    assert lib.kda_rope_append(ctypes.byref(p), None) == kda.KDA_OK
    a = fake_attention()
    a.num_tokens = 0
    assert lib.kda_paged_attention(ctypes.byref(a), None, 0, None) == kda.KDA_OK
    assert lib.kda_paged_attention_workspace_bytes(0) == lib.kda_paged_attention_workspace_bytes(257) == 0


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("rot", [2, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling,factor,original,low,high", [
    (0, 1.0, 0.0, 0.0, 0.0), (1, 8.0, 0.0, 0.0, 0.0), (2, 4.0, 0.0, 0.0, 0.0), (3, 8.0, 8192.0, 1.0, 4.0),
    (3, 32.0, 4096.0, 1.0, 32.0)])
def test_frequencies(lib, rot, scaling, factor, original, low, high):
    """Each within half a unit (2^-65 turns) of the 64-bit formula, and 2^-46 relatively: a power, products and
    divisions in doubles."""
    if scaling == 2 and rot == 2:
        pytest.skip("one pair has no slowest and fastest")
    got = [int(x) % (1 << 64) for x in kda.rope_freqs(rot, 500000.0, scaling, factor, original, low, high, device="cpu")]
    ref = oracle.rope_frequencies(rot, 500000.0, scaling, factor, original, low, high)
    for g, f in zip(got, ref):
        assert abs(g / 2.0 ** 64 * 2 * np.pi - f) <= 2.0 ** -46 * f + 2 * np.pi * 2.0 ** -65


def test_scaled_frequencies_have_their_ends(lib):
    plain = oracle.rope_frequencies(128, 10000.0, 0, 1, 0, 0, 0)
    based = oracle.rope_frequencies(128, 10000.0, 2, 4.0, 0, 0, 0)
    assert based[0] == plain[0] and abs(based[-1] * 4.0 / plain[-1] - 1) < 1e-12
    parts = oracle.rope_frequencies(128, 10000.0, 3, 4.0, 4096.0, 1.0, 32.0)
    turns = plain * 4096.0 / (2 * np.pi)
    assert np.allclose(parts[turns >= 32], plain[turns >= 32], rtol=1e-14)
    assert np.allclose(parts[turns <= 1], plain[turns <= 1] / 4.0, rtol=1e-14)


@pytest.mark.parametrize("args,message", [
    ((63, 10000.0, 0, 1.0, 0.0, 0.0, 0.0), "rotary_dim"), ((258, 10000.0, 0, 1.0, 0.0, 0.0, 0.0), "rotary_dim"),
    ((64, 1.0, 0, 1.0, 0.0, 0.0, 0.0), "base"), ((64, 10000.0, 4, 1.0, 0.0, 0.0, 0.0), "scaling"),
    ((64, 10000.0, 1, 0.5, 0.0, 0.0, 0.0), "factor"), ((2, 10000.0, 2, 2.0, 0.0, 0.0, 0.0), "KDA_ROPE_BASE"),
    ((64, 10000.0, 3, 2.0, 0.0, 1.0, 4.0), "KDA_ROPE_PARTS"), ((64, 10000.0, 3, 2.0, 8192.0, 4.0, 4.0), "KDA_ROPE_PARTS"),
])
def test_frequency_refusals(lib, args, message):
    host = (ctypes.c_uint64 * 256)()
    assert lib.kda_rope_freqs(ctypes.addressof(host), *args) == INVALID
    assert message in kda.kda_last_error()
    assert lib.kda_rope_freqs(None, 64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0) == INVALID


# ---------------------------------------------------------------- the oracle

def test_oracle_plan_by_hand():
    table = [[7, -1, -1], [3, -1, -1], [-1, -1, -1]]
    t, cu, kv, pos, slots, left, err = oracle.paged_plan([3, 4, 0], [2, 1, 0], table, [9, 8, 5], 3, 4, 10, 4)
    assert t.tolist() == [[7, 5, -1], [3, 8, -1], [-1, -1, -1]]
    assert cu.tolist() == [0, 2, 3, 3] and kv.tolist() == [5, 5, 0] and left == 1 and err == 0
    assert pos.tolist() == [3, 4, 4, -1] and slots.tolist() == [7 * 4 + 3, 5 * 4, 8 * 4, -1]


def test_oracle_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 2, 6))
    quarter = [1 << 62, 1 << 62]  # a quarter turn per position
    for inter, a, b in ((True, [0, 2], [1, 3]), (False, [0, 1], [2, 3])):
        y = oracle.rope_rotate(x, [0, 1, 2, 5], quarter, inter, 1.0)
        assert np.allclose(y[0], x[0]) and np.allclose(y[..., 4:], x[..., 4:])
        assert np.allclose(y[1][:, a], -x[1][:, b]) and np.allclose(y[1][:, b], x[1][:, a])
        assert np.allclose(y[2][..., :4], -x[2][..., :4]) and np.allclose(y[3][:, a], -x[3][:, b])
    # a score depends on the distance alone
    f = [int(2.0 ** 64 * 0.01), int(2.0 ** 64 * 0.0003)]
    p = oracle.rope_rotate(np.repeat(x[:1], 2, 0), [5, 105], f, False, 1.0)
    q = oracle.rope_rotate(np.repeat(x[1:2], 2, 0), [2, 102], f, False, 1.0)
    assert np.allclose((p[0] * q[0]).sum(-1), (p[1] * q[1]).sum(-1))


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(1)
    k = np.zeros((3, 4, 1, 5))
    v = rng.standard_normal((3, 4, 1, 5))
    q = rng.standard_normal((4, 2, 5))
    table = np.array([[2, 0, 1]])
    flat = v[[2, 0, 1]].reshape(12, 5)
    out, lse, _, _, count, err = oracle.paged_attention(q, k, v, table, [0, 4], [9], 0.5, 0)
    assert err == 0 and count.tolist() == [6, 7, 8, 9]
    for j in range(4):  # keys of zero: the mean of the values seen
        assert np.allclose(out[j], flat[:6 + j].mean(0)) and np.allclose(lse[j], np.log(6 + j))
    out, lse, *_ = oracle.paged_attention(q, k, v, table, [0, 4], [9], 0.5, 1)
    assert np.allclose(out[:, 0], flat[5:9])  # a window of one: the row's own value
    out, lse, *_ = oracle.paged_attention(q, k, v, table, [0, 4], [2], 0.5, 0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2], flat[0])
