"""The calls on a paged cache in 8 bits on the host, without a GPU: struct layouts, refusals before any launch, the
oracle against closed forms and brute force, and mistakes planted in it."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import oracle
from linear_attention_ssm_step_gb300 import _build, kda
from oracle import kda_paged_fp8_oracle as fp8
from paged_fp8_cases import Attention, half_step
from test_paged_host import BASE, INVALID, MB, UNSUPPORTED, fake_attention, fake_rope, no_gpu, put

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load_library()


# ---------------------------------------------------------------- header and binding

def test_header_and_binding(tmp_path):
    text = open(os.path.join(ROOT, "include", "kda_paged_fp8.h")).read()
    assert int(re.search(r"#define\s+KDA_FP8_SCALE_TOKENS\s+(\d+)", text).group(1)) == kda.KDA_FP8_SCALE_TOKENS == fp8.SCALE_TOKENS
    structs = {"kda_page_scales": kda.KdaPageScales, "kda_paged_scales": kda.KdaPagedScales, "kda_read_params": kda.KdaReadParams}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kda_paged_fp8.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        key, val = line.rsplit(" ", 1)
        name, _, field = key.partition(".")
        assert (getattr(structs[name], field).offset if field else ctypes.sizeof(structs[name])) == int(val), key


# ---------------------------------------------------------------- refusals

def fake_scales():
    return kda.KdaPagedScales(kda.KdaPageScales(BASE + 12 * MB, 2, 2, 1), kda.KdaPageScales(BASE + 13 * MB, 2, 2, 1))


def fake_read():
    p = kda.KdaReadParams()
    p.num_requests, p.num_tokens = 3, 40
    p.cache = fake_attention().cache
    p.k_out, p.k_out_b_stride, p.k_out_h_stride = BASE + 2 * MB, 256, 128
    p.v_out, p.v_out_b_stride, p.v_out_h_stride = BASE + 3 * MB, 256, 128
    p.cu_rows, p.kv_len, p.table = BASE + 4 * MB, BASE + 5 * MB, BASE + 6 * MB
    p.table_stride, p.table_width = 4, 4
    return p


def status(lib, p, sc):
    ref = ctypes.byref(sc) if sc is not None else None
    if isinstance(p, kda.KdaRopeParams):
        return lib.kda_rope_append_fp8(ctypes.byref(p), ref, None)
    if isinstance(p, kda.KdaReadParams):
        return lib.kda_paged_read_fp8(ctypes.byref(p), ref, None)
    return lib.kda_paged_attention_fp8(ctypes.byref(p), ref, BASE + 9 * MB, 1 << 30, None)


@no_gpu
@pytest.mark.parametrize("make", [fake_rope, fake_attention, fake_read])
@pytest.mark.parametrize("path,value,want,message", [
    ("k.ptr", None, INVALID, "scales.k.ptr is NULL"),
    ("v.ptr", BASE + 13 * MB + 2, INVALID, "scales.v.ptr is not 4-byte aligned"),
    ("k.page_stride", -1, INVALID, "scales.k has a negative stride"),
    ("v.block_stride", 1 << 31, UNSUPPORTED, "scales.v has a stride of 2^31"),
    ("v.head_stride", -4, INVALID, "scales.v has a negative stride"),
])
def test_scales_refusals(lib, make, path, value, want, message):
    sc = fake_scales()
    put(path, value)(sc)
    assert status(lib, make(), sc) == want
    assert message in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("make", [fake_rope, fake_attention, fake_read])
def test_scales_missing_and_params_missing(lib, make):
    assert status(lib, make(), None) == INVALID and "scales is NULL" in kda.kda_last_error()
    assert lib.kda_rope_append_fp8(None, None, None) == INVALID
    assert lib.kda_paged_read_fp8(None, None, None) == INVALID
    assert lib.kda_paged_attention_fp8(None, None, None, 0, None) == INVALID


@no_gpu
@pytest.mark.parametrize("path,value,want,message", [
    ("num_tokens", -1, INVALID, "num_tokens"),
    ("num_tokens", (1 << 30) + 1, UNSUPPORTED, "2^30"),
    ("rotary_dim", 63, INVALID, "rotary_dim"),
    ("mscale", float("inf"), INVALID, "mscale"),
    ("q_out", BASE + 100, INVALID, "cache overlaps"),
    ("q_out", BASE + 12 * MB, INVALID, "scales overlap"),
    ("k.ptr", BASE + 13 * MB + 4, INVALID, "scales overlap"),
    ("cache.k.ptr", None, INVALID, "cache.k.ptr is NULL"),
    ("cache.head_dim", 257, UNSUPPORTED, "head_dim"),
    ("cache.v.page_stride", 1 << 31, UNSUPPORTED, "2^31"),
    ("slots", None, INVALID, "slots"),
])
def test_append_refusals(lib, path, value, want, message):
    p = fake_rope()
    put(path, value)(p)
    assert status(lib, p, fake_scales()) == want
    assert message in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("path,value,want,message", [
    ("num_requests", 4097, UNSUPPORTED, "num_requests"),
    ("num_q_heads", 5, INVALID, "multiple"),
    ("window", -1, INVALID, "window"),
    ("scale", 0.0, INVALID, "scale is not"),
    ("out", BASE + 12 * MB, INVALID, "out overlaps scales.k"),
    ("lse", BASE + 13 * MB, INVALID, "lse overlaps scales.v"),
    ("lse", BASE + 64, INVALID, "lse overlaps cache.k"),
    ("kv_len", None, INVALID, "kv_len"),
    ("table_stride", 3, INVALID, "table_stride"),
])
def test_attention_refusals(lib, path, value, want, message):
    p = fake_attention()
    put(path, value)(p)
    assert status(lib, p, fake_scales()) == want
    assert message in kda.kda_last_error()


@no_gpu
@pytest.mark.parametrize("path,value,want,message", [
    ("num_requests", -1, INVALID, "num_requests"),
    ("num_tokens", -1, INVALID, "num_tokens"),
    ("k_out", None, INVALID, "k_out is NULL"),
    ("v_out", BASE + 3 * MB + 1, INVALID, "v_out is not 2-byte aligned"),
    ("v_out_b_stride", -1, INVALID, "v_out has a negative stride"),
    ("k_out_b_stride", 1 << 40, UNSUPPORTED, "2^40"),
    ("v_out", BASE + 2 * MB + 128, INVALID, "k_out overlaps v_out"),
    ("k_out", BASE + 64, INVALID, "k_out overlaps cache.k"),
    ("v_out", BASE + 13 * MB, INVALID, "v_out overlaps scales.v"),
    ("cu_rows", None, INVALID, "cu_rows"),
    ("kv_len", BASE + 5 * MB + 1, INVALID, "kv_len is not 4-byte aligned"),
    ("table", None, INVALID, "table is NULL"),
    ("table_width", 0, INVALID, "table_width"),
    ("error_word", BASE + 1, INVALID, "error_word"),
    ("cache.num_heads", 0, INVALID, "num_heads"),
])
def test_read_refusals(lib, path, value, want, message):
    p = fake_read()
    put(path, value)(p)
    assert status(lib, p, fake_scales()) == want
    assert message in kda.kda_last_error()


@no_gpu
def test_what_is_allowed(lib):
    """Codes of odd addresses, rows of keys and values side by side, calls without rows; and a cache without pages needs
    no pointers. KDA_ELAUNCH: the checks passed, and there is no device."""
    p = fake_attention()
    p.cache.k.ptr = BASE + 1
    assert status(lib, p, fake_scales()) == kda.KDA_ELAUNCH
    r = fake_read()
    r.v_out, r.k_out_b_stride, r.v_out_b_stride = r.k_out + 2 * 256, 512, 512
    assert status(lib, r, fake_scales()) == kda.KDA_ELAUNCH
    r.num_tokens = 0
    assert status(lib, r, fake_scales()) == kda.KDA_OK
    p = fake_rope()
    p.num_tokens = 0
    assert status(lib, p, fake_scales()) == kda.KDA_OK
    p.cache.num_pages, p.cache.k.ptr, p.cache.v.ptr = 0, None, None
    assert status(lib, p, kda.KdaPagedScales()) == kda.KDA_OK


def test_binding_checks():
    with pytest.raises(ValueError):  # before any address is taken
        kda._scales(torch.zeros(2, 1, 1), torch.zeros(2, 1, 1), fake_attention().cache)  # not on a GPU
    with pytest.raises(TypeError):
        kda._need(torch.zeros(1, dtype=torch.int8), "k_codes", torch.uint8)


# ---------------------------------------------------------------- the oracle

def test_scale_exponent():
    assert [fp8.scale_exponent(x) for x in (0.0, 448.0, 448.0001, 449.0, 224.0, 224.1, 1.0, 3.5, 3.51)] == [
        -40, 0, 1, 1, -1, 0, -8, -7, -6]
    assert fp8.scale_exponent(448.0 * 2.0 ** -40) == -40 and fp8.scale_exponent(2.0 ** -60) == -40
    assert fp8.scale_exponent(448.0 * 2.0 ** 40) == 40 and fp8.scale_exponent(2.0 ** 60) == 40 == fp8.scale_exponent(np.inf)


def small_write(rows=24, start=5, page=32, seed=0):
    rng = np.random.default_rng(seed)
    codes = oracle.e4m3_encode(rng.normal(size=(3, page, 2, 4)) * 100)
    scales = 2.0 ** rng.integers(-8, -4, (3, page // 16, 2)).astype(float)
    x = rng.normal(size=(rows, 2, 4)) * np.exp(rng.normal(size=(rows, 1, 1)))
    slots = [page + start + i for i in range(rows)]
    return x, slots, codes, scales


def pins(write_side):
    """What the append must do, stated apart from it: raises AssertionError where it does not."""
    x, slots, codes, scales = small_write()
    got, after, exact, kind = write_side(x, slots, codes, scales)
    page, first, n = 1, 5, 24
    values = oracle.dequantized(got, after)
    for h in range(2):
        for b, (lo, hi) in enumerate(((0, 16), (16, 32))):
            new = [t for t in range(n) if lo <= first + t < hi]
            top = np.abs(x[new, h]).max()
            need = after[page, b, h]
            old = scales[page, b, h]
            fits = 2.0 ** np.ceil(np.log2(top / 448))
            assert need == (fits if b == 1 else max(fits, old))  # block 1 begins with its first token
            for t in new:  # new codes: nearest
                assert (np.abs(values[page, first + t, h] - x[t, h]) <= half_step(x[t, h] / need) * need).all()
                assert (oracle.e4m3_encode(x[t, h] / need) == got[page, first + t, h]).all()
        for j in range(first):  # earlier tokens: their numbers, to a rounding
            was = oracle.e4m3_decode(codes[page, j, h]) * scales[page, 0, h]
            s = after[page, 0, h]
            if s == scales[page, 0, h]:
                assert np.array_equal(got[page, j, h], codes[page, j, h])
            assert (np.abs(values[page, j, h] - was) <= half_step(was / s) * s).all()
    assert np.array_equal(got[page, first + n:], codes[page, first + n:])
    for p in (0, 2):
        assert np.array_equal(got[p], codes[p]) and np.array_equal(after[p], scales[p])
    # a block that begins anew forgets a scale that is larger, one with earlier tokens keeps it
    big = np.full_like(scales, 64.0)
    assert (write_side(x, slots, codes, big)[1][page, 0] == 64.0).all()
    assert (write_side(x, slots, codes, big)[1][page, 1] < 64.0).all()
    # and a small one grows, with the earlier codes rounded anew
    tiny = np.full_like(scales, 2.0 ** -30)
    got, after, _, kind = write_side(x, slots, codes, tiny)
    assert (after[page, 0] > 2.0 ** -12).all() and (got[page, :first] & 0x7F == 0).all() and (kind[page, :first] == 1).all()
    # magnitudes count, not numbers
    assert np.array_equal(write_side(-np.abs(x), slots, codes, scales)[1], write_side(np.abs(x), slots, codes, scales)[1])
    # rows that are not stored change nothing; a NaN is stored and does not count
    got, after, _, _ = write_side(x, [-1] * n, codes, scales)
    assert np.array_equal(got, codes) and np.array_equal(after, scales)
    y = x.copy()
    y[14, 0, 2] = np.nan  # in the second block
    got, after, _, _ = write_side(y, slots, codes, scales)
    y[14, 0, 2] = 0.0
    assert got[page, first + 14, 0, 2] & 0x7F == 0x7F
    assert np.array_equal(after, write_side(y, slots, codes, scales)[1])


def test_write_side():
    pins(fp8.write_side)


MISTAKES = [
    ("new = max(old, need) if first > start else need", "new = max(old, need)"),
    ("new = max(old, need) if first > start else need", "new = need"),
    ("if first > start and need > old:", "if False:"),
    ("e4m3_encode(held / new)", "e4m3_encode(held / old)"),
    ("e4m3_encode(x[t, h] / new)", "e4m3_encode(x[t, h] * new)"),
    ("top = top[~np.isnan(top)].max(initial=0.0)", "top = np.nan_to_num(top, nan=1e9).max(initial=0.0)"),
    ("np.abs(x[rows, h])", "x[rows, h]"),
    ("codes[p, start:first, h]) * old", "codes[p, start:first, h]) * need"),
    ("slot % page // SCALE_TOKENS", "slot % page // 8"),
    ("start = b * SCALE_TOKENS", "start = 0"),
]


@pytest.mark.parametrize("mistake", range(len(MISTAKES)))
def test_planted_mistakes_fail_a_pin(mistake):
    source = open(fp8.__file__).read()
    was, now = MISTAKES[mistake]
    assert source.count(was) >= 1
    space = {"__name__": "oracle.planted", "__package__": "oracle"}
    exec(compile(source.replace(was, now), "planted", "exec"), space)
    with pytest.raises((AssertionError, IndexError, ValueError)):
        pins(space["write_side"])


def test_paged_read_against_brute_force():
    a = Attention([3, 0, 40, 2], [3, 0, 33, 20], 2, 2, 5, 16, seed=1)
    a.kv[3] = -1
    a.table[2, 1] = 99
    T = 47
    k, v, bits = oracle.paged_read_fp8(a.k.numpy(), a.v.numpy(), a.ks.double().numpy(), a.vs.double().numpy(), a.table, a.cu, a.kv, T)
    assert bits == kda.KDA_ERR_LENGTHS | kda.KDA_ERR_PAGES
    for out, codes, scales in ((k, a.k, a.ks), (v, a.v, a.vs)):
        assert np.isnan(out[45:]).all() and (out[43:45] == 0).all()
        for t in range(43):
            r = 0 if t < 3 else 2
            token = t if r == 0 else t - 3 + 33 - 40
            for h in range(2):
                for c in range(5):
                    want = 0.0
                    if token >= 0 and not (r == 2 and token // 16 == 1):
                        page = int(a.table[r, token // 16])
                        want = float(oracle.e4m3_decode(codes[page, token % 16, h, c].numpy())) * float(scales[page, 0, h])
                    assert out[t, h, c] == want


def test_split_queries():
    """The two E4M3 numbers that stand for a bf16 one: exact from 2^-9 of the head's largest on, off by less than 2^-17 of
    that below."""
    gen = torch.Generator().manual_seed(2)
    x = (torch.randn((400, 64), generator=gen) * torch.exp(2 * torch.randn((400, 64), generator=gen))).to(torch.bfloat16).double().numpy()
    top = np.abs(x).max(axis=1, keepdims=True)
    scale = 2.0 ** np.ceil(np.log2(top / 448.0))
    y = x / scale
    hi = oracle.e4m3_decode(oracle.e4m3_encode(y))
    off = np.abs(y - hi - oracle.e4m3_decode(oracle.e4m3_encode(y - hi))) * scale
    assert (off[np.abs(x) >= 2.0 ** -9 * top] == 0).all()
    assert (off < 2.0 ** -17 * top).all() and off.max() > 0


def test_three_codes_of_a_weight():
    """A weight p <= 2^8 of fp16 as p1 + 2^-5 p2 + 2^-10 p3: off by 2^-20 or 2^-12 of itself at most, whichever is more."""
    p = np.concatenate([np.exp2(np.random.default_rng(3).uniform(-24, 8, 20000)), [2.0 ** 8, 0.0, 2.0 ** -20, 255.9, 2.0 ** 7]])
    p = p.astype(np.float16).astype(np.float64)
    p = np.minimum(p, 256.0)
    rest, total = p, np.zeros_like(p)
    for k in range(3):
        c = oracle.e4m3_decode(oracle.e4m3_encode(rest))
        assert (rest <= 448).all()
        total = total + c * 2.0 ** (-5 * k)
        rest = (rest - c) * 32
    assert (np.abs(total - p) <= np.maximum(2.0 ** -20, 2.0 ** -12 * p)).all()
