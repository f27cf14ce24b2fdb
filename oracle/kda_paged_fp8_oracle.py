"""fp64 oracle of the paged cache held in 8 bits (include/kda_paged_fp8.h): the
append, reading back, and what the attention attends over. Plain numpy, no code
shared with the CUDA path; codes are decoded and encoded by the fp8 state pool's
oracle (pinned in tests/oracle_pins_fp8.py)."""

import numpy as np

from .kda_fp8_oracle import e4m3_decode, e4m3_encode
from .kda_paged_oracle import ERR_LENGTHS, ERR_PAGES, ERR_SEQLENS, rope_rotate

SCALE_TOKENS = 16
LOW, HIGH = -40, 40


def scale_exponent(top):
    """The smallest integer e in [LOW, HIGH] with top * 2^-e <= 448, HIGH if there is none."""
    for e in range(LOW, HIGH):
        if top <= 448.0 * 2.0 ** e:
            return e
    return HIGH


def dequantized(codes, scales):
    """Values [pages, page, heads, dim] of codes and scales [pages, blocks, heads]."""
    page = codes.shape[1]
    return e4m3_decode(codes) * np.asarray(scales, dtype=np.float64)[:, np.arange(page) // SCALE_TOKENS][..., None]


def write_side(x, slots, codes, scales):
    """One side's append of rows x [T, heads, dim] at slots (-1: not stored), row by row of each block.

    Returns (codes, scales, exact, kind): exact holds the number that each touched code rounds, before it is divided by
    its scale; kind 0 where nothing changed, 1 for codes rounded anew, 2 for new ones."""
    codes, scales = np.array(codes), np.array(scales, dtype=np.float64)
    page = codes.shape[1]
    exact, kind = np.zeros(codes.shape), np.zeros(codes.shape[:3], dtype=np.int64)
    runs = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            runs.setdefault((slot // page, slot % page // SCALE_TOKENS), []).append(t)
    for (p, b), rows in runs.items():
        first = slots[rows[0]] % page
        start = b * SCALE_TOKENS
        for h in range(codes.shape[2]):
            top = np.abs(x[rows, h])
            top = top[~np.isnan(top)].max(initial=0.0)
            need = 2.0 ** scale_exponent(top)
            old = scales[p, b, h]
            new = max(old, need) if first > start else need
            if first > start and need > old:
                held = e4m3_decode(codes[p, start:first, h]) * old
                exact[p, start:first, h] = held
                kind[p, start:first, h] = 1
                codes[p, start:first, h] = e4m3_encode(held / new)
            for t in rows:
                place = slots[t] % page
                exact[p, place, h] = x[t, h]
                kind[p, place, h] = 2
                codes[p, place, h] = e4m3_encode(x[t, h] / new)
            scales[p, b, h] = new
    return codes, scales, exact, kind


def rope_append_fp8(q, k, v, positions, slots, freqs, k_codes, v_codes, k_scales, v_scales, interleaved, mscale):
    """(q_out, keys, values, rows written, error bits), keys and values as write_side returns them."""
    limit = k_codes.shape[0] * k_codes.shape[1]
    qo = rope_rotate(q, positions, freqs, interleaved, mscale)
    ko = rope_rotate(k, positions, freqs, interleaved, mscale)
    err, at = 0, []
    for pos, slot in zip(positions, slots):
        stored = pos >= 0 and 0 <= slot < limit
        if pos >= 0 and not stored and slot != -1:
            err |= ERR_PAGES
        at.append(int(slot) if stored else -1)
    return (qo, write_side(ko, at, k_codes, k_scales), write_side(np.asarray(v, dtype=np.float64), at, v_codes, v_scales),
            np.asarray(positions) >= 0, err)


def paged_read_fp8(k_codes, v_codes, k_scales, v_scales, table, cu_rows, kv_len, num_tokens):
    """(k, v, error bits); rows that no request covers are NaN."""
    num_pages, page, heads, dim = k_codes.shape
    width = table.shape[1]
    sides = dequantized(k_codes, k_scales), dequantized(v_codes, v_scales)
    out = [np.full((num_tokens, heads, dim), np.nan) for _ in sides]
    err = 0
    for r in range(len(kv_len)):
        a, b, L = int(cu_rows[r]), int(cu_rows[r + 1]), int(kv_len[r])
        if L < 0 or L > width * page:
            err |= ERR_LENGTHS
            L = 0
        if a < 0 or b < a or b > num_tokens:
            err |= ERR_SEQLENS
            continue
        for t in range(a, b):
            token = L - (b - a) + (t - a)
            p = int(table[r, token // page]) if token >= 0 else -1
            if token >= 0 and not 0 <= p < num_pages:
                err |= ERR_PAGES
            for o, x in zip(out, sides):
                o[t] = x[p, token % page] if token >= 0 and 0 <= p < num_pages else 0.0
    return out[0], out[1], err
