"""fp64 oracle of the paged-attention operators (include/kda_paged.h): the page
plan in plain integers, rotary positions with the append, and attention of each
request's new tokens over the paged cache. Plain numpy, no rounding to bf16
(the comparisons bound it), no code shared with the CUDA path."""

import numpy as np

ERR_SEQLENS, ERR_PAGES, ERR_LENGTHS = 8, 16, 32


def ceil_div(a, b):
    return -((-a) // b)


def paged_plan(cached, new_len, table, free_pages, free_count, page_size, num_pages, num_tokens):
    """(table, cu_new, kv_len, positions, slots, free_count, error bits), in the order of the requests."""
    table = np.array(table)
    R = len(cached)
    free_count = min(max(int(free_count), 0), len(free_pages))
    cu, kv = [0], []
    positions, slots = [-1] * num_tokens, [-1] * num_tokens
    asked = taken = err = 0
    for r in range(R):
        c, n = int(cached[r]), int(new_len[r])
        rows = max(n, 0)
        start = cu[-1]
        cu.append(start + rows)
        if c < 0 or n < 0 or c + n > table.shape[1] * page_size or start + rows > num_tokens:
            err |= ERR_LENGTHS
            kv.append(0)
            continue
        have = ceil_div(c, page_size)
        need = ceil_div(c + n, page_size) - have
        asked += need
        if need > 0 and asked > free_count:
            err |= ERR_PAGES
            kv.append(0)
            continue
        for i in range(need):
            table[r, have + i] = free_pages[free_count - 1 - taken]
            taken += 1
        kv.append(c + n)
        for j in range(n):
            positions[start + j] = c + j
            page = int(table[r, (c + j) // page_size])
            if 0 <= page < num_pages:
                slots[start + j] = page * page_size + (c + j) % page_size
            else:
                err |= ERR_PAGES
    return (table, np.minimum(cu, 2 ** 31 - 1), np.array(kv, dtype=np.int64), np.array(positions, dtype=np.int64),
            np.array(slots, dtype=np.int64), free_count - taken, err)


def rope_rotate(x, positions, freqs, interleaved, mscale):
    """x [T, H, D] turned by the exact phases positions * freqs (freqs: integers in units of 2^-64 turns)."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        for i, f in enumerate(freqs):
            turn = ((int(pos) * int(f)) % (1 << 64)) / 2.0 ** 64
            c, s = mscale * np.cos(2 * np.pi * turn), mscale * np.sin(2 * np.pi * turn)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            u, w = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            y[t, :, a], y[t, :, b] = u * c - w * s, w * c + u * s
    return y


def rope_append(q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved, mscale):
    """(q_out, k_cache, v_cache, rows written, error bits); caches [pages, page_size, heads, dim]."""
    num_pages, page = k_cache.shape[:2]
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    qo = rope_rotate(q, positions, freqs, interleaved, mscale)
    ko = rope_rotate(k, positions, freqs, interleaved, mscale)
    err = 0
    for t, (pos, slot) in enumerate(zip(positions, slots)):
        if pos < 0 or slot == -1:
            continue
        if slot < 0 or slot >= num_pages * page:
            err |= ERR_PAGES
            continue
        kc[slot // page, slot % page] = ko[t]
        vc[slot // page, slot % page] = v[t]
    return qo, kc, vc, np.asarray(positions) >= 0, err


def rope_frequencies(rotary_dim, base, scaling, factor, original_len, low, high):
    """Radians per position of each pair (include/kda_paged.h, KDA_ROPE_*)."""
    if scaling == 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-np.arange(0, rotary_dim, 2, dtype=np.float64) / rotary_dim)
    if scaling == 1:
        f = f / factor
    if scaling == 3:
        w = np.clip((f * original_len / (2 * np.pi) - low) / (high - low), 0, 1)
        f = w * f + (1 - w) * f / factor
    return f


def paged_attention(q, k_cache, v_cache, table, cu_new, kv_len, scale, window):
    """Per row and head: out, lse, and for the bounds the weighted |v| (A), the
    largest scale * sum |q||k| over the keys seen (S) and the number of keys (n).
    Rows no request covers are NaN in lse and out. Also the error bits."""
    T, Hq, D = q.shape
    num_pages, page, Hkv = k_cache.shape[:3]
    g = Hq // Hkv
    width = table.shape[1]
    out = np.full((T, Hq, D), np.nan)
    A = np.zeros((T, Hq, D))
    lse, S = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    count = np.zeros(T, dtype=np.int64)
    err = 0
    for r in range(len(kv_len)):
        a, b, L = int(cu_new[r]), int(cu_new[r + 1]), int(kv_len[r])
        if L < 0 or L > width * page:
            err |= ERR_LENGTHS
            L = 0
        if a < 0 or b < a or b > T:
            err |= ERR_SEQLENS
            continue
        for t in range(a, b):
            p = L - (b - a) + (t - a)
            lo, hi = (max(0, p - window + 1) if window > 0 else 0), p + 1
            if hi <= lo:
                out[t], lse[t] = 0.0, -np.inf
                continue
            count[t] = hi - lo
            at = np.arange(lo, hi)
            pages = table[r, at // page]
            ok = (pages >= 0) & (pages < num_pages)
            if not ok.all():
                err |= ERR_PAGES
            pages = np.where(ok, pages, 0)
            k = np.where(ok[:, None, None], k_cache[pages, at % page], 0.0)
            v = np.where(ok[:, None, None], v_cache[pages, at % page], 0.0)
            for h in range(Hq):
                kh, vh = k[:, h // g], v[:, h // g]
                s = scale * (kh @ q[t, h])
                S[t, h] = scale * np.max(np.abs(kh) @ np.abs(q[t, h]))
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                out[t, h] = (w @ vh) / total
                A[t, h] = (w @ np.abs(vh)) / total
                lse[t, h] = m + np.log(total)
    return out, lse, A, S, count, err
