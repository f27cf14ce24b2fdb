"""Cases, plain forms and exact values of the paged-attention operators.

Three operators of a hybrid decoder's attention layers, which stand beside the KDA layers:

  plan       block tables and slot maps built from the request lengths (kda_paged_plan)
  rope       rotary positions on q and k, k and v appended to the paged cache (kda_rope_append)
  attention  a chunk of new tokens per request over the paged cache (kda_paged_attention)
"""

import math
import random

import torch

own = False

DEV = "cuda"
TWO_PI = 2.0 * math.pi


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a full batch: every request brings one token
        {"name": "plan-decode-256", "op": "plan", "R": 256, "new": 1, "ragged_new": False, "ctx": 8192, "page": 64,
         "spread": 1},
        # the smallest step: a single stream
        {"name": "plan-decode-1", "op": "plan", "R": 1, "new": 1, "ragged_new": False, "ctx": 2000, "page": 16,
         "spread": 2},
        # chunked prefill of many requests, ragged chunks, small pages
        {"name": "plan-chunks-48", "op": "plan", "R": 48, "new": 700, "ragged_new": True, "ctx": 12000, "page": 16,
         "spread": 3},
        # one decode step, whole heads rotated in halves
        {"name": "rope-decode-256", "op": "rope", "T": 256, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "base": 10000.0, "factor": 1.0, "maxpos": 8192, "page": 64, "fused": True,
         "heads_first": False},
        # a long prefill chunk, half of each head rotated in pairs, frequencies scaled for 128k positions
        {"name": "rope-chunk-8192", "op": "rope", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "rot": 64,
         "interleaved": True, "base": 500000.0, "factor": 8.0, "maxpos": 131072, "page": 64, "fused": False,
         "heads_first": False},
        # an odd chunk of small heads without sharing (12 heads as the KDA layers have), cache with heads before tokens
        {"name": "rope-odd-1037", "op": "rope", "T": 1037, "Hq": 12, "Hkv": 12, "D": 64, "rot": 64,
         "interleaved": False, "base": 10000.0, "factor": 4.0, "maxpos": 32768, "page": 16, "fused": True,
         "heads_first": True},
        # a single stream's decode step: latency
        {"name": "attn-decode-1", "op": "attention", "R": 1, "new": 1, "ragged_new": False, "ctx": 1000, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 4},
        # a served batch's decode step
        {"name": "attn-decode-64", "op": "attention", "R": 64, "new": 1, "ragged_new": False, "ctx": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 5},
        # speculative verify: eight draft tokens a request, 12 heads in groups of three
        {"name": "attn-verify-32", "op": "attention", "R": 32, "new": 8, "ragged_new": False, "ctx": 6000, "Hq": 12,
         "Hkv": 4, "D": 128, "page": 32, "window": 0, "heads_first": True, "spread": 6},
        # the first chunk of a prompt
        {"name": "attn-prefill-4096", "op": "attention", "R": 1, "new": 4096, "ragged_new": False, "ctx": 0,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 7},
        # later chunks of long prompts over what is cached
        {"name": "attn-chunk-2x2048", "op": "attention", "R": 2, "new": 2048, "ragged_new": False, "ctx": 16384,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "window": 0, "heads_first": False, "spread": 8},
        # ragged chunks and decode tokens in one step, a sliding window, small heads and pages
        {"name": "attn-mixed-window", "op": "attention", "R": 24, "new": 300, "ragged_new": True, "ctx": 5000,
         "Hq": 16, "Hkv": 4, "D": 64, "page": 16, "window": 1024, "heads_first": False, "spread": 9},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "attention", "attention"])
    if op == "plan":
        R = _log(rng, 1, 512)
        decode = rng.random() < 0.5
        return {"op": "plan", "R": R, "new": 1 if decode else _log(rng, 2, max(2, 30000 // R)),
                "ragged_new": not decode, "ctx": _log(rng, 16, 12000), "page": rng.choice([16, 32, 64, 128]),
                "spread": rng.randrange(1 << 20)}
    if op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 12])
        Hq = Hkv * (1 if Hkv == 12 else rng.choice([1, 2, 3, 4]))
        rot = rng.choice([D, D // 2, D // 4])
        return {"op": "rope", "T": _log(rng, 1, 8192), "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
                "interleaved": rng.random() < 0.5, "base": rng.choice([10000.0, 500000.0]),
                "factor": rng.choice([1.0, 4.0, 8.0]), "maxpos": rng.choice([8192, 32768, 131072]),
                "page": rng.choice([16, 32, 64, 128]), "fused": rng.random() < 0.5,
                "heads_first": rng.random() < 0.5}
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    while Hkv * g > 32:
        g = g // 2
    kind = rng.choice(["decode", "decode", "verify", "chunk", "chunk"])
    if kind == "decode":
        R, new, ctx = _log(rng, 1, 96), 1, _log(rng, 32, 8192)
    elif kind == "verify":
        R, new, ctx = _log(rng, 1, 48), rng.choice([2, 4, 8]), _log(rng, 32, 6000)
    else:
        R = _log(rng, 1, 12)
        new = _log(rng, 16, 2048)
        # scores of the padded plain form, and the flops, within those of the largest listed case
        ctx = _log(rng, 16, max(17, min(12000, (1 << 31) // (R * Hkv * g * new * 2) - new)))
    return {"op": "attention", "R": R, "new": new, "ragged_new": kind == "chunk" and rng.random() < 0.6, "ctx": ctx,
            "Hq": Hkv * g, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128]),
            "window": rng.choice([0, 0, 0, 512, 1024]), "heads_first": rng.random() < 0.5,
            "spread": rng.randrange(1 << 20)}


def _lengths(case):
    """New and cached tokens of each request: the case's largest, and others down to a quarter of it (ragged
    chunks: down to a single token, as decode requests in a prefill step are)."""
    r = random.Random(case["spread"])
    new, cached = [], []
    for i in range(case["R"]):
        n, c = case["new"], case["ctx"]
        if i > 0:
            c = r.randint(c // 4, c)
            if case["ragged_new"]:
                n = 1 if r.random() < 0.3 else r.randint(1, n)
        new.append(n)
        cached.append(c)
    return new, cached


# ---------------------------------------------------------------- inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _cache(pages, page, heads, dim, heads_first, gen):
    """A cache [pages, page, heads, dim]; heads_first: stored with the heads before a page's tokens."""
    if heads_first:
        return _randn((pages, heads, page, dim), gen).transpose(1, 2)
    return _randn((pages, page, heads, dim), gen)


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits: base^(-2i/rot), and for factor > 1 interpolated by
    parts: a pair that turns less than once in the original context is slowed by the factor, one that turns over
    four times keeps its frequency, linearly in between."""
    rot, factor = case["rot"], case["factor"]
    f = case["base"] ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor > 1.0:
        keep = ((f * (case["maxpos"] / factor) / TWO_PI - 1.0) / 3.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def _mscale(case):
    return 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"plan": _prepare_plan, "rope": _prepare_rope, "attention": _prepare_attention}[case["op"]](case, gen)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(new, cached, page, gen, total_pages):
    """A table whose cached pages are taken from a shuffled pool, and the rest of the pool as the free list."""
    R = len(new)
    have = [-(-c // page) for c in cached]
    width = max(-(-(c + n) // page) for n, c in zip(new, cached))
    pool = torch.randperm(total_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, device=DEV)
    h = _int(have)
    taken = torch.arange(width, device=DEV)[None, :] < h[:, None]
    table[taken] = pool[:sum(have)]
    return table, pool[sum(have):].contiguous()


def _prepare_plan(case, gen):
    new, cached = _lengths(case)
    page = case["page"]
    total = sum(-(-(c + n) // page) for n, c in zip(new, cached)) + 64
    table, free = _tables(new, cached, page, gen, total)
    T = sum(new)
    s = {"case": case, "page": page, "T": T, "new": _int(new), "cached": _int(cached), "table": table,
         "free": free, "free_count": _int([free.numel()]), "pages": total}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        s["call"] = kda.prepare_paged_plan(s["cached"], s["new"], table, free, s["free_count"], page_size=page,
                                           num_pages=total, num_tokens=T)
    return s


def _prepare_rope(case, gen):
    T, Hq, Hkv, D, page = case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["fused"]:  # views into the rows of one projection
        row = _randn((T, (Hq + 2 * Hkv) * D), gen)
        q = row[:, :Hq * D].view(T, Hq, D)
        k = row[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = row[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    else:
        q, k, v = _randn((T, Hq, D), gen), _randn((T, Hkv, D), gen), _randn((T, Hkv, D), gen)
    pages = -(-T // page) + 8
    kc = _cache(pages, page, Hkv, D, case["heads_first"], gen)
    vc = _cache(pages, page, Hkv, D, case["heads_first"], gen)
    # decode tokens stand anywhere, a chunk's tokens follow one another; pages lie scattered
    if T <= 512:
        pos = torch.randint(0, case["maxpos"], (T,), generator=gen, device=DEV)
    else:
        start = torch.randint(0, case["maxpos"] - T + 1, (1,), generator=gen, device=DEV)
        pos = start + torch.arange(T, device=DEV)
    order = torch.randperm(pages, generator=gen, device=DEV)
    t = torch.arange(T, device=DEV)
    slots = order[t // page] * page + t % page
    # 64-bit fixed-point turns a position: what both forms rotate by
    turns = [int(round(f / TWO_PI * 2.0 ** 64)) for f in _frequencies(case).tolist()]
    freqs = torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in turns], dtype=torch.int64, device=DEV)
    s = {"case": case, "q": q, "k": k, "v": v, "kc": kc, "vc": vc, "pos": pos.to(torch.int32),
         "slots": slots.to(torch.int32), "freqs": freqs, "mscale": _mscale(case)}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        s["call"] = kda.prepare_rope_append(q, k, v, s["pos"], s["slots"], freqs, kc, vc,
                                            interleaved=case["interleaved"], mscale=s["mscale"])
    return s


def _prepare_attention(case, gen):
    new, cached = _lengths(case)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    kv = [n + c for n, c in zip(new, cached)]
    total = sum(-(-x // page) for x in kv) + 8
    table, _ = _tables([0] * len(kv), kv, page, gen, total)
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": case, "q": _randn((T, Hq, D), gen), "kc": _cache(total, page, Hkv, D, case["heads_first"], gen),
         "vc": _cache(total, page, Hkv, D, case["heads_first"], gen), "table": table, "cu": _int(cu),
         "kv": _int(kv), "new_max": max(new), "kv_max": max(kv), "scale": D ** -0.5, "window": case["window"]}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=DEV)
        work = kda.paged_attention_workspace(D, torch.device(DEV))
        s["call"] = kda.prepare_paged_attention(s["q"], s["kc"], s["vc"], table, s["cu"], s["kv"], out=out, lse=lse,
                                                scale=s["scale"], window=s["window"], workspace=work)
        s["out"], s["lse"] = out, lse
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        got = state["call"]()
        if op == "plan":
            return [state["table"], got.cu_new, got.kv_len, got.positions, got.slots, got.free_count]
        if op == "rope":
            return [got, state["kc"], state["vc"]]
        return [state["out"], state["lse"]]
    return {"plan": _plain_plan, "rope": _plain_rope, "attention": _plain_attention}[op](state)


def _plain_plan(s):
    page, table = s["page"], s["table"]
    new, cached = s["new"].long(), s["cached"].long()
    have = (cached + page - 1) // page
    need = (cached + new + page - 1) // page - have
    before = need.cumsum(0) - need
    column = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = (column >= have[:, None]) & (column < (have + need)[:, None])
    taken = s["free_count"].long() - 1 - (before[:, None] + column - have[:, None])
    table.copy_(torch.where(fresh, s["free"][taken.clamp(0, s["free"].numel() - 1)], table))
    ends = new.cumsum(0)
    t = torch.arange(s["T"], device=DEV)
    r = (t[:, None] >= ends[None, :]).sum(1)
    pos = cached[r] + t - (ends - new)[r]
    slots = table[r, pos // page].long() * page + pos % page
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends])
    return [table, cu.int(), (cached + new).int(), pos.int(), slots.int(), (s["free_count"] - need.sum()).int()]


def _turn(x, cos, sin, rot, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = y[..., :h], y[..., h:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], dim=-1)
    return y.to(torch.bfloat16)


def _plain_rope(s):
    case = s["case"]
    page = case["page"]
    # the phase in 2^-64 turns, wrapping as whole turns drop out; its upper bits as an angle in (-pi, pi)
    phase = s["pos"].long()[:, None] * s["freqs"][None, :]
    angle = (phase >> 32).float() * (TWO_PI / 2.0 ** 32)
    cos = (angle.cos() * s["mscale"])[:, None, :]
    sin = (angle.sin() * s["mscale"])[:, None, :]
    q = _turn(s["q"], cos, sin, case["rot"], case["interleaved"])
    k = _turn(s["k"], cos, sin, case["rot"], case["interleaved"])
    at = s["slots"].long()
    s["kc"][at // page, at % page] = k
    s["vc"][at // page, at % page] = s["v"]
    return [q, s["kc"], s["vc"]]


def _plain_attention(s):
    case = s["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    g, N, L = Hq // Hkv, s["new_max"], s["kv_max"]
    cu, kv = s["cu"].long(), s["kv"].long()
    n = cu[1:] - cu[:-1]
    R = n.numel()
    i = torch.arange(N, device=DEV)
    j = torch.arange(L, device=DEV)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(R, N, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, g * N, D)
    pages = s["table"][:, j // page].clamp(min=0).long()
    k = s["kc"][pages, j % page].float()
    v = s["vc"][pages, j % page].float()
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).view(R, Hkv, g, N, L).mul_(s["scale"])
    p = (kv - n)[:, None] + i[None, :]
    seen = j[None, None, :] <= p[:, :, None]
    if s["window"] > 0:
        seen &= j[None, None, :] > p[:, :, None] - s["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights.view(R, Hkv, g * N, L), v.permute(0, 2, 1, 3)).view(R, Hkv, g, N, D) / total
    lse = (top + total.log()).squeeze(-1)
    there = i[None, :] < n[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(R, N, Hq, D)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(R, N, Hq)[there]
    return [out.to(torch.bfloat16), lse]


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_attention(s)


def _exact_rope(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    z = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device=DEV),
                    s["pos"].double()[:, None] * _frequencies(case).to(DEV)[None, :])[:, None, :]

    def rotated(x):
        y = x.double().clone()
        part = y[..., :rot]
        pair = part.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, rot // 2)).mT
        w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        y[..., :rot] = (w if case["interleaved"] else w.mT).flatten(-2)
        return y

    kc, vc = s["kc"].double(), s["vc"].double()
    at = s["slots"].long()
    kc[at // page, at % page] = rotated(s["k"])
    vc[at // page, at % page] = s["v"].double()
    return [rotated(s["q"]), kc, vc]


def _exact_attention(s):
    case = s["case"]
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    g, window = Hq // Hkv, case["window"]
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    out, lse = [], []
    for r in range(len(kv)):
        n, L = cu[r + 1] - cu[r], kv[r]
        at = s["table"][r, :-(-L // page)].long()
        k = s["kc"][at].reshape(-1, Hkv, D)[:L].double()
        v = s["vc"][at].reshape(-1, Hkv, D)[:L].double()
        key = torch.arange(L, device=DEV)
        o = torch.empty((n, Hq, D), dtype=torch.float64, device=DEV)
        z = torch.empty((n, Hq), dtype=torch.float64, device=DEV)
        for a in range(0, n, 512):
            b = min(n, a + 512)
            own_pos = (L - n) + torch.arange(a, b, device=DEV)
            hidden = key[None, :] > own_pos[:, None]
            if window > 0:
                hidden = hidden | (key[None, :] <= own_pos[:, None] - window)
            x = torch.einsum("nhgd,lhd->hgnl", s["q"][cu[r] + a:cu[r] + b].double().view(-1, Hkv, g, D), k)
            x = torch.where(hidden, torch.full((), -math.inf, dtype=torch.float64, device=DEV), x * s["scale"])
            z[a:b] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(b - a, Hq)
            o[a:b] = torch.einsum("hgnl,lhd->nhgd", torch.softmax(x, -1), v).reshape(b - a, Hq, D)
        out.append(o)
        lse.append(z)
    return [torch.cat(out), torch.cat(lse)]


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "plan":
        new, cached = _lengths(case)
        page = case["page"]
        need = sum(-(-(n + c) // page) - -(-c // page) for n, c in zip(new, cached))
        partial = sum(c % page > 0 for c in cached)
        # lengths, open pages and free pages read; table entries, offsets, lengths, positions and slots written
        return {"bytes": 4 * (2 * case["R"] + partial + need + 1) + 4 * (need + 2 * case["R"] + 2 + 2 * sum(new)),
                "flops": 0}
    if case["op"] == "rope":
        T, heads = case["T"], case["Hq"] + 2 * case["Hkv"]
        return {"bytes": 4 * T * heads * case["D"] + 8 * T + 4 * case["rot"],
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    new, cached = _lengths(case)
    Hq, Hkv, D, window = case["Hq"], case["Hkv"], case["D"], case["window"]
    pairs, keys = 0, 0
    for n, c in zip(new, cached):
        if window > 0:
            pairs += sum(min(c + i + 1, window) for i in range(n))
            keys += min(n + c, window + n - 1)
        else:
            pairs += n * c + n * (n + 1) // 2
            keys += n + c
    T = sum(new)
    return {"bytes": 4 * keys * Hkv * D + 4 * T * Hq * D + 4 * T * Hq, "flops": 4 * pairs * Hq * D}
