"""Cases, plain forms and exact values of the operators of a paged cache held in 8 bits.

The attention layers of a hybrid decoder keep keys and values as E4M3 codes with a power-of-two scale for each block of
16 tokens and head; a value is its code times its block's scale:

  append     rotary positions on q and k, k and v quantised as they are written to the cache (kda_rope_append_fp8)
  read       the cached tokens of requests as packed bf16 rows (kda_paged_read_fp8)
  attention  a chunk of new tokens per request over the cache (kda_paged_attention_fp8)
"""

import math
import random

import torch

own = False

DEV = "cuda"
TWO_PI = 2.0 * math.pi
BLOCK = 16            # tokens a scale
LOW, HIGH = -40, 40   # exponents of the scales


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a full batch, whole heads rotated in halves, blocks filled to anywhere
        {"name": "append-decode-256", "op": "append", "T": 256, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128,
         "interleaved": False, "base": 10000.0, "maxpos": 8192, "page": 64, "fused": True, "heads_first": False},
        # a long prefill chunk, half of each head rotated in pairs
        {"name": "append-chunk-8192", "op": "append", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "rot": 64,
         "interleaved": True, "base": 500000.0, "maxpos": 131072, "page": 64, "fused": False, "heads_first": False},
        # an odd chunk of small heads without sharing (12 heads as the KDA layers have), that begins inside a block
        {"name": "append-odd-1037", "op": "append", "T": 1037, "Hq": 12, "Hkv": 12, "D": 64, "rot": 64,
         "interleaved": False, "base": 10000.0, "maxpos": 32768, "page": 16, "fused": True, "heads_first": True},
        # one short request read back
        {"name": "read-1", "op": "read", "R": 1, "ctx": 500, "Hkv": 4, "D": 64, "page": 32, "heads_first": True,
         "spread": 1},
        # a batch's caches read back, to move them to a machine that keeps them in 16 bits
        {"name": "read-32", "op": "read", "R": 32, "ctx": 6000, "Hkv": 8, "D": 128, "page": 64, "heads_first": False,
         "spread": 2},
        # a single stream's decode step: latency
        {"name": "attn8-decode-1", "op": "attention", "R": 1, "new": 1, "ragged_new": False, "ctx": 1000, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 4},
        # a served batch's decode step
        {"name": "attn8-decode-64", "op": "attention", "R": 64, "new": 1, "ragged_new": False, "ctx": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 5},
        # a few long contexts: what a cache of half the bytes is for
        {"name": "attn8-decode-long", "op": "attention", "R": 4, "new": 1, "ragged_new": False, "ctx": 65536, "Hq": 32,
         "Hkv": 4, "D": 128, "page": 128, "window": 0, "heads_first": True, "spread": 6},
        # speculative verify: eight draft tokens a request, 12 heads in groups of three
        {"name": "attn8-verify-32", "op": "attention", "R": 32, "new": 8, "ragged_new": False, "ctx": 6000, "Hq": 12,
         "Hkv": 4, "D": 128, "page": 32, "window": 0, "heads_first": True, "spread": 7},
        # the first chunk of a prompt
        {"name": "attn8-prefill-4096", "op": "attention", "R": 1, "new": 4096, "ragged_new": False, "ctx": 0,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "window": 0, "heads_first": False, "spread": 8},
        # later chunks of long prompts over what is cached
        {"name": "attn8-chunk-2x2048", "op": "attention", "R": 2, "new": 2048, "ragged_new": False, "ctx": 16384,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "window": 0, "heads_first": False, "spread": 9},
        # ragged chunks and decode tokens in one step, a sliding window, small heads and pages
        {"name": "attn8-mixed-window", "op": "attention", "R": 24, "new": 300, "ragged_new": True, "ctx": 5000,
         "Hq": 16, "Hkv": 4, "D": 64, "page": 16, "window": 1024, "heads_first": False, "spread": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 12])
        return {"op": "append", "T": _log(rng, 1, 8192), "Hq": Hkv * (1 if Hkv == 12 else rng.choice([1, 2, 3, 4])),
                "Hkv": Hkv, "D": D, "rot": rng.choice([D, D // 2, D // 4]), "interleaved": rng.random() < 0.5,
                "base": rng.choice([10000.0, 500000.0]), "maxpos": rng.choice([8192, 32768, 131072]), "page": page,
                "fused": rng.random() < 0.5, "heads_first": rng.random() < 0.5}
    if op == "read":
        R = _log(rng, 1, 64)
        return {"op": "read", "R": R, "ctx": _log(rng, 16, min(12000, 190000 // R)), "Hkv": rng.choice([1, 2, 4, 8]),
                "D": rng.choice([64, 128]), "page": page, "heads_first": rng.random() < 0.5,
                "spread": rng.randrange(1 << 20)}
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 6, 8])
    while Hkv * g > 32:
        g = g // 2
    kind = rng.choice(["decode", "decode", "verify", "chunk", "chunk"])
    if kind == "decode":
        R = _log(rng, 1, 96)
        new, ctx = 1, _log(rng, 32, min(65536, 600000 // R))
    elif kind == "verify":
        R, new, ctx = _log(rng, 1, 48), rng.choice([2, 4, 8]), _log(rng, 32, 6000)
    else:
        R = _log(rng, 1, 12)
        new = _log(rng, 16, 2048)
        # scores of the padded plain form, and the flops, within those of the largest listed case
        ctx = _log(rng, 16, max(17, min(12000, (1 << 31) // (R * Hkv * g * new * 2) - new)))
    return {"op": "attention", "R": R, "new": new, "ragged_new": kind == "chunk" and rng.random() < 0.6, "ctx": ctx,
            "Hq": Hkv * g, "Hkv": Hkv, "D": D, "page": page, "window": rng.choice([0, 0, 0, 512, 1024]),
            "heads_first": rng.random() < 0.5, "spread": rng.randrange(1 << 20)}


def _lengths(case):
    """New and cached tokens of each request: the case's largest, and others down to a quarter of it (ragged
    chunks: down to a single token, as decode requests in a prefill step are)."""
    r = random.Random(case["spread"])
    new, cached = [], []
    for i in range(case["R"]):
        n, c = case.get("new", 0), case["ctx"]
        if i > 0:
            c = r.randint(c // 4, c)
            if case.get("ragged_new"):
                n = 1 if r.random() < 0.3 else r.randint(1, n)
        new.append(n)
        cached.append(c)
    return new, cached


# ---------------------------------------------------------------- inputs

def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _needed(top):
    """Exponent of the smallest power of two by which `top` comes down to 448, the largest code, within the range."""
    part, exponent = torch.frexp(top)  # part in [1/2, 1), 448 = 7/8 2^9
    exponent = torch.where(part <= 0.875, exponent - 9, exponent - 8)
    return torch.where(top > 0, exponent, LOW).clamp(LOW, HIGH)


def _cache(pages, page, heads, dim, heads_first, gen):
    """Codes [pages, page, heads, dim] (uint8) and scales [pages, blocks, heads] of one side of a cache whose blocks
    differ in size, as heads and tokens of a model do."""
    x = torch.randn((pages, page, heads, dim), generator=gen, device=DEV)
    size = torch.randn((pages, page // BLOCK, heads), generator=gen, device=DEV).mul_(0.3).exp_()
    x = x.view(pages, page // BLOCK, BLOCK, heads, dim) * size[:, :, None, :, None]
    scale = torch.ldexp(torch.ones_like(size), _needed(x.abs().amax((2, 4))))
    x /= scale[:, :, None, :, None]
    codes = x.view(pages, page, heads, dim).to(torch.float8_e4m3fn).view(torch.uint8)
    if heads_first:  # the same view, stored with the heads before a page's tokens
        codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
    return codes, scale


def _table(lengths, page, gen, total):
    """Pages of `lengths` tokens a request, taken from a shuffled pool."""
    have = [-(-n // page) for n in lengths]
    pool = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(have), max(have)), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max(have), device=DEV)[None, :] < _int(have)[:, None]] = pool[:sum(have)]
    return table


def _starts(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return _int(cu)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"append": _prepare_append, "read": _prepare_read, "attention": _prepare_attention}[case["op"]](case, gen)


def _frequencies(case):
    """Radians per position of each rotated pair, in 64 bits."""
    return case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])


def _prepare_append(case, gen):
    T, Hq, Hkv, D, page = case["T"], case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["fused"]:  # views into the rows of one projection
        row = _randn((T, (Hq + 2 * Hkv) * D), gen)
        q = row[:, :Hq * D].view(T, Hq, D)
        k = row[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = row[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    else:
        q, k, v = _randn((T, Hq, D), gen), _randn((T, Hkv, D), gen), _randn((T, Hkv, D), gen)
    if T <= 512:  # decode tokens stand anywhere, each in a page of its own request
        pos = torch.randint(0, case["maxpos"], (T,), generator=gen, device=DEV)
        pages = T + 8
        slots = torch.randperm(pages, generator=gen, device=DEV)[:T] * page + pos % page
    else:  # a chunk's tokens follow one another; pages lie scattered
        pos = torch.randint(0, case["maxpos"] - T + 1, (1,), generator=gen, device=DEV) + torch.arange(T, device=DEV)
        pages = -(-T // page) + 8
        at = pos - pos[0] // page * page
        slots = torch.randperm(pages, generator=gen, device=DEV)[at // page] * page + at % page
    kc, ks = _cache(pages, page, Hkv, D, case["heads_first"], gen)
    vc, vs = _cache(pages, page, Hkv, D, case["heads_first"], gen)
    # 64-bit fixed-point turns a position: what both forms rotate by
    turns = [int(round(f / TWO_PI * 2.0 ** 64)) for f in _frequencies(case).tolist()]
    freqs = torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in turns], dtype=torch.int64, device=DEV)
    s = {"case": case, "q": q, "k": k, "v": v, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "pos": pos.to(torch.int32),
         "slots": slots.to(torch.int32), "freqs": freqs}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        s["call"] = kda.prepare_rope_append_fp8(q, k, v, s["pos"], s["slots"], freqs, kc, vc, ks, vs,
                                                interleaved=case["interleaved"])
    return s


def _prepare_read(case, gen):
    _, kv = _lengths(case)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    total = sum(-(-n // page) for n in kv) + 8
    kc, ks = _cache(total, page, Hkv, D, case["heads_first"], gen)
    vc, vs = _cache(total, page, Hkv, D, case["heads_first"], gen)
    s = {"case": case, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": _table(kv, page, gen, total), "cu": _starts(kv),
         "kv": _int(kv), "rows": sum(kv)}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        s["call"] = kda.prepare_paged_read_fp8(kc, vc, ks, vs, s["table"], s["cu"], s["kv"], num_tokens=s["rows"])
    return s


def _prepare_attention(case, gen):
    new, cached = _lengths(case)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    kv = [n + c for n, c in zip(new, cached)]
    total = sum(-(-x // page) for x in kv) + 8
    T = sum(new)
    q = _randn((T, Hq, D), gen)
    kc, ks = _cache(total, page, Hkv, D, case["heads_first"], gen)
    vc, vs = _cache(total, page, Hkv, D, case["heads_first"], gen)
    s = {"case": case, "q": q, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": _table(kv, page, gen, total),
         "cu": _starts(new), "kv": _int(kv), "new_max": max(new), "kv_max": max(kv), "scale": D ** -0.5,
         "window": case["window"]}
    if own:
        from linear_attention_ssm_step_gb300 import kda
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=DEV)
        work = kda.paged_attention_workspace(D, torch.device(DEV))
        s["call"] = kda.prepare_paged_attention_fp8(q, kc, vc, ks, vs, s["table"], s["cu"], s["kv"], out=out, lse=lse,
                                                    scale=s["scale"], window=s["window"], workspace=work)
        s["out"], s["lse"] = out, lse
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        got = state["call"]()
        if op == "append":
            return [got] + _whole(state)
        return list(got) if op == "read" else [state["out"], state["lse"]]
    return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention}[op](state)


def _whole(s):
    """The cache: the numbers that its codes are, and the scales by which these count."""
    return [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn), s["ks"], s["vs"]]


def _turn(x, cos, sin, rot, interleaved):
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        return y
    h = rot // 2
    a, b = y[..., :h], y[..., h:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rot:]], dim=-1)


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _write(x, codes, scales, slots, page):
    """x (fp32 [T, heads, dim]) into the blocks of its slots: a block's scale is the smallest that its largest new value
    needs, or its old one where that is larger and the block has earlier tokens, which are then rounded anew."""
    block, which = torch.unique(slots // BLOCK, return_inverse=True)
    B, H = block.numel(), x.shape[1]
    top = torch.zeros((B, H), device=DEV).scatter_reduce_(0, which[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    first = torch.full((B,), BLOCK, device=DEV).scatter_reduce_(0, which, slots % BLOCK, "amin")
    at, part = block // (page // BLOCK), block % (page // BLOCK)
    before = scales[at, part]
    need = torch.ldexp(torch.ones_like(top), _needed(top))
    after = torch.where(first[:, None] > 0, torch.maximum(before, need), need)
    token = torch.arange(BLOCK, device=DEV)
    places = part[:, None] * BLOCK + token[None, :]
    old = codes[at[:, None], places]
    again = _codes(old.view(torch.float8_e4m3fn).float() * (before / after)[:, None, :, None])
    kept = (token[None, :] < first[:, None])[:, :, None, None]
    codes[at[:, None], places] = torch.where(kept, again, old)
    codes[slots // page, slots % page] = _codes(x / after[which][:, :, None])
    scales[at, part] = after


def _plain_append(s):
    case = s["case"]
    # the phase in 2^-64 turns, wrapping as whole turns drop out; its upper bits as an angle in (-pi, pi)
    phase = s["pos"].long()[:, None] * s["freqs"][None, :]
    angle = (phase >> 32).float() * (TWO_PI / 2.0 ** 32)
    cos, sin = angle.cos()[:, None, :], angle.sin()[:, None, :]
    slots = s["slots"].long()
    _write(_turn(s["k"], cos, sin, case["rot"], case["interleaved"]), s["kc"], s["ks"], slots, case["page"])
    _write(s["v"].float(), s["vc"], s["vs"], slots, case["page"])
    return [_turn(s["q"], cos, sin, case["rot"], case["interleaved"]).to(torch.bfloat16)] + _whole(s)


def _values(codes, scales, pages, places):
    """The fp32 values of tokens `places` of `pages`."""
    return codes[pages, places].view(torch.float8_e4m3fn).float() * scales[pages, places // BLOCK][..., None]


def _plain_read(s):
    page = s["case"]["page"]
    cu = s["cu"].long()
    t = torch.arange(s["rows"], device=DEV)
    r = torch.searchsorted(cu, t, right=True) - 1
    place = t - cu[r]
    pages = s["table"][r, place // page].long()
    return [_values(s["kc"], s["ks"], pages, place % page).to(torch.bfloat16),
            _values(s["vc"], s["vs"], pages, place % page).to(torch.bfloat16)]


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
    k = _values(s["kc"], s["ks"], pages, j % page)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).view(R, Hkv, g, N, L).mul_(s["scale"])
    del k
    p = (kv - n)[:, None] + i[None, :]
    seen = j[None, None, :] <= p[:, :, None]
    if s["window"] > 0:
        seen &= j[None, None, :] > p[:, :, None] - s["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    v = _values(s["vc"], s["vs"], pages, j % page)
    out = torch.matmul(weights.view(R, Hkv, g * N, L), v.permute(0, 2, 1, 3)).view(R, Hkv, g, N, D) / total
    lse = (top + total.log()).squeeze(-1)
    there = i[None, :] < n[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(R, N, Hq, D)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(R, N, Hq)[there]
    return [out.to(torch.bfloat16), lse]


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention}[case["op"]](s)


def _exact_write(x, codes, scales, slots, page):
    """The cache after the append, its codes before they are rounded."""
    per = page // BLOCK
    P, _, H, D = codes.shape
    held = codes.view(torch.float8_e4m3fn).double().reshape(P * per, BLOCK, H, D)
    scale = scales.double().reshape(P * per, H).clone()
    fresh = torch.full((P * per, BLOCK, H, D), math.nan, dtype=torch.float64, device=DEV)
    fresh.view(P * page, H, D)[slots] = x
    new = ~fresh[:, :, :1, 0].isnan()                              # [blocks, 16, 1]
    before = ~new & (new.long().cumsum(1) == 0) & new.any(1, keepdim=True)  # tokens of written blocks ahead of the new ones
    top = fresh.nan_to_num(0.0).abs().amax((1, 3))
    e = torch.ceil(torch.log2(top / 448.0)).clamp(LOW, HIGH)
    e = torch.where(top * torch.exp2(-e) > 448.0, e + 1, e)        # the logarithm's rounding
    e = torch.where((top * torch.exp2(1 - e) <= 448.0) & (e > LOW), e - 1, e)
    need = torch.exp2(e)
    after = torch.where(before.any(1), torch.maximum(need, scale), need)
    after = torch.where(new.any(1), after, scale)
    ratio = (scale / after)[:, None, :, None]
    held = torch.where(before[..., None], held * ratio, held)
    held = torch.where(new[..., None], fresh / after[:, None, :, None], held)
    return held.reshape(P, page, H, D), after.reshape(P, per, H)


def _exact_append(s):
    case = s["case"]
    rot = case["rot"]
    z = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                    s["pos"].double()[:, None] * _frequencies(case).to(DEV)[None, :])[:, None, :]

    def rotated(x):
        y = x.double().clone()
        part = y[..., :rot]
        pair = part.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, rot // 2)).mT
        w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        y[..., :rot] = (w if case["interleaved"] else w.mT).flatten(-2)
        return y

    slots = s["slots"].long()
    kc, ks = _exact_write(rotated(s["k"]), s["kc"], s["ks"], slots, case["page"])
    vc, vs = _exact_write(s["v"].double(), s["vc"], s["vs"], slots, case["page"])
    return [rotated(s["q"]), kc, vc, ks, vs]


def _request(s, codes, scales, r, L):
    """Tokens [0, L) of request r in 64 bits: [L, heads, dim]."""
    at = s["table"][r, :-(-L // s["case"]["page"])].long()
    x = codes[at].view(torch.float8_e4m3fn).double()
    x = x.unflatten(1, (-1, BLOCK)) * scales[at].double()[:, :, None, :, None]
    return x.flatten(0, 2)[:L]


def _exact_read(s):
    kv = s["kv"].tolist()
    return [torch.cat([_request(s, c, f, r, L) for r, L in enumerate(kv)]) for c, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]


def _exact_attention(s):
    case = s["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    g, window = Hq // Hkv, case["window"]
    cu, kv = s["cu"].tolist(), s["kv"].tolist()
    out, lse = [], []
    for r in range(len(kv)):
        n, L = cu[r + 1] - cu[r], kv[r]
        k, v = _request(s, s["kc"], s["ks"], r, L), _request(s, s["vc"], s["vs"], r, L)
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
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "append":
        T, Hq, rot = case["T"], case["Hq"], case["rot"]
        blocks = T if T <= 512 else -(-T // BLOCK) + 1
        # rows read, turned queries, codes and scales written, positions, slots and frequencies read
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D + 2 * T * Hq * D + 2 * T * Hkv * D + 16 * blocks * Hkv + 8 * T + 4 * rot,
                "flops": 3 * T * (Hq + Hkv) * rot + 2 * T * Hkv * D}
    new, cached = _lengths(case)
    if case["op"] == "read":
        tokens = sum(cached)
        blocks = sum(-(-c // BLOCK) for c in cached)
        return {"bytes": 2 * tokens * Hkv * D * 3 + 8 * blocks * Hkv, "flops": 2 * tokens * Hkv * D}
    Hq, window = case["Hq"], case["window"]
    pairs, keys = 0, 0
    for n, c in zip(new, cached):
        if window > 0:
            pairs += sum(min(c + i + 1, window) for i in range(n))
            keys += min(n + c, window + n - 1)
        else:
            pairs += n * c + n * (n + 1) // 2
            keys += n + c
    T = sum(new)
    return {"bytes": 2 * keys * Hkv * D + 8 * (keys // BLOCK) * Hkv + 4 * T * Hq * D + 4 * T * Hq,
            "flops": 4 * pairs * Hq * D}
