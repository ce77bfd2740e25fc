"""The attention half of a decode step, operator by operator: what is measured.

Three operators stand between the ternary projections of a layer (q/k/v before
them, o after them):

  rope   RMS norm of every query and key head and the position rotation
  cache  keys and values quantised to 4 bits as they are written into a paged
         cache, and read back
  attn   attention over that cache: single tokens, draft tokens, prompt chunks

With `own` false `run` computes the plain form in elementary torch operations
(32 bits, angles in 64, one rounding at the end); with `own` true it makes the
library's calls.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


# ---- the cases ----

def _rope(T, Hq, Hk, D, rot, pairs, norm, src, dst, far):
    """T tokens, Hq query and Hk key heads of D values, the first `rot` of
    them rotated (pairs: "halves" or "adjacent"), positions up to `far`."""
    return {"op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot, "pairs": pairs, "norm": norm,
            "src": src, "dst": dst, "far": far}


def _cache(T, Hk, D, page, src, dst, order):
    """T tokens of Hk heads of D values; order "run": consecutive slots (a
    prompt), "spread": a slot of its own for each (one token of T sequences)."""
    return {"op": "cache", "T": T, "Hk": Hk, "D": D, "page": page, "src": src, "dst": dst, "order": order}


def _attn(B, S, ctx, Hk, G, D, page, dtype, window=0, ragged=False, lse=False):
    """B sequences with up to S new tokens and ctx tokens in the cache, Hk
    key heads with G query heads each."""
    return {"op": "attn", "B": B, "S": S, "ctx": ctx, "Hk": Hk, "G": G, "D": D, "page": page, "dtype": dtype,
            "window": window, "ragged": ragged, "lse": lse}


def listed():
    return [
        # one token of the 8B stack's layer (q 4096, k 256 wide), straight from the fp32 outputs of its matvecs
        {"name": "rope one token", **_rope(1, 32, 2, 128, 128, "halves", False, "f32", "f16", 32768)},
        # a prompt through the same heads, with norms of the heads
        {"name": "rope prompt 4096", **_rope(4096, 32, 2, 128, 128, "halves", True, "bf16", "bf16", 8192)},
        # an odd batch with rotation of half of the head in adjacent pairs, far positions, fp32 out
        {"name": "rope 333 partial", **_rope(333, 12, 4, 64, 32, "adjacent", True, "f32", "f32", 1000000)},
        # one new token of each of 64 sequences
        {"name": "cache 64 tokens", **_cache(64, 2, 128, 64, "f16", "f16", "spread")},
        # an odd number of fp32 tokens over small heads
        {"name": "cache 1001 tokens", **_cache(1001, 5, 64, 32, "f32", "f32", "run")},
        # a long prompt
        {"name": "cache prompt 16383", **_cache(16383, 8, 128, 64, "bf16", "bf16", "run")},
        # the first answers of a chat: latency
        {"name": "attn 1 x 200", **_attn(1, 1, 200, 2, 16, 128, 32, "f16")},
        # one long document, one token
        {"name": "attn 1 x 131000", **_attn(1, 1, 131000, 2, 16, 128, 64, "f16")},
        # a serving batch of unequal sequences
        {"name": "attn 64 ragged 32768", **_attn(64, 1, 32768, 2, 16, 128, 64, "f16", ragged=True)},
        # a sliding window, four query heads a key head
        {"name": "attn 16 window 4095", **_attn(16, 1, 8192, 8, 4, 128, 64, "bf16", window=4095)},
        # draft tokens of speculative decoding, seven query heads a key head, small heads
        {"name": "attn 8 x 5 drafts", **_attn(8, 5, 8191, 4, 7, 64, 32, "f16", ragged=True, lse=True)},
        # prompt chunks of unequal length behind cached text
        {"name": "attn prefill 1500", **_attn(3, 1500, 5000, 2, 16, 128, 64, "f16", ragged=True)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rope", "cache", "attn", "attn"))
    if op == "rope":
        D = rng.choice((64, 80, 96, 128, 192, 256))
        Hq, Hk = rng.randint(1, 40), rng.randint(1, 8)
        T = _log(rng, 1, max(1, 4096 * 34 * 128 // ((Hq + Hk) * D)))
        rot = rng.choice((D, D, 16 * rng.randint(1, D // 16)))
        src = rng.choice(("f16", "bf16", "f32"))
        return _rope(T, Hq, Hk, D, rot, rng.choice(("halves", "adjacent")), rng.random() < 0.5, src,
                     rng.choice(("f16", "bf16", "f32")), _log(rng, 1, 1000000))
    if op == "cache":
        D, Hk = rng.choice((64, 128, 256)), rng.randint(1, 16)
        T = _log(rng, 1, 16383 * 8 * 128 // (Hk * D))
        return _cache(T, Hk, D, rng.choice((32, 64, 128, 256)), rng.choice(("f16", "bf16", "f32")),
                      rng.choice(("f16", "bf16", "f32")), rng.choice(("run", "spread")))
    D, Hk, G = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 4, 5, 7, 8, 12, 16, 24))
    S = rng.choice((1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 700)))
    B = _log(rng, 1, 64 if S == 1 else 8)
    most = 64 * 32768 * 2 * 128 // (B * Hk * D * 3)                       # cached values, for few tokens
    most = min(most, 3 * 1500 * 32 * 128 * 4000 // (B * S * Hk * G * D))  # products, for many
    ctx = max(S, _log(rng, 1, max(2, min(131000, most))))
    return _attn(B, S, ctx, Hk, G, D, rng.choice((32, 64, 128)), rng.choice(("f16", "bf16")),
                 window=rng.choice((0, 0, 0, _log(rng, 1, ctx))), ragged=rng.random() < 0.6, lse=rng.random() < 0.3)


def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of every sequence.
    In a ragged batch the first is the longest; the last of a larger batch of
    single tokens is a place without a sequence (nothing cached)."""
    B, S, ctx = case["B"], case["S"], case["ctx"]
    if not case["ragged"]:
        return [S] * B, [ctx] * B
    r = random.Random(1000003 * B + 1009 * S + ctx)
    n = [S] + [r.randint(1, S) for _ in range(B - 1)]
    c = [ctx] + [max(n[b], _log(r, max(1, ctx // 64), ctx)) for b in range(1, B)]
    if S == 1 and B >= 4:
        c[-1] = 0
    return n, c


def _visible(n, c, window):
    """(cached tokens that some new token sees, pairs of tokens that see each other)"""
    tokens = pairs = 0
    for nb, cb in zip(n, c):
        first = max(0, cb - nb + 1 - window) if window else 0
        tokens += cb - first
        for i in range(nb):
            seen = max(0, cb - nb + i + 1)
            pairs += min(seen, window) if window else seen
    return tokens, pairs


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": n * (SIZE[case["src"]] + SIZE[case["dst"]]) + 4 * case["T"] + 2 * case["rot"], "flops": 10 * n}
    if case["op"] == "cache":
        n = 2 * case["T"] * case["Hk"]
        held = D // 2 + 4
        return {"bytes": n * (D * (SIZE[case["src"]] + SIZE[case["dst"]]) + 2 * held) + 16 * case["T"], "flops": 8 * n * D}
    n, c = _lengths(case)
    tokens, pairs = _visible(n, c, case["window"])
    heads = case["Hk"] * case["G"]
    moved = tokens * case["Hk"] * (D + 8) + 2 * sum(n) * heads * D * SIZE[case["dtype"]] + 4 * tokens // case["page"]
    return {"bytes": moved + (4 * sum(n) * heads if case["lse"] else 0), "flops": 4 * D * heads * pairs}


# ---- inputs ----

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _heads(g, T, H, D, dtype):
    """Head outputs: a spread of sizes over the channels, a few of them far larger, and an offset."""
    spread = torch.exp(0.3 * _normal(g, H, D))
    spread = torch.where(torch.rand((H, D), generator=g, device=DEV) < 0.02, 6 * spread, spread)
    return (_normal(g, T, H, D) * spread + 0.5 * _normal(g, H, D)).to(dtype)


def _levels(x):
    """The 4-bit form of the last axis: codes, scale and middle.  The two
    quotients go through 64 bits, which rounds them to 32 as a division does:
    a code next to a border depends on the last bit."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    z = ((hi + lo) * 0.5).half()
    s = ((hi - lo).double() / 15).float().half()
    c = ((x - z.float()).double() / torch.where(s == 0, 1, s.double())).float()
    c = (c + 7.5).round().clamp(0, 15)
    return torch.where(s == 0, 0, c).to(torch.uint8), s, z


def _value_bytes(D):
    """Where byte j of a token's value codes stands in its tile of 32 tokens, less the token's own part."""
    d = 2 * torch.arange(D // 2, device=DEV)
    n, h, byte = d // (D // 16), d % (D // 16) // 4, d % 4 // 2
    return (n * (D // 64) + h) * 16 + byte


def _places(case, slots):
    """Byte offsets in the cache of every (slot, head): key codes, value codes
    [T, Hk, D/2], and the (scale, middle) pairs of keys and of values [T, Hk, 4]."""
    Hk, D, page = case["Hk"], case["D"], case["page"]
    head = torch.arange(Hk, device=DEV)
    base = ((slots // page)[:, None] * Hk + head) * (page * (D + 8))
    at = (slots % page)[:, None]
    j = torch.arange(D // 2, device=DEV)
    keys = (base + at * (D // 2))[..., None] + j
    tile = page * (D // 2) + at // 32 * (16 * D) + at % 32 // 8 * (4 * D) + at % 8 * 2
    values = (base + tile)[..., None] + _value_bytes(D)
    pair = torch.arange(4, device=DEV)
    kp = (base + page * D + at * 4)[..., None] + pair
    return keys, values, kp, kp + page * 4


def _pair_bytes(s, z):
    return torch.cat((s, z), -1).contiguous().view(torch.uint8)


def _write(case, cache, slots, k, v):
    flat = cache.view(-1)
    keys, values, kp, vp = _places(case, slots)
    for x, codes_at, pair_at in ((k, keys, kp), (v, values, vp)):
        c, s, z = _levels(x)
        flat[codes_at] = c[..., 0::2] | (c[..., 1::2] << 4)
        flat[pair_at] = _pair_bytes(s, z)


def _read(case, cache, slots, dtype):
    flat = cache.view(-1)
    keys, values, kp, vp = _places(case, slots)
    out = []
    for codes_at, pair_at in ((keys, kp), (values, vp)):
        b = flat[codes_at]
        c = torch.stack((b & 15, b >> 4), -1).flatten(-2).float()
        p = flat[pair_at].view(torch.float16).float()
        out.append((p[..., 1:2] + p[..., 0:1] * (c - 7.5)).to(dtype))
    return out


def prepare(case, seed):
    g = _generator(seed)
    D, Hk = case["D"], case["Hk"]
    if case["op"] == "rope":
        T, Hq = case["T"], case["Hq"]
        # the outputs of one q/k/v call: [T, q heads | k heads | v heads]
        x = _heads(g, T, Hq + 2 * Hk, D, TYPES[case["src"]])
        far = case["far"]
        start = int(torch.randint(max(1, far - T), (1,), generator=g, device=DEV))
        positions = start + torch.arange(T, device=DEV, dtype=torch.int32)
        inv_freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        w = [(1 + 0.2 * _normal(g, D)) if case["norm"] else None for _ in range(2)]
        return {"case": case, "q": x[:, :Hq], "k": x[:, Hq:Hq + Hk], "positions": positions,
                "inv_freq": inv_freq.float(), "qw": w[0], "kw": w[1],
                "q_out": torch.empty((T, Hq, D), dtype=TYPES[case["dst"]], device=DEV),
                "k_out": torch.empty((T, Hk, D), dtype=TYPES[case["dst"]], device=DEV)}
    page = case["page"]
    if case["op"] == "cache":
        T = case["T"]
        x = _heads(g, T, 2 * Hk, D, TYPES[case["src"]])
        if case["order"] == "run":  # a prompt: pages in an order of their own, tokens in theirs
            pages = -(-(T + 1) // page) + 3
            order = torch.randperm(pages, generator=g, device=DEV)
            at = torch.arange(T, device=DEV) + int(torch.randint(page, (1,), generator=g, device=DEV)) % (pages * page - T)
            slots = order[at // page] * page + at % page
        else:  # one token somewhere in a page of each sequence
            pages = T + 3
            slots = torch.randperm(pages, generator=g, device=DEV)[:T] * page
            slots = slots + torch.randint(page, (T,), generator=g, device=DEV)
        cache = torch.zeros((pages, Hk, page * (D + 8)), dtype=torch.uint8, device=DEV)
        outs = [torch.empty((T, Hk, D), dtype=TYPES[case["dst"]], device=DEV) for _ in range(2)]
        return {"case": case, "k": x[:, :Hk], "v": x[:, Hk:], "slots": slots, "cache": cache, "outs": outs}
    n, c = _lengths(case)
    B, heads, dtype = case["B"], Hk * case["G"], TYPES[case["dtype"]]
    T = sum(n)
    need = [-(-cb // page) for cb in c]
    width, pages = max(1, max(need)), sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    used = 0
    for b in range(B):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
    # pages of keys whose channels differ in size and values around zero; what
    # stands behind a sequence's last token is what its page held before
    cache = torch.empty((pages, Hk, page * (D + 8)), dtype=torch.uint8, device=DEV)
    spread = torch.exp(0.3 * _normal(g, Hk, 1, D))
    spread = torch.where(torch.rand((Hk, 1, D), generator=g, device=DEV) < 0.02, 6 * spread, spread)
    offset = 0.5 * _normal(g, Hk, 1, D)
    step = max(1, (1 << 26) // (Hk * page * D))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        kc, ks, kz = _levels(_normal(g, m, Hk, page, D) * spread + offset)
        vc, vs, vz = _levels(_normal(g, m, Hk, page, D))
        kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(m, Hk, -1)
        vb = vc[..., 0::2] | (vc[..., 1::2] << 4)
        # tokens (tile, g, i) x bytes (n, h, byte) -> tile, g, n, h, i, byte
        vb = vb.view(m, Hk, page // 32, 4, 8, 16, D // 64, 2).permute(0, 1, 2, 3, 5, 6, 4, 7).reshape(m, Hk, -1)
        cache[p:p + m] = torch.cat((kb, vb, _pair_bytes(ks, kz).reshape(m, Hk, -1),
                                    _pair_bytes(vs, vz).reshape(m, Hk, -1)), -1)
    # queries that make the scores spread over a few units
    q = (_normal(g, T, heads, D) * 0.7).to(dtype)
    starts = [0]
    for nb in n:
        starts.append(starts[-1] + nb)
    return {"case": case, "q": q, "cache": cache, "table": table,
            "ctx": torch.tensor(c, dtype=torch.int32, device=DEV),
            "starts": torch.tensor(starts, dtype=torch.int32, device=DEV) if case["ragged"] else None,
            "out": torch.empty_like(q), "scale": 1 / math.sqrt(D),
            "lse": torch.empty((T, heads), device=DEV) if case["lse"] else None,
            # scratch that a program keeps for all its layers
            "ws": torch.empty(64 << 20, dtype=torch.uint8, device=DEV)}


# ---- plain forms ----

def _plain_rope(state):
    case = state["case"]
    R = case["rot"]
    # angles of far positions need 64 bits before they are reduced
    a = state["positions"].double()[:, None] * state["inv_freq"].double()
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    outs = []
    for x, w, out in ((state["q"], state["qw"], state["q_out"]), (state["k"], state["kw"], state["k_out"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        if case["pairs"] == "halves":
            u, v = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
        else:
            u, v = y[..., 0:R:2], y[..., 1:R:2]
            turned = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
        out.copy_(torch.cat((turned, y[..., R:]), -1))
        outs.append(out)
    return outs


def _plain_attn(state):
    case = state["case"]
    B, S, Hk, G, D, page = (case[k] for k in ("B", "S", "Hk", "G", "D", "page"))
    q, table, ctx = state["q"], state["table"], state["ctx"].long()
    T, width = q.shape[0], table.shape[1]
    L = width * page
    held = state["cache"][table.clamp(min=0).long()].transpose(1, 2)        # [B, Hk, width, bytes]

    def values(codes, pairs):
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
        p = pairs.contiguous().view(torch.float16).view(B, Hk, L, 2).float()
        return p[..., 1:] + p[..., :1] * (c.view(B, Hk, L, D) - 7.5)

    half = page * D // 2
    k = values(held[..., :half].reshape(B, Hk, L, D // 2), held[..., 2 * half:2 * half + 4 * page])
    vc = held[..., half:2 * half].reshape(B, Hk, width, page // 32, 4, 16, D // 64, 8, 2)
    v = values(vc.permute(0, 1, 2, 3, 4, 7, 5, 6, 8).reshape(B, Hk, L, D // 2), held[..., 2 * half + 4 * page:])
    # new tokens in a padded batch, [B, S]
    if state["starts"] is None:
        n = torch.full((B,), S, device=DEV)
        first = S * torch.arange(B, device=DEV)
    else:
        first = state["starts"][:-1].long()
        n = state["starts"][1:].long() - first
    i = torch.arange(S, device=DEV)
    rows = (first[:, None] + i).clamp(max=T - 1)
    qp = q[rows].float().view(B, S, Hk, G, D).transpose(1, 2).reshape(B * Hk, S * G, D)
    x = torch.bmm(qp * state["scale"], k.view(B * Hk, L, D).transpose(1, 2)).view(B, Hk, S, G, L)
    last = (ctx - n)[:, None] + i                                            # [B, S], the token's own place
    j = torch.arange(L, device=DEV)
    seen = (j <= last[..., None]) & (j < ctx[:, None, None])
    if case["window"]:
        seen &= j > last[..., None] - case["window"]
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(B * Hk, S * G, L), v.view(B * Hk, L, D)).view(B, Hk, S, G, D)
    o = torch.where(total > 0, o / total, 0)
    sequence = torch.searchsorted(first + n, torch.arange(T, device=DEV), right=True)
    at = torch.arange(T, device=DEV) - first[sequence]
    state["out"].copy_(o.transpose(1, 2).reshape(B, S, Hk * G, D)[sequence, at])
    if state["lse"] is None:
        return state["out"]
    lse = (torch.log(total) + m).transpose(1, 2).reshape(B, S, Hk * G)
    state["lse"].copy_(lse[sequence, at])
    return state["out"], state["lse"]


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "rope":
            return _plain_rope(state)
        if case["op"] == "attn":
            return _plain_attn(state)
        _write(case, state["cache"], state["slots"], state["k"], state["v"])
        return _read(case, state["cache"], state["slots"], TYPES[case["dst"]])
    from ternary_packed_weight_amd import tq2
    if case["op"] == "rope":
        return tq2.tq2_qk_norm_rope(state["q"], state["k"], state["positions"], state["inv_freq"],
                                    q_weight=state["qw"], k_weight=state["kw"], eps=1e-6,
                                    interleaved=case["pairs"] == "adjacent", q_out=state["q_out"], k_out=state["k_out"])
    if case["op"] == "cache":
        tq2.tq2_kv4_store(state["cache"], state["k"], state["v"], state["slots"])
        return tq2.tq2_kv4_load(state["cache"], state["slots"], case["D"], k_out=state["outs"][0], v_out=state["outs"][1])
    out = tq2.tq2_kv4_attn(state["q"], state["cache"], state["table"], state["ctx"], q_start=state["starts"],
                           max_q=case["S"], scale=state["scale"], window=case["window"], out=state["out"],
                           lse=state["lse"], ws=state["ws"])
    return out if state["lse"] is None else (out, state["lse"])


# ---- the definitions in 64 bits ----

def _exact_levels(x):
    """The value that each entry of the last axis stands for: the steps of the
    definition that are fp32 (the difference, the quotient and the sum) are
    rounded to it one by one, the value itself is not."""
    lo, hi = x.min(dim=-1, keepdim=True).values, x.max(dim=-1, keepdim=True).values

    def f32(t):
        return t.to(torch.float32).to(torch.float64)

    z = f32(f32(hi + lo) / 2).to(torch.float16).double()
    s = f32(f32(hi - lo) / 15).to(torch.float16).double()
    c = f32(f32(f32(x - z) / s) + 7.5)
    c = torch.nan_to_num(torch.minimum(torch.maximum(torch.round(c), torch.zeros_like(c)), torch.full_like(c, 15.0)))
    return torch.where(s == 0, z.expand_as(c), z + s * (c - 7.5))


def _exact_held(case, cache, slots, h):
    """Keys and values of head h that the cache holds for the slots, [len(slots), D] in 64 bits, entry by entry."""
    D, page = case["D"], case["page"]
    block = cache[slots // page, h]                                          # [L, bytes of the page]
    t, d = (slots % page)[:, None], torch.arange(D, device=DEV)[None, :]
    kb = torch.gather(block, 1, t * (D // 2) + d // 2).long()
    unit = (((t // 32) * 4 + t % 32 // 8) * 16 + d // (D // 16)) * (D // 64) + d % (D // 16) // 4
    vb = torch.gather(block, 1, page * D // 2 + (unit * 8 + t % 8) * 2 + d % 4 // 2).long()
    shift = 4 * (d % 2)
    pairs = block[:, page * D:].contiguous().view(torch.float16).view(-1, 2, page, 2)[torch.arange(len(slots), device=DEV), :, t[:, 0]]
    pairs = pairs.double()                                                   # [L, key or value, scale and middle]
    return tuple(pairs[:, w, 1:] + pairs[:, w, :1] * (((b >> shift) & 15).double() - 7.5) for w, b in ((0, kb), (1, vb)))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "cache":
        return [_exact_levels(state[name].double()) for name in ("k", "v")]
    if case["op"] == "rope":
        R, outs = case["rot"], []
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.outer(state["positions"].double(), state["inv_freq"].double()))
        for name, weight in (("q", "qw"), ("k", "kw")):
            y = state[name].double().clone()
            if state[weight] is not None:
                y /= torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6)
                y *= state[weight].double()
            if case["pairs"] == "halves":
                z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * turn[:, None, :]
                y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
            else:
                z = torch.view_as_complex(y[..., :R].reshape(*y.shape[:-1], R // 2, 2).contiguous()) * turn[:, None, :]
                y[..., :R] = torch.view_as_real(z).flatten(-2)
            outs.append(y)
        return outs
    Hk, G, page, window = (case[k] for k in ("Hk", "G", "page", "window"))
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (nb, cb) in enumerate(zip(*_lengths(case))):
        j = torch.arange(cb, device=DEV)
        slots = state["table"][b].long()[j // page] * page + j % page
        place = cb - nb + torch.arange(nb, device=DEV)
        hidden = j[None] > place[:, None]
        if window:
            hidden |= j[None] <= place[:, None] - window
        for h in range(Hk if cb else 0):
            heads = slice(h * G, h * G + G)
            k, v = _exact_held(case, state["cache"], slots, h)
            q = state["q"][t0:t0 + nb, heads].double()                       # [nb, G, D]
            x = (q.reshape(nb * G, -1) @ k.T.contiguous() * state["scale"]).view(nb, G, cb)
            x.masked_fill_(hidden[:, None], -math.inf)
            e = torch.logsumexp(x, -1)
            x -= torch.where(torch.isfinite(e), e, 0.0)[..., None]
            out[t0:t0 + nb, heads] = (x.exp_().view(nb * G, cb) @ v).view(nb, G, -1)
            lse[t0:t0 + nb, heads] = e
        t0 += nb
    return (out, lse) if case["lse"] else out
