"""The attention over the 4-bit cache at sizes where its work is split and
dealt, the cache's calls on long prompts, and the binding's short way, on the
GPU.  References: 64-bit products of the values that the cache's bytes stand
for, or the same calls made in other pieces."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_kv4_gpu import check_attn, filled, layer_inputs, set_place

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


# ---- small oracle cases where tokens are split among workgroups ----

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_rows_split(tq2, D, dtype):
    check_attn(tq2, [40, 9], [700, 300], 1, 4, D, 64, dtype, seed=D)


@pytest.mark.parametrize("G,ns,ctx,window", [(33, [3, 1], [900, 40], 0), (1, [70, 130], [333, 130], 0), (16, [20, 4, 0, 7], [600, 5, 9, 7], 0),
                                             (5, [30], [1000], 100), (7, [64, 2], [64, 900], 33), (2, [200], [150], 0)])
def test_many_rows_shapes(tq2, G, ns, ctx, window):
    check_attn(tq2, ns, ctx, 1, G, 64, 32, F16, window=window, seed=G)


@pytest.mark.parametrize("B", [3, 65, 130])
def test_few_rows_of_many_sequences(tq2, B):
    """Lengths are summed by 64 lanes: one, two and three sequences a lane."""
    g = np.random.default_rng(B)
    ctx = [int(c) for c in np.floor(np.exp(g.uniform(0, 6, B)))]
    ctx[B // 2], ctx[B - 1], ctx[0] = 2000, 0, 1
    check_attn(tq2, [1] * B, ctx, 1, 3, 64, 32, F16, seed=B, ragged=False)


def test_more_sequences_than_threads_that_deal(tq2):
    """1500 sequences, two for each thread of the workgroup that writes the list; places without a sequence among them."""
    g = np.random.default_rng(7)
    ctx = [int(c) for c in np.floor(np.exp(g.uniform(0, 3.5, 1500)))]
    ctx[3], ctx[1024], ctx[1499], ctx[700] = 0, 1800, 900, 0
    check_attn(tq2, [1] * 1500, ctx, 1, 2, 64, 32, F16, seed=7, ragged=False)


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16), (256, F16)])
def test_many_rows_of_long_text(tq2, D, dtype):
    check_attn(tq2, [21, 0, 9], [1300, 40, 1111], 1, 5, D, 64, dtype, seed=D + 1)
    check_attn(tq2, [70], [1200], 1, 1, D, 32, dtype, window=1000, seed=D + 2)


def test_drafts_split(tq2):
    check_attn(tq2, [5, 3, 1], [1500, 40, 700], 2, 7, 64, 32, F16, seed=1)      # 35 rows: two row tiles
    check_attn(tq2, [2, 2], [900, 1100], 1, 12, 256, 64, BF16, window=700, seed=2)


def test_split_pages_that_are_not_there(tq2):
    cache, g = filled(5, 30, 1, 32, 64)
    table = g.permutation(30).astype(np.int32)[None].repeat(2, 0)
    table[0, 3], table[0, 17], table[1, ::2] = -1, 30, 2147483647
    check_attn(tq2, [1, 1], [950, 900], 1, 8, 64, 32, F16, cache=cache, table=table, seed=3)
    check_attn(tq2, [20, 20], [950, 900], 1, 5, 64, 32, F16, cache=cache, table=table, seed=4)


@pytest.mark.parametrize("bad", [0x7e00, 0x7c00, 0xffff])
def test_many_rows_unseen_places_hold_anything(tq2, bad):
    """What later new tokens, and places behind the end, hold does not act on a row."""
    P, D = 32, 64
    cache, g = filled(6, 20, 1, P, D)
    pairs = cache.bytes[..., P * D:].view(np.uint16).reshape(20, 1, 2, P, 2)
    table = np.arange(20, dtype=np.int32)[None]
    q = torch.from_numpy(g.standard_normal((40, 4, D))).to(F16).to(DEV)
    run = lambda: tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                                   torch.tensor([600], dtype=torch.int32, device=DEV)).cpu()
    clean = run()
    for t in range(600, 640):
        pairs[t // P, :, :, t % P] = bad
    assert torch.equal(run(), clean)
    pairs[599 // P, :, :, 599 % P] = bad                                        # the last new token's place
    assert torch.equal(run()[:39], clean[:39])


# ---- long ones against 64-bit products on the GPU ----

def dequantized(cache):
    """Keys, values and |scale * (code - 7.5)| of the values, [pages, Hk, P, D] in 64 bits, from the layout."""
    P, D, pages, Hk = cache.P, cache.D, cache.pages, cache.Hk
    half = P * D // 2
    b = torch.from_numpy(cache.bytes).to(DEV)
    pairs = b[..., 2 * half:].contiguous().view(torch.float16).view(pages, Hk, 2, P, 2).double()
    nibbles = lambda x: torch.stack((x & 15, x >> 4), -1).flatten(-2).double()
    kc = nibbles(b[..., :half].reshape(pages, Hk, P, D // 2))
    v = b[..., half:2 * half].reshape(pages, Hk, P // 8, D // 4, 8, 2).transpose(3, 4)
    vc = nibbles(v.reshape(pages, Hk, P, D // 2))
    held = lambda c, p: p[..., 1:] + p[..., :1] * (c - 7.5)
    return held(kc, pairs[:, :, 0]), held(vc, pairs[:, :, 1]), (pairs[:, :, 1, :, :1] * (vc - 7.5)).abs()


def check_long(tq2, ns, ctx, Hk, G, D, P, dtype, window=0, seed=0):
    B, T, scale = len(ns), sum(ns), D ** -0.5
    need = [-(-c // P) for c in ctx]
    cache, g = filled(seed, sum(need) + 1, Hk, P, D)
    order, table, used = g.permutation(cache.pages), np.full((B, max(need)), -1, np.int32), 0
    for b in range(B):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
    q = torch.from_numpy(g.standard_normal((T, Hk * G, D)) * 0.8).to(dtype).to(DEV)
    start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    lse = torch.full((T, Hk * G), float("nan"), device=DEV)
    call = lambda: tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                                    torch.tensor(ctx, dtype=torch.int32, device=DEV), q_start=torch.from_numpy(start).to(DEV),
                                    max_q=max(ns), window=window, lse=lse)
    out = call()
    again = call()
    assert torch.equal(out, again)
    # few rows keep 22 bits of a weight times its scale, many one rounding to binary16
    kept = 2.0 ** -22 if max(ns) * G <= 64 else 2.0 ** -11
    K, V, C = dequantized(cache)
    pairs = torch.from_numpy(cache.bytes[..., P * D:].copy()).view(torch.float16).view(cache.pages, Hk, 2, P, 2).double().abs()
    kmag = float((7.5 * pairs[:, :, 0, :, 0] + pairs[:, :, 0, :, 1]).max())
    vmag = float((15 * pairs[:, :, 1, :, 0] + pairs[:, :, 1, :, 1]).max())
    eps = torch.finfo(dtype).eps
    for b in range(B):
        t0, n, c = int(start[b]), ns[b], ctx[b]
        if n == 0:
            continue
        j = torch.arange(c, device=DEV)
        pages = torch.from_numpy(table[b]).to(DEV).long()
        place = c - n + torch.arange(n, device=DEV)
        seen = j[None] <= place[:, None]
        if window:
            seen &= j[None] > place[:, None] - window
        for h in range(Hk):
            k, v, cen = (x[pages[j // P], h, j % P].contiguous() for x in (K, V, C))
            for g0 in range(G):
                qh = q[t0:t0 + n, h * G + g0].double()
                x = qh @ k.T.contiguous() * scale
                x = torch.where(seen, x, -torch.inf)
                top = x.amax(-1, keepdim=True)
                p = torch.exp(x - top)
                total = p.sum(-1, keepdim=True)
                l = (top + torch.log(total))[:, 0]
                p = p / total
                o = p @ v
                # as the small oracle's: 16 fp32 roundings of a score's magnitudes, sums over 32 accumulators
                score = 16 * 2.0 ** -24 * (kmag * qh.abs().sum(-1, keepdim=True) * scale + top.abs())
                sums = (seen.sum(-1, keepdim=True) / 32 + 64) * 2.0 ** -24
                tol = (eps / 2 * o.abs() + ref.F16_STEP + kept * (p @ cen) + 2 * score * (p @ v.abs() + o.abs()) + sums * vmag)
                bad = (out[t0:t0 + n, h * G + g0].double() - o).abs() / tol
                assert float(bad.max()) <= 1, (b, h, g0, float(bad.max()))
                ltol = (2 * score + sums)[:, 0] + 2.0 ** -22 * l.abs()
                assert bool(((lse[t0:t0 + n, h * G + g0].double() - l).abs() <= ltol).all())


def test_one_long_sequence(tq2):
    check_long(tq2, [1], [70001], 2, 16, 128, 64, F16, seed=1)
    check_long(tq2, [1], [20000], 1, 4, 256, 64, BF16, window=17000, seed=2)


def test_unequal_sequences(tq2):
    g = np.random.default_rng(3)
    ctx = [int(c) for c in np.floor(np.exp(g.uniform(3, 9, 40)))] + [30000]
    check_long(tq2, [1] * 41, ctx, 2, 8, 128, 64, F16, seed=3)


def test_long_drafts(tq2):
    check_long(tq2, [5, 2, 4], [9000, 100, 3000], 2, 7, 64, 32, F16, seed=4)


def test_prompt_chunks_dealt_from_a_list(tq2):
    """More row tiles than workgroups at once, unequal lengths."""
    check_long(tq2, [600, 90, 333], [3900, 90, 400], 8, 4, 128, 64, BF16, seed=5)
    check_long(tq2, [300, 1], [5000, 4000], 1, 16, 64, 32, F16, window=3500, seed=6)


def test_prompt_of_few_rows_tiles(tq2):
    """Few row tiles over long text: many parts each."""
    check_long(tq2, [10], [8000], 1, 16, 128, 64, F16, seed=7)
    check_long(tq2, [9], [4000], 2, 12, 256, 32, BF16, seed=8)


# ---- prompts into the cache ----

@pytest.mark.parametrize("D,T,Hk", [(64, 16500, 1), (128, 2100, 8), (256, 1111, 16)])
@pytest.mark.parametrize("first", [0, 5, 31])
def test_long_prompt_stores_what_short_ones_do(tq2, D, T, Hk, first):
    """A long run of slots, page by page in an order of their own, in one call
    and in pieces; some slots name no page."""
    P = 64
    g = torch.Generator(device=DEV).manual_seed(D + first)
    x = torch.randn((T, 2 * Hk, D), generator=g, device=DEV).to(BF16)
    pages = -(-(T + first) // P) + 1
    at = torch.arange(T, device=DEV) + first
    slots = torch.randperm(pages, generator=g, device=DEV)[at // P] * P + at % P
    slots[7], slots[T // 2] = -1, pages * P
    whole = torch.full((pages, Hk, P * (D + 8)), 0x5a, dtype=torch.uint8, device=DEV)
    parts = whole.clone()
    tq2.tq2_kv4_store(whole, x[:, :Hk], x[:, Hk:], slots)
    for t in range(0, T, 97):
        tq2.tq2_kv4_store(parts, x[t:t + 97, :Hk], x[t:t + 97, Hk:], slots[t:t + 97].contiguous())
    assert torch.equal(whole, parts)
    k, v = tq2.tq2_kv4_load(whole, slots, D, dtype=F32)
    rows = torch.randint(0, T, (40,), generator=g, device=DEV).tolist() + [0, 7, T // 2, T - 1]
    for y, x0 in ((k, x[:, :Hk]), (v, x[:, Hk:])):
        want = torch.from_numpy(ref.held(*ref.quantize(x0[rows].float().cpu().numpy()))).float()
        for i, t in enumerate(rows):
            if t in (7, T // 2):
                want[i] = 0
        assert torch.equal(y[rows].cpu(), want)
    for t in range(0, T, 97):
        kt, vt = tq2.tq2_kv4_load(whole, slots[t:t + 97].contiguous(), D, dtype=F32)
        assert torch.equal(kt, k[t:t + 97]) and torch.equal(vt, v[t:t + 97])


def test_scales_between_two_halves(tq2):
    """Heads whose (largest - least) / 15 is half way between two binary16
    numbers: the quotient is rounded to fp32 first, then to the even one."""
    D, Hk, T = 64, 4, 3000
    g = np.random.default_rng(4)
    x = (g.random((T * 2 * Hk, D)) - 0.5).astype(np.float32) * np.float32(1e-3)
    tie = (g.integers(1024, 2048, len(x)) + 0.5) * np.exp2(g.integers(-14, -6, len(x)))
    hi = np.floor(g.uniform(0.2, 0.8, len(x)) * 15 * tie * 2 ** 14) * 2.0 ** -14
    lo = hi - 15 * tie
    exact = lo.astype(np.float32).astype(np.float64) == lo
    assert exact.mean() > 0.5
    x[:, 0], x[:, 1] = hi, lo
    x = x.reshape(T, 2 * Hk, D)
    cache = torch.zeros((-(-T // 32), Hk, 32 * (D + 8)), dtype=torch.uint8, device=DEV)
    xd = torch.from_numpy(x).to(DEV)
    slots = torch.arange(T, device=DEV)
    tq2.tq2_kv4_store(cache, xd[:, :Hk], xd[:, Hk:], slots)
    k, v = tq2.tq2_kv4_load(cache, slots, D, dtype=F32)
    for y, x0 in ((k, x[:, :Hk]), (v, x[:, Hk:])):
        assert torch.equal(y.cpu(), torch.from_numpy(ref.held(*ref.quantize(x0))).float())


def test_many_tokens_average_out(tq2):
    """An output far smaller than the values that it averages keeps its relative
    precision: half a step of binary16, and 2^-13 of the output's size for the
    rest.  Nor do the channels whose codes are the lowest in a byte lean to one
    side: roundings of up to half a step, 2^-12 of the size, average to about
    2^-17 over 1024 outputs."""
    n, D, P, Hk = 131000, 128, 64, 1
    cache, g = filled(21, -(-n // P), Hk, P, D)
    pairs = cache.bytes[..., P * D:].view(np.float16).reshape(-1, Hk, 2, P, 2)
    pairs[:, :, 1, :, 1] = 0
    q = torch.from_numpy(0.3 * np.random.default_rng(3).standard_normal((1, 16, D))).to(F16).to(DEV)
    table = torch.arange(cache.pages, dtype=torch.int32, device=DEV)[None]
    out = tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), table, torch.tensor([n], dtype=torch.int32, device=DEV))[0].double()
    K, V, _ = dequantized(cache)
    k, v = K.reshape(-1, D)[:n].contiguous(), V.reshape(-1, D)[:n].contiguous()
    want = torch.softmax(q[0].double() @ k.T.contiguous() * D ** -0.5, -1) @ v
    size = want.pow(2).mean().sqrt()
    assert float(size) < 0.01
    off = out - want
    assert bool((off.abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -25 + 2.0 ** -13 * size * 4).all())
    assert float(off[:, ::2].mean().abs() / size) <= 2.0 ** -15


def test_sequences_behind_each_other_in_one_store(tq2):
    """Runs that start at different places of a page, in one call."""
    P, D, Hk = 32, 128, 4
    lengths, firsts = [4000, 1, 700, 33, 1300], [3, 30, 0, 17, 8]
    slots, page = [], 0
    for n, f in zip(lengths, firsts):
        slots.append(page * P + f + torch.arange(n))
        page += -(-(n + f) // P)
    slots = torch.cat(slots).to(DEV)
    T = len(slots)
    x = torch.randn((T, 2 * Hk, D), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).half()
    a = torch.zeros((page, Hk, P * (D + 8)), dtype=torch.uint8, device=DEV)
    b = a.clone()
    tq2.tq2_kv4_store(a, x[:, :Hk], x[:, Hk:], slots)
    order = torch.randperm(T, device=DEV)
    tq2.tq2_kv4_store(b, x[order, :Hk], x[order, Hk:], slots[order])
    assert torch.equal(a, b)


# ---- the binding's short way ----

def test_short_way_is_the_long_way(tq2, monkeypatch):
    def all_calls():
        s = layer_inputs(3)
        set_place(s, 5)
        Hq, Hk = s["Hq"], s["Hk"]
        q, k = tq2.tq2_qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hk], s["pos"], s["inv"], q_out=s["q"], k_out=s["k"])
        s["v"].copy_(s["qkv"][:, Hq + Hk:])
        tq2.tq2_kv4_store(s["cache"], k, s["v"], s["slots"])
        lk, lv = tq2.tq2_kv4_load(s["cache"], s["slots"], s["D"], k_out=torch.empty_like(k), v_out=torch.empty_like(s["v"]))
        lse = torch.empty((s["B"], Hq), device=DEV)
        out = tq2.tq2_kv4_attn(q, s["cache"], s["table"], s["ctx"], out=s["out"], ws=s["ws"], lse=lse, scale=0.2)
        torch.cuda.synchronize()
        return q, k, s["cache"], lk, lv, out, lse

    calls = []

    class Count:
        def __getattr__(self, name):
            def f(*a):
                status = getattr(real, name)(*a)
                calls.append((name, status))
                return status
            return f

    class Never:
        def __getattr__(self, name):
            return lambda *a: None

    real = tq2._tq2call
    monkeypatch.setattr(tq2, "_tq2call", Count())
    short = all_calls()
    assert calls == [("qk_norm_rope", 0), ("kv4_store", 0), ("kv4_load", 0), ("kv4_attn", 0)]
    monkeypatch.setattr(tq2, "_tq2call", Never())
    assert all(torch.equal(a, b) for a, b in zip(short, all_calls()))


def test_short_way_refuses_as_the_long_way(tq2):
    s = layer_inputs(4)
    q, k, v, out, Hq = s["q"].zero_(), s["k"].zero_(), s["v"].zero_(), s["out"], s["Hq"]
    attn = lambda **kw: tq2.tq2_kv4_attn(*[kw.pop(n, d) for n, d in (("q", q), ("cache", s["cache"]), ("table", s["table"]),
                                                                    ("ctx", s["ctx"]))], out=kw.pop("out", out), **kw)
    for match, kw in [("q must have dtype", dict(q=q.float())), ("cache must have dtype", dict(cache=s["cache"].to(torch.int8))),
                      ("table must be", dict(table=s["table"].long())), ("ctx_len must hold", dict(ctx=s["ctx"][:2])),
                      ("device tensor", dict(ctx=s["ctx"].cpu())), ("out must have dtype", dict(out=out.float())),
                      ("out must hold", dict(out=out[:2])), ("lse must have dtype", dict(lse=torch.zeros((3, Hq), device=DEV).half())),
                      ("needs max_q", dict(q_start=torch.zeros(4, dtype=torch.int32, device=DEV))), ("not max_q tokens", dict(max_q=2))]:
        with pytest.raises(ValueError, match=match):
            attn(**kw)
    with pytest.raises(tq2.Tq2Error):
        attn(window=-1)
    with pytest.raises(tq2.Tq2Error):
        attn(scale=float("nan"))
    with pytest.raises(ValueError, match="ws must hold"):
        wide = torch.zeros((3, 64), dtype=torch.int32, device=DEV)
        attn(table=wide, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(tq2.Tq2Error):
        tq2.tq2_qk_norm_rope(q, k, s["pos"], s["inv"], q_out=q, k_out=k)       # over its input
    with pytest.raises(ValueError, match="q_out must hold"):
        tq2.tq2_qk_norm_rope(q, k, s["pos"], s["inv"], q_out=out[:1], k_out=torch.empty_like(k))
    with pytest.raises(ValueError, match="slots must have dtype"):
        tq2.tq2_kv4_store(s["cache"], k, v, s["slots"].int())
    with pytest.raises(ValueError, match="k_out must hold"):
        tq2.tq2_kv4_load(s["cache"], s["slots"], s["D"], k_out=k[:1], v_out=v)


# ---- graphs of the split paths ----

@pytest.mark.parametrize("S,G", [(1, 16), (40, 4)])
def test_split_attention_in_a_graph(tq2, S, G):
    """Replays with other lengths, tables and queries equal eager calls."""
    B, Hk, D, P, width = 3, 2, 64, 32, 40
    cache, g = filled(9, 130, Hk, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    s = dict(q=torch.zeros((B * S, Hk * G, D), dtype=F16, device=DEV), table=torch.zeros((B, width), dtype=torch.int32, device=DEV),
             ctx=torch.ones(B, dtype=torch.int32, device=DEV), start=torch.zeros(B + 1, dtype=torch.int32, device=DEV),
             out=torch.zeros((B * S, Hk * G, D), dtype=F16, device=DEV), lse=torch.zeros((B * S, Hk * G), device=DEV))
    ws = [torch.full((tq2.tq2_kv4_attn_workspace_bytes(B * S, Hk * G, Hk, D, P, width, B, S),), 0xff, dtype=torch.uint8, device=DEV)
          for _ in range(2)]
    assert ws[0].numel() > 0
    call = lambda w, **kw: tq2.tq2_kv4_attn(s["q"], c, s["table"], s["ctx"], q_start=s["start"], max_q=S, ws=w, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws[0], out=s["out"], lse=s["lse"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws[0], out=s["out"], lse=s["lse"])
    for it in range(5):
        n = [S, int(g.integers(0, S + 1)), int(g.integers(1, S + 1))]
        s["q"].copy_(torch.from_numpy(g.standard_normal(s["q"].shape)))
        s["table"].copy_(torch.from_numpy(g.integers(0, 130, (B, width))))
        s["ctx"].copy_(torch.tensor([int(g.integers(S, width * P + 1)) for _ in range(B)]))
        s["start"].copy_(torch.tensor([0, n[0], n[0] + n[1], sum(n)]))
        s["out"].fill_(7)
        s["lse"].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        lse = torch.full_like(s["lse"], 7)
        out = call(ws[1], out=torch.full_like(s["out"], 7), lse=lse)
        torch.cuda.synchronize()
        assert torch.equal(out, s["out"]) and torch.equal(lse, s["lse"]), it
        assert bool((out[sum(n):] == 7).all())
