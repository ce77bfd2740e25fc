"""The attention half of a decode step on the GPU against the 64-bit oracles
of oracle/attention.py: head norms and rotation, the 4-bit cache written and
read back, and the attention over it."""
import numpy as np
import pytest

from oracle import attention as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def f64(t):
    return t.double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---- norms and rotation ----

def check_rope(tq2, T, Hq, Hk, D, rot, inter, norm, src, dst, start, seed, strided=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hk + 1, D), generator=g).to(src)
    x[:, :, 0] *= 8
    xd = x.to(DEV)
    q, k = (xd[:, :Hq], xd[:, Hq:Hq + Hk]) if strided else (xd[:, :Hq].contiguous(), xd[:, Hq:Hq + Hk].contiguous())
    pos = (start + torch.arange(T, dtype=torch.int64) * 3 % 1000).to(torch.int32)
    inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
    w = [(1 + 0.3 * torch.randn(D, generator=g)) for _ in range(2)] if norm else [None, None]
    got = tq2.tq2_qk_norm_rope(q, k, pos.to(DEV), inv.to(DEV), *[v if v is None else v.to(DEV) for v in w], eps=1e-5,
                               interleaved=inter, out_dtype=dst)
    torch.cuda.synchronize()
    for y, x0, wt in ((got[0], x[:, :Hq], w[0]), (got[1], x[:, Hq:Hq + Hk], w[1])):
        assert y.dtype == dst and y.is_contiguous()
        want, mag = ref.norm_rope(f64(x0), None if wt is None else wt.numpy(), np.float32(1e-5), pos.numpy(), inv.numpy(), inter)
        # 24 fp32 roundings: 13 in the norm (a sum of squares over 8 + 6 steps,
        # a square root, a quotient, two products), 4 in an angle's sine, the
        # products and their sum; then the output's own, which near zero is a step of binary16
        tol = 24 * 2.0 ** -24 * mag + half_step(dst) * np.abs(want) + (ref.F16_STEP if dst == F16 else 0)
        assert np.all(np.abs(f64(y) - want) <= tol), float((np.abs(f64(y) - want) / tol).max())


@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (64, 64), (96, 96), (80, 16), (256, 128), (16, 16), (512, 48), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_head_sizes(tq2, D, rot, inter):
    check_rope(tq2, 5, 3, 2, D, rot, inter, True, F32, F32, 900, D + rot)


@pytest.mark.parametrize("src", [F16, BF16, F32])
@pytest.mark.parametrize("dst", [F16, BF16, F32])
def test_rope_types(tq2, src, dst):
    check_rope(tq2, 7, 4, 1, 128, 128, False, True, src, dst, 0, 3)
    check_rope(tq2, 7, 4, 1, 128, 128, True, False, src, dst, 1000000, 4, strided=False)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 32, 2), (1, 1, 1), (33, 17, 5), (2048, 7, 1), (1500, 32, 2)])
def test_rope_token_counts(tq2, T, Hq, Hk):
    check_rope(tq2, T, Hq, Hk, 64, 64, False, True, F16, F16, 2147482000, T)


def test_rope_queries_or_keys_alone(tq2):
    x = torch.randn((6, 3, 128), device=DEV)
    pos, inv = torch.arange(6, dtype=torch.int32, device=DEV), torch.rand(64, device=DEV)
    none = x[:, :0]
    a, b = tq2.tq2_qk_norm_rope(x, x, pos, inv)
    c, d = tq2.tq2_qk_norm_rope(x, none, pos, inv)
    e, f = tq2.tq2_qk_norm_rope(none, x, pos, inv)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, f) and d.numel() == 0 and e.numel() == 0
    a, b = tq2.tq2_qk_norm_rope(x[:0], x[:0], pos[:0], inv)
    assert a.shape == (0, 3, 128)


def test_rope_zero_head(tq2):
    x = torch.zeros((2, 2, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    pos, inv = torch.arange(2, dtype=torch.int32, device=DEV), torch.rand(32, device=DEV)
    a, _ = tq2.tq2_qk_norm_rope(x, x, pos, inv, w, w)
    assert torch.equal(a, x)


# ---- the cache ----

def heads_of(g, T, H, D, dtype):
    x = torch.randn((T, H, D), generator=g) * torch.exp(torch.randn((1, H, D), generator=g))
    x[:, :, 3] *= 10
    return x.to(dtype)


def check_cache(tq2, T, Hk, D, P, src, slots, pages, seed):
    g = torch.Generator().manual_seed(seed)
    x = heads_of(g, T, 2 * Hk, D, src)
    if T > 2:
        x[1] = 0.375                      # no spread: the middle alone
        x[2, :, 1:] = x[2, :, :1]
    xd = x.to(DEV)
    want = ref.Cache(pages, Hk, P, D, fill=0xa5)
    cache = torch.from_numpy(want.bytes.copy()).to(DEV)
    sd = torch.tensor(slots, dtype=torch.int64, device=DEV)
    tq2.tq2_kv4_store(cache, xd[:, :Hk], xd[:, Hk:], sd)
    want.store(f64(x[:, :Hk]).astype(np.float32), f64(x[:, Hk:]).astype(np.float32), slots)
    torch.cuda.synchronize()
    assert np.array_equal(cache.cpu().numpy(), want.bytes)  # bit for bit, other slots untouched
    for dst in (F16, BF16, F32):
        k, v = tq2.tq2_kv4_load(cache, sd, D, dtype=dst)
        torch.cuda.synchronize()
        for y, x0 in ((k, x[:, :Hk]), (v, x[:, Hk:])):
            values = ref.held(*ref.quantize(f64(x0).astype(np.float32)))
            values[[not 0 <= s < pages * P for s in slots]] = 0
            exact = torch.from_numpy(values).float().to(dst)  # the fp32 value, rounded once more
            assert torch.equal(y.cpu(), exact)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("src", [F16, BF16, F32])
def test_cache_bits(tq2, D, src):
    g = np.random.default_rng(D)
    check_cache(tq2, 45, 3, D, 32, src, list(g.permutation(4 * 32)[:45]), 4, D)


@pytest.mark.parametrize("T,first,P", [(1, 0, 32), (1, 63, 64), (8, 8, 32), (33, 5, 32), (64, 32, 64), (100, 27, 128), (70, 64, 4096)])
def test_cache_runs(tq2, T, first, P):
    check_cache(tq2, T, 2, 128, P, F16, list(range(first, first + T)), 1 + (first + T) // P, T)
    check_cache(tq2, T, 1, 64, P, F32, list(range(first, first + T)), 1 + (first + T) // P, T + 1)


def test_cache_slots_without_a_page(tq2):
    check_cache(tq2, 12, 2, 64, 32, F16, [-1, 5, 96, 40, -32, 7, 1 << 40, 95, 0, -(1 << 62), 31, 64], 3, 1)
    check_cache(tq2, 16, 1, 128, 32, BF16, [8, 9, 10, 11, 12, 13, 14, 96] + list(range(90, 98)), 3, 2)


def test_cache_nothing_to_store(tq2):
    cache = torch.full((2, 1, 32 * 72), 7, dtype=torch.uint8, device=DEV)
    x = torch.zeros((0, 1, 64), device=DEV)
    slots = torch.zeros(0, dtype=torch.int64, device=DEV)
    tq2.tq2_kv4_store(cache, x, x, slots)
    k, v = tq2.tq2_kv4_load(cache, slots, 64)
    assert bool((cache == 7).all()) and k.shape == v.shape == (0, 1, 64)


def test_cache_halves_and_borders(tq2):
    """Values on the borders between codes: ties go to the even code."""
    D = 64
    base = torch.zeros((1, 1, D))
    base[0, 0, :16] = torch.arange(16) - 7.5            # s = 1, z = 0: code d stands for d - 7.5
    base[0, 0, 16:31] = torch.arange(15) - 7.0          # borders
    base[0, 0, 31:46] = torch.nextafter(torch.arange(15) - 7.0, torch.tensor(100.0))
    base[0, 0, 46:61] = torch.nextafter(torch.arange(15) - 7.0, torch.tensor(-100.0))
    want = ref.Cache(1, 1, 32, D)
    want.store(base.numpy(), base.numpy(), [9])
    cache = torch.zeros((1, 1, 32 * (D + 8)), dtype=torch.uint8, device=DEV)
    tq2.tq2_kv4_store(cache, base.to(DEV), base.to(DEV), torch.tensor([9], device=DEV))
    assert np.array_equal(cache.cpu().numpy(), want.bytes)


# ---- attention ----

def filled(seed, pages, Hk, P, D, kscale=1.0, vscale=1.0):
    """A cache of random tokens in every slot."""
    g = np.random.default_rng(seed)
    cache = ref.Cache(pages, Hk, P, D)
    half = P * D // 2
    cache.bytes[..., :2 * half] = g.integers(0, 256, (pages, Hk, 2 * half))
    pairs = np.empty((pages, Hk, 2, P, 2), np.float16)
    pairs[..., 0] = np.exp(0.3 * g.standard_normal((pages, Hk, 2, P))) * 0.3
    pairs[..., 1] = 0.4 * g.standard_normal((pages, Hk, 2, P))
    pairs[:, :, 0] *= np.float16(kscale)
    pairs[:, :, 1] *= np.float16(vscale)
    cache.bytes[..., 2 * half:] = pairs.reshape(pages, Hk, -1).view(np.uint8)
    return cache, g


def check_attn(tq2, ns, ctx, Hk, G, D, P, dtype, window=0, scale=None, seed=0, cache=None, table=None, q=None,
               ragged=True, strided=False, want_lse=True):
    B, T = len(ns), sum(ns)
    width = max(1, max(-(-c // P) for c in ctx))
    pages = sum(-(-c // P) for c in ctx) + 1
    if cache is None:
        cache, g = filled(seed, pages, Hk, P, D)
    else:
        g = np.random.default_rng(seed)
    if table is None:
        order, table, used = g.permutation(cache.pages), np.full((B, width), -1, np.int32), 0
        for b in range(B):
            need = -(-ctx[b] // P)
            table[b, :need] = order[used:used + need]
            used += need
    if q is None:
        q = torch.from_numpy(g.standard_normal((T, Hk * G, D)) * 0.8).to(dtype)
    start = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    sc = D ** -0.5 if scale is None else scale
    qd = q.to(DEV)
    if strided:
        wide = torch.zeros((T, Hk * G + 3, D + 8), dtype=dtype, device=DEV)
        wide[:, 1:1 + Hk * G, :D] = qd
        qd = wide[:, 1:1 + Hk * G, :D]
    out = torch.full((T, Hk * G, D), float("nan"), dtype=dtype, device=DEV)
    lse = torch.full((T, Hk * G), float("nan"), device=DEV) if want_lse else None
    got = tq2.tq2_kv4_attn(qd, torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                           torch.tensor(ctx, dtype=torch.int32, device=DEV),
                           q_start=torch.from_numpy(start).to(DEV) if ragged else None,
                           max_q=max(ns) if ragged else None, scale=scale, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    want, wl, tol, ltol = ref.attention(f64(q), cache, table, ctx, start, np.float32(sc).astype(np.float64), window,
                                        torch.finfo(dtype).eps)
    y = f64(out)
    assert np.all(np.isfinite(y))
    worst = np.abs(y - want) / np.maximum(tol, 1e-300)
    assert np.all(np.abs(y - want) <= tol), (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))
    if want_lse:
        l = f64(lse)
        assert np.array_equal(np.isinf(l), np.isinf(wl))
        f = np.isfinite(wl)
        assert np.all(np.abs(l[f] - wl[f]) <= ltol[f])
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attn_one_token(tq2, D, dtype):
    check_attn(tq2, [1, 1, 1], [77, 1, 300], 2, 4, D, 32, dtype, seed=D)


@pytest.mark.parametrize("ctx", [1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 513, 1000])
def test_attn_lengths(tq2, ctx):
    check_attn(tq2, [1], [ctx], 1, 16, 128, 64, F16, seed=ctx, ragged=False)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 12, 15, 16, 17, 24, 32, 33])
def test_attn_groups(tq2, G):
    check_attn(tq2, [1, 1], [90, 41], 3, G, 64, 32, F16, seed=G)


@pytest.mark.parametrize("P", [32, 64, 256, 4096])
def test_attn_pages(tq2, P):
    check_attn(tq2, [1, 2], [333, 40], 1, 8, 128, P, BF16, seed=P)


@pytest.mark.parametrize("ns,ctx", [([5], [5]), ([3], [40]), ([17], [17]), ([1, 4, 2], [9, 100, 64]), ([33, 1], [70, 1]),
                                    ([64], [131])])
@pytest.mark.parametrize("G", [1, 7, 16])
def test_attn_many_tokens(tq2, ns, ctx, G):
    check_attn(tq2, ns, ctx, 2, G, 64, 32, F16, seed=sum(ns) + G)


@pytest.mark.parametrize("D", [128, 256])
def test_attn_chunk(tq2, D):
    check_attn(tq2, [40, 23], [100, 23], 1, 5, D, 64, BF16, seed=D)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 2000000000])
def test_attn_window(tq2, window):
    check_attn(tq2, [1, 9, 1], [200, 140, 20], 2, 4, 64, 32, F16, window=window, seed=window % 97)


def test_attn_split_rows(tq2):
    """Long single sequences are split over workgroups and joined."""
    check_attn(tq2, [1], [5000], 1, 2, 64, 32, F16, seed=5, ragged=False)
    check_attn(tq2, [2], [2500], 1, 16, 128, 64, BF16, seed=6)
    check_attn(tq2, [1, 1], [3100, 30], 1, 1, 256, 64, F16, window=1111, seed=7)


def test_attn_rows_that_see_nothing(tq2):
    check_attn(tq2, [1, 1, 1], [0, 50, 0], 2, 3, 64, 32, F16, seed=1)
    check_attn(tq2, [4, 2], [2, 1], 1, 4, 128, 32, BF16, seed=2)  # fewer cached tokens than new ones
    check_attn(tq2, [0, 3, 0, 1], [10, 30, 0, 5], 1, 4, 64, 32, F16, seed=3)  # sequences without new tokens


def test_attn_strided_queries_without_lse(tq2):
    check_attn(tq2, [2, 1], [60, 9], 2, 4, 64, 32, F16, seed=4, strided=True, want_lse=False)


def test_attn_pages_that_are_not_there(tq2):
    """Table entries that name no page stand for tokens that no row sees."""
    cache, g = filled(3, 6, 2, 32, 64)
    table = np.array([[2, -1, 4, 6, 1], [-2147483648, 2147483647, 99, -1, 6]], np.int32)
    check_attn(tq2, [2, 1], [150, 140], 2, 4, 64, 32, F16, cache=cache, table=table, seed=9)


@pytest.mark.parametrize("bad", [0x7e00, 0x7c00, 0xfc00, 0xffff, 0x7bff])
def test_attn_unseen_places_hold_anything(tq2, bad):
    """Pairs of NaN, infinity or the largest value behind a sequence's end, in
    front of its window and at later new tokens do not act on a row."""
    P, D, Hk = 32, 64, 1
    cache, g = filled(4, 4, Hk, P, D)
    pairs = cache.bytes[..., P * D:].view(np.uint16).reshape(4, Hk, 2, P, 2)
    clean = cache.bytes.copy()
    table = np.array([[0, 1, 2, 3]], np.int32)
    q = torch.from_numpy(g.standard_normal((1, 16, D))).to(F16)
    for page, t in [(2, range(7, 32)), (3, range(32)), (0, range(32)), (1, range(3))]:
        pairs[page, :, :, list(t)] = bad
    # one token that sees places 35 .. 70
    out, lse = check_attn(tq2, [1], [71], Hk, 16, D, P, F16, window=36, cache=cache, table=table, q=q, seed=1)
    cache.bytes[:] = clean
    out2, lse2 = check_attn(tq2, [1], [71], Hk, 16, D, P, F16, window=36, cache=cache, table=table, q=q, seed=1)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    # the last new token's own place is bad: the earlier ones do not see it
    q = torch.from_numpy(g.standard_normal((3, 16, D))).to(F16)
    state = {}
    for name in ("clean", "bad"):
        if name == "bad":
            pairs[2, :, :, 6] = bad
        y = tq2.tq2_kv4_attn(q.to(DEV), torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                             torch.tensor([71], dtype=torch.int32, device=DEV))
        state[name] = y.cpu()
    assert torch.equal(state["clean"][:2], state["bad"][:2])


@pytest.mark.parametrize("kscale,vscale,scale", [(1, 1, 3.0), (40, 1, None), (1, 3000, None), (1, 1e-4, None), (1, 1, 0.0),
                                                 (1, 1, -0.2), (1e-3, 100, 1.0)])
def test_attn_sizes_of_values(tq2, kscale, vscale, scale):
    cache, _ = filled(8, 12, 1, 32, 64, kscale, vscale)
    check_attn(tq2, [1, 6], [200, 150], 1, 8, 64, 32, F16, scale=scale, cache=cache, seed=8)


def test_attn_value_scales_of_all_sizes(tq2):
    """Scales from binary16's least to large ones in one row, and none at all."""
    cache, g = filled(11, 10, 1, 32, 64)
    pairs = cache.bytes[..., 32 * 64:].view(np.float16).reshape(10, 1, 2, 32, 2)
    pairs[:, :, 1, :, 0] = np.exp2(g.uniform(-24, 8, (10, 1, 32))).astype(np.float16)
    check_attn(tq2, [1], [310], 1, 8, 64, 32, F16, cache=cache, seed=2)
    pairs[..., 0] = 0                      # every channel of a token alike
    check_attn(tq2, [1], [310], 1, 8, 64, 32, F16, cache=cache, seed=2)


def test_attn_zero_and_small_queries(tq2):
    for size in (0.0, 2.0 ** -24, 1e-6, 300.0):
        g = np.random.default_rng(5)
        q = torch.from_numpy(g.standard_normal((2, 8, 64)) * size).to(F16)
        check_attn(tq2, [2], [100], 1, 8, 64, 32, F16, q=q, seed=5, scale=0.1 / max(size, 0.1))
    q = torch.zeros((1, 8, 64), dtype=BF16)
    q[0, :, 0], q[0, :, 1] = 1e30, 1e-30   # far apart in one row
    check_attn(tq2, [1], [100], 1, 8, 64, 32, BF16, q=q, seed=5, scale=1e-30)


def test_attn_rising_scores(tq2):
    """The largest score comes last, tile after tile: every reference moves."""
    cache, g = filled(12, 20, 1, 32, 64)
    pairs = cache.bytes[..., 32 * 64:].view(np.float16).reshape(20, 1, 2, 32, 2)
    pairs[:, :, 0, :, 1] = (np.arange(640).reshape(20, 1, 32) / 40).astype(np.float16)
    q = torch.full((1, 4, 64), 1.0, dtype=F16)
    q[0, 1] = -1.0                         # and falling
    table = np.arange(20, dtype=np.int32)[None]
    check_attn(tq2, [1], [640], 1, 4, 64, 32, F16, cache=cache, table=table, q=q, scale=0.5, seed=3)


def test_attn_lengths_outside_the_table_are_held(tq2):
    cache, g = filled(13, 3, 1, 32, 64)
    table = np.array([[2, 0]], np.int32)
    q = torch.from_numpy(g.standard_normal((1, 4, 64))).to(F16).to(DEV)
    c, t = torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV)
    call = lambda n: tq2.tq2_kv4_attn(q, c, t, torch.tensor([n], dtype=torch.int32, device=DEV))
    assert torch.equal(call(64), call(65)) and torch.equal(call(64), call(2 ** 31 - 1))
    assert bool((call(-5) == 0).all()) and torch.equal(call(-5), call(0))


def test_attn_rows_outside_the_sequences(tq2):
    """q_start that runs past T or backwards stays inside q and out."""
    cache, g = filled(14, 4, 1, 32, 64)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    c, ctx = torch.from_numpy(cache.bytes).to(DEV), torch.tensor([40, 50], dtype=torch.int32, device=DEV)
    q = torch.from_numpy(g.standard_normal((6, 4, 64))).to(F16).to(DEV)
    for start in ([0, 2, 100], [-7, 3, 6], [4, 1, 5], [9, 9, 9], [-5, -2, 2 ** 31 - 1]):
        out = torch.full((6, 4, 64), 9.0, dtype=F16, device=DEV)
        tq2.tq2_kv4_attn(q, c, table, ctx, q_start=torch.tensor(start, dtype=torch.int32, device=DEV), max_q=3, out=out)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(out).all())


def test_attn_same_bits_twice_and_by_batch(tq2):
    """Deterministic, and a row does not depend on the other sequences' values."""
    cache, g = filled(15, 60, 2, 32, 128)
    c = torch.from_numpy(cache.bytes).to(DEV)
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(2, 30)
    ctx = torch.tensor([900, 500], dtype=torch.int32, device=DEV)
    q = torch.from_numpy(g.standard_normal((2, 8, 128))).to(F16).to(DEV)
    a = tq2.tq2_kv4_attn(q, c, table, ctx)
    assert torch.equal(a, tq2.tq2_kv4_attn(q, c, table, ctx))
    q2 = q.clone()
    q2[1] *= 3
    assert torch.equal(a[0], tq2.tq2_kv4_attn(q2, c, table, ctx)[0])


# ---- streams and graphs ----

def layer_inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    B, Hq, Hk, D, P, pages = 3, 8, 2, 64, 32, 24
    qkv = torch.randn((B, Hq + 2 * Hk, D), generator=g).to(DEV)
    return dict(B=B, Hq=Hq, Hk=Hk, D=D, P=P, pages=pages, qkv=qkv,
                cache=torch.zeros((pages, Hk, P * (D + 8)), dtype=torch.uint8, device=DEV),
                table=torch.arange(pages, dtype=torch.int32, device=DEV).view(B, 8),
                inv=(10000.0 ** (-torch.arange(0, D, 2).double() / D)).float().to(DEV),
                pos=torch.zeros(B, dtype=torch.int32, device=DEV), ctx=torch.zeros(B, dtype=torch.int32, device=DEV),
                slots=torch.zeros(B, dtype=torch.int64, device=DEV),
                q=torch.empty((B, Hq, D), dtype=F16, device=DEV), k=torch.empty((B, Hk, D), dtype=F16, device=DEV),
                v=torch.empty((B, Hk, D), dtype=F16, device=DEV),
                out=torch.empty((B, Hq, D), dtype=F16, device=DEV),
                ws=torch.empty(8 << 20, dtype=torch.uint8, device=DEV))


def layer_step(tq2, s, stream=None):
    Hq, Hk = s["Hq"], s["Hk"]
    tq2.tq2_qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hk], s["pos"], s["inv"], q_out=s["q"], k_out=s["k"], stream=stream)
    s["v"].copy_(s["qkv"][:, Hq + Hk:])
    tq2.tq2_kv4_store(s["cache"], s["k"], s["v"], s["slots"], stream=stream)
    return tq2.tq2_kv4_attn(s["q"], s["cache"], s["table"], s["ctx"], out=s["out"], ws=s["ws"], stream=stream)


def set_place(s, at):
    s["pos"].fill_(at)
    s["ctx"].fill_(at + 1)
    s["slots"].copy_(torch.arange(s["B"], device=DEV) * 8 * s["P"] + at)


def test_step_in_a_graph(tq2):
    """A captured step replayed at moving places equals the eager one each time."""
    s, e = layer_inputs(), layer_inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_step(tq2, s)
    torch.cuda.current_stream().wait_stream(side)
    s["cache"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(tq2, s)
    for at in range(5):
        for x in (s, e):
            x["qkv"].copy_(torch.randn(x["qkv"].shape, generator=torch.Generator().manual_seed(at)))
            set_place(x, at)
        graph.replay()
        torch.cuda.synchronize()
        layer_step(tq2, e)
        torch.cuda.synchronize()
        assert torch.equal(s["out"], e["out"]) and torch.equal(s["cache"], e["cache"]), at


def test_step_on_a_side_stream(tq2):
    s, e = layer_inputs(1), layer_inputs(1)
    set_place(s, 3)
    set_place(e, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer_step(tq2, s)
    layer_step(tq2, e)
    torch.cuda.synchronize()
    assert torch.equal(s["out"], e["out"])
