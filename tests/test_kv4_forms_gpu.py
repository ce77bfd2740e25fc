"""Every form of the attention at the precision that it promises, with the form
asserted: the form for many rows with one tile of 16 rows a wave, short and
split; rows that are many by name but few by the rule; sums over long texts."""
import numpy as np
import pytest

from oracle import attention as ref
from tests import kv4_forms as forms
from tests.test_kv4_gpu import f64, filled
from tests.test_kv4_long_gpu import dequantized

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def batch(seed, ns, ctx, Hk, G, D, P, width, dtype):
    need = [-(-c // P) for c in ctx]
    cache, g = filled(seed, sum(need) + 1, Hk, P, D)
    order, table, used = g.permutation(cache.pages), np.full((len(ns), max(width, max(need))), -1, np.int32), 0
    for b in range(len(ns)):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
    q = torch.from_numpy(g.standard_normal((sum(ns), Hk * G, D)) * 0.8).to(dtype)
    return cache, table, q, np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def run(tq2, cache, table, q, start, ctx, max_q, window):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), float("nan"), dtype=q.dtype, device=DEV)
    lse = torch.full((T, Hq), float("nan"), device=DEV)
    tq2.tq2_kv4_attn(q.to(DEV), torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                     torch.tensor(ctx, dtype=torch.int32, device=DEV), q_start=torch.from_numpy(start).to(DEV), max_q=max_q,
                     window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def check(tq2, ns, ctx, Hk, G, D, P, width, dtype, max_q, window=0, seed=0):
    """Against the oracle, within what the form that the call takes keeps; its plan."""
    cache, table, q, start = batch(seed, ns, ctx, Hk, G, D, P, width, dtype)
    plan = forms.plan(Hk * G, Hk, D, P, table.shape[1], len(ns), max_q, window)
    out, lse = run(tq2, cache, table, q, start, ctx, max_q, window)
    want, wl, tol, ltol = ref.attention(f64(q), cache, table, ctx, start, np.float64(np.float32(D ** -0.5)), window,
                                        torch.finfo(dtype).eps, kept=forms.kept(plan.few))
    worst = np.abs(f64(out) - want) / np.maximum(tol, 1e-300)
    assert np.all(np.abs(f64(out) - want) <= tol), (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))
    l, f = f64(lse), np.isfinite(wl)
    assert np.array_equal(np.isinf(l), ~f) and np.all(np.abs(l[f] - wl[f]) <= ltol[f])
    return plan


# name, sequences, most new tokens, key heads, query heads of each, table, window, dealt from a list
MANY_ONE = [
    ("batched drafts, dealt", 33, 8, 1, 16, 300, 0, True),
    ("batched drafts, dealt, a window", 33, 8, 1, 16, 300, 1200, True),
    ("several key heads, dealt", 12, 30, 3, 5, 300, 0, True),
    ("batched drafts, short texts", 260, 8, 1, 16, 32, 0, False),
    ("batched drafts, a short window", 260, 8, 1, 16, 150, 700, False),
]


@pytest.mark.parametrize("case", MANY_ONE, ids=[c[0] for c in MANY_ONE])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_rows_one_tile_a_wave(tq2, case, D, dtype):
    """65 to 256 rows a key head.  Some sequences are long: parts of an even and
    an odd number of tiles, joined; most have few new tokens or none."""
    name, B, mq, Hk, G, width, window, dealt = case
    g = np.random.default_rng(B + D)
    ns = [int(n) for n in g.integers(0, 3, B)]
    ctx = [max(n, int(c)) for n, c in zip(ns, np.exp(g.uniform(0, 5.3, B)))]
    ns[1], ns[B // 2], ns[B - 1] = mq, mq - 1, 1
    if dealt:
        ctx[1], ctx[B // 2], ctx[B - 1] = 1500, 1263, 800
    else:
        ctx[1], ctx[B // 2], ctx[B - 1] = 1000, 933, 33
    plan = check(tq2, ns, ctx, Hk, G, D, 32, width, dtype, mq, window=window, seed=D)
    assert not plan.few and plan.mt == 1 and plan.list == dealt
    if dealt:
        assert plan.least < 1263 // 32 // 2      # the long ones are split


@pytest.mark.parametrize("D,dtype", [(64, F16), (128, BF16), (256, F16)])
def test_rows_that_are_few_by_the_rule(tq2, D, dtype):
    """Prompts of a few hundred rows are few by the rule, and keep 22 bits."""
    for ns, ctx, G, window in (([40, 9], [700, 300], 4, 0), ([21, 0, 9], [1300, 40, 1111], 5, 0), ([70], [1200], 1, 1000),
                               ([200], [150], 2, 0), ([130, 60], [300, 200], 16, 0)):
        assert check(tq2, ns, ctx, 1, G, D, 32, 1, dtype, max(ns), window=window, seed=D).few


@pytest.mark.parametrize("G", [1, 7, 16, 33])
def test_single_tokens_and_drafts_keep_22_bits(tq2, G):
    assert check(tq2, [1, 1, 1], [77, 1, 1800], 2, G, 64, 32, 1, F16, 1, seed=G).few
    if G <= 16:
        assert check(tq2, [5, 3, 1], [1500, 40, 700], 2, G, 128, 64, 1, BF16, 5, seed=G).few


@pytest.mark.parametrize("ns,ctx,Hk,G,D,P,dtype,few", [
    ([10], [8000], 1, 16, 128, 64, F16, True), ([9], [4000], 2, 12, 256, 32, BF16, True), ([64], [4000], 1, 16, 64, 64, F16, True),
    ([1, 1], [30000, 70], 2, 16, 128, 64, F16, True), ([300], [5000], 1, 16, 128, 64, F16, True),
    ([300], [7500], 1, 16, 128, 64, F16, False),
    ([8] * 40, [7500] * 40, 1, 16, 64, 64, F16, False)])
def test_long_texts(tq2, ns, ctx, Hk, G, D, P, dtype, few):
    """64-bit products on the GPU; the bound of each term weighted by its probability."""
    cache, table, q, start = batch(3, ns, ctx, Hk, G, D, P, 1, dtype)
    assert forms.plan(Hk * G, Hk, D, P, table.shape[1], len(ns), max(ns)).few == few
    out, lse = run(tq2, cache, table, q, start, ctx, max(ns), 0)
    K, V, C = dequantized(cache)
    pairs = torch.from_numpy(cache.bytes[..., P * D:].copy()).view(F16).view(cache.pages, Hk, 2, P, 2).double().abs().to(DEV)
    eps, scale, kept = torch.finfo(dtype).eps, D ** -0.5, forms.kept(few)
    for b in range(len(ns)):
        if b > 2:
            break
        j = torch.arange(ctx[b], device=DEV)
        at = torch.from_numpy(table[b]).to(DEV).long()[j // P]
        rows = torch.arange(0, ns[b], max(1, ns[b] // 16), device=DEV)
        seen = j[None] <= (ctx[b] - ns[b] + rows)[:, None]
        for h in range(Hk):
            k, v, cen = (x[at, h, j % P].contiguous() for x in (K, V, C))
            kmag = float((7.5 * pairs[at, h, 0, j % P, 0] + pairs[at, h, 0, j % P, 1]).max())
            s = pairs[at, h, 1, j % P, 0]
            vmag = (15 * s + pairs[at, h, 1, j % P, 1])[:, None].contiguous()
            for g0 in range(0, G, 3):
                x0 = q[start[b]:start[b + 1], h * G + g0].to(DEV)[rows].double()
                x = torch.where(seen, x0 @ k.T.contiguous() * scale, -torch.inf)
                top = x.amax(-1, keepdim=True)
                p = torch.exp(x - top)
                total = p.sum(-1, keepdim=True)
                l, p = (top + torch.log(total))[:, 0], p / total
                o = p @ v
                n = seen.sum(-1, keepdim=True)
                score = 16 * 2.0 ** -24 * (kmag * x0.abs().sum(-1, keepdim=True) * scale + top.abs())
                sums = (n / 32 + 64) * 2.0 ** -24
                held16 = kept * (p @ cen) + n * ref.F16_STEP * 7.5 * (p * s).amax(-1, keepdim=True) / 2 ** 4
                tol = eps / 2 * o.abs() + ref.F16_STEP + held16 + 2 * score * (p @ v.abs() + o.abs()) + sums * (p @ vmag)
                got = out[start[b]:start[b + 1], h * G + g0][rows].double()
                assert bool(((got - o).abs() <= tol).all()), (b, h, g0, float(((got - o).abs() / tol).max()))
                got = lse[start[b]:start[b + 1], h * G + g0][rows].double()
                assert bool(((got - l).abs() <= (2 * score + sums)[:, 0] + 2.0 ** -22 * l.abs()).all())


@pytest.mark.parametrize("S,few,cut", [(1, True, 2.0 ** -15), (264, False, 2.0 ** -13)])
def test_no_channel_of_a_word_leans(tq2, S, few, cut):
    """Over 131000 tokens, where an output is far smaller than its terms, what the
    matrix cores cut off a subnormal code must not lean to one side in any of the
    four channels of a 16-bit unit.  Bound: what cutting left at the form's place
    of the codes (`cut`, of the outputs' size), and four deviations of the mean of
    the outputs' roundings (2^-12.2 of the size each)."""
    n, D, P, G = 131000, 128, 64, 16
    cache, g = filled(21, -(-n // P), 1, P, D)
    cache.bytes[..., P * D:].view(np.float16).reshape(-1, 1, 2, P, 2)[:, :, 1, :, 1] = 0
    q = torch.from_numpy(0.3 * g.standard_normal((S, G, D))).to(F16).to(DEV)
    table = torch.arange(cache.pages, dtype=torch.int32, device=DEV)[None]
    assert forms.plan(G, 1, D, P, cache.pages, 1, S).few == few
    out = tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), table, torch.tensor([n], dtype=torch.int32, device=DEV))
    K, V, _ = dequantized(cache)
    k, v = K.reshape(-1, D)[:n].contiguous(), V.reshape(-1, D)[:n].contiguous()
    off, size, rows = [], [], range(0, S, max(1, S // 16))
    for i in rows:
        c = n - S + 1 + i
        want = torch.softmax(q[i].double() @ k[:c].T.contiguous() * D ** -0.5, -1) @ v[:c].contiguous()
        off.append(out[i].double() - want)
        size.append(want.pow(2).mean())
    off, size = torch.stack(off), torch.stack(size).mean().sqrt()
    assert float(size) < 0.01
    lean = off.view(-1, D // 4, 4).mean((0, 1)).abs() / size
    assert float(lean.max()) <= cut + 4 * 2.0 ** -12.2 / (len(rows) * G * D / 4) ** 0.5, lean
