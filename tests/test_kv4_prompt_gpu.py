"""The form of the attention whose waves own rows (prompts), at sizes small
enough for the oracle: it is taken where the rows are more than 4096 in all and
the table is wide, whatever the lengths are."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_kv4_gpu import check_attn, filled

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def wide(tq2, ns, ctx, Hk, G, D, P, dtype, window=0, seed=0, spoil=None):
    """As check_attn, with a table of 300 tiles (100 if each key head has rows enough)."""
    B = len(ns)
    assert B * Hk * max(ns) * G > 4096 and B * Hk * max(ns) * G * 300 > 1 << 20
    need = [-(-c // P) for c in ctx]
    cache, g = filled(seed, sum(need) + 1, Hk, P, D)
    order, table, used = g.permutation(cache.pages), np.full((B, max(300 * 32 // P, max(need))), -1, np.int32), 0
    for b in range(B):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
    if spoil:
        spoil(table)
    return check_attn(tq2, ns, ctx, Hk, G, D, P, dtype, window=window, seed=seed, cache=cache, table=table)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_prompts_of_unequal_length(tq2, D, dtype):
    wide(tq2, [130, 9], [400, 40], 1, 16, D, 64, dtype, seed=D)


@pytest.mark.parametrize("ns,ctx,G,P", [([260], [260], 16, 32), ([131, 1, 0, 3], [131, 200, 9, 3], 8, 32), ([420, 100], [430, 100], 5, 64),
                                        ([140], [33], 33, 32), ([129], [1000], 32, 4096), ([4100], [150], 1, 32)])
def test_prompt_shapes(tq2, ns, ctx, G, P):
    wide(tq2, ns, ctx, 1, G, 64, P, F16, seed=G)


@pytest.mark.parametrize("window", [1, 33, 100])
def test_prompt_windows(tq2, window):
    wide(tq2, [140, 20], [300, 150], 1, 16, 64, 32, F16, window=window, seed=window)


def test_prompt_pages_that_are_not_there(tq2):
    def spoil(table):
        table[0, 2], table[0, 5], table[1, 0], table[1, 3] = -1, 2147483647, -2147483648, 99

    wide(tq2, [130, 60], [300, 200], 1, 16, 64, 32, F16, seed=3, spoil=spoil)


def test_prompts_of_several_key_heads(tq2):
    wide(tq2, [60, 33], [200, 33], 3, 12, 128, 64, BF16, seed=4)


@pytest.mark.parametrize("bad", [0x7e00, 0x7c00, 0xffff])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_unseen_places_hold_anything(tq2, bad, D):
    P, n, G, c = 32, 260, 16, 300
    cache, g = filled(6, 12, 1, P, D)
    pairs = cache.bytes[..., P * D:].view(np.uint16).reshape(12, 1, 2, P, 2)
    table = np.full((1, 300), -1, np.int32)
    table[0, :12] = np.arange(12)
    q = torch.from_numpy(g.standard_normal((n, G, D))).to(F16).to(DEV)
    run = lambda: tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                                   torch.tensor([c], dtype=torch.int32, device=DEV)).cpu()
    clean = run()
    assert bool(torch.isfinite(clean).all())
    for t in range(c, 12 * P):
        pairs[t // P, :, :, t % P] = bad
    assert torch.equal(run(), clean)
    for t in (c - 1, c - 40):                                    # a later new token's place
        pairs[t // P, :, :, t % P] = bad
        seen = n - (c - t)
        assert torch.equal(run()[:seen], clean[:seen])


def test_prompt_value_and_key_sizes(tq2):
    for kscale, vscale, seed in ((40, 1, 1), (1, 3000, 2), (1e-3, 1, 3)):
        P, D, ns, ctx = 32, 64, [260], [300]
        cache, g = filled(seed, 10, 1, P, D, kscale, vscale)
        table = np.full((1, 300), -1, np.int32)
        table[0, :10] = np.arange(10)
        check_attn(tq2, ns, ctx, 1, 16, D, P, F16, cache=cache, table=table, seed=seed)


def test_prompt_strided_queries(tq2):
    P, D = 32, 128
    cache, g = filled(9, 10, 1, P, D)
    table = np.full((1, 300), -1, np.int32)
    table[0, :10] = np.arange(10)
    check_attn(tq2, [260], [290], 1, 16, D, P, BF16, cache=cache, table=table, seed=9, strided=True, want_lse=False)


def test_prompt_in_a_graph(tq2):
    """Replays with other lengths and tables equal eager calls."""
    B, S, Hk, G, D, P, width = 2, 130, 1, 16, 64, 32, 300
    cache, g = filled(10, 40, Hk, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    new = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device=DEV)
    q, out, lse = new(B * S, G, D, dtype=F16), new(B * S, G, D, dtype=F16), new(B * S, G, dtype=torch.float32)
    table, ctx, start = new(B, width), new(B), new(B + 1)
    need = tq2.tq2_kv4_attn_workspace_bytes(B * S, G, Hk, D, P, width, B, S)
    assert need > 0
    ws = [torch.full((need,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]
    call = lambda w, o, l: tq2.tq2_kv4_attn(q, c, table, ctx, q_start=start, max_q=S, ws=w, out=o, lse=l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws[0], out, lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws[0], out, lse)
    for it in range(5):
        n = [S - 7 * it, int(g.integers(0, S + 1))]
        q.copy_(torch.from_numpy(g.standard_normal(q.shape)))
        table.copy_(torch.from_numpy(g.integers(0, 40, (B, width))))
        ctx.copy_(torch.tensor([int(g.integers(S, 9000)), int(g.integers(0, 500))]))
        start.copy_(torch.tensor([0, n[0], sum(n)]))
        out.fill_(7)
        lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        o, l = torch.full_like(out, 7), torch.full_like(lse, 7)
        call(ws[1], o, l)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse) and bool((o[sum(n):] == 7).all()), it
