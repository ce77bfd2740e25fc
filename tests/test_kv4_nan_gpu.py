"""NaN in what a row sees: it shows in the row's output and log-sum-exp, and in
no other row's.  (What rows do not see is tested beside the rest of the
attention.)"""
import numpy as np
import pytest

from tests.test_kv4_gpu import filled

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16 = torch.float16


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


# one workgroup; parts joined by row; many rows alone; many rows in parts
FORMS = [(1, 1, 40, 2), (1, 1, 5000, 157), (2, 260, 300, 300), (1, 400, 9000, 300)]


@pytest.mark.parametrize("B,S,ctx,width", FORMS)
def test_a_query_of_nan(tq2, B, S, ctx, width):
    G, D, P = 16, 64, 32
    cache, g = filled(1, 300, 1, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    table = torch.from_numpy(g.integers(0, 300, (B, width)).astype(np.int32)).to(DEV)
    lens = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    q = torch.from_numpy(g.standard_normal((B * S, G, D))).to(F16).to(DEV)

    def run(x):
        lse = torch.zeros((B * S, G), device=DEV)
        return tq2.tq2_kv4_attn(x, c, table, lens, lse=lse), lse

    out, lse = run(q)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    bad = q.clone()
    bad[B * S // 2, 5, 7] = float("nan")
    out2, lse2 = run(bad)
    assert bool(out2[B * S // 2, 5].isnan().all()) and bool(lse2[B * S // 2, 5].isnan())
    out2[B * S // 2, 5], lse2[B * S // 2, 5] = out[B * S // 2, 5], lse[B * S // 2, 5]
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,S,ctx,width", FORMS)
def test_a_key_of_nan(tq2, B, S, ctx, width):
    """Seen by the last new token of a sequence alone, and by all of them."""
    G, D, P = 16, 64, 32
    cache, g = filled(2, 300, 1, P, D)
    pairs = cache.bytes[..., P * D:].view(np.uint16).reshape(300, 1, 2, P, 2)
    table = g.permutation(300)[:width].astype(np.int32)[None].repeat(B, 0)
    if ctx > 300 * P // 2:
        ctx = P * width - 5
    lens = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    q = torch.from_numpy(g.standard_normal((B * S, G, D))).to(F16).to(DEV)

    def run():
        lse = torch.zeros((B * S, G), device=DEV)
        out = tq2.tq2_kv4_attn(q, torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV), lens, lse=lse)
        return out.view(B, S, G, D), lse.view(B, S, G)

    out, lse = run()
    pairs[table[0, (ctx - 1) // P], 0, 0, (ctx - 1) % P] = 0x7e00
    out2, lse2 = run()
    assert bool(out2[:, -1].isnan().all()) and bool(lse2[:, -1].isnan().all())
    assert torch.equal(out[:, :-1], out2[:, :-1]) and torch.equal(lse[:, :-1], lse2[:, :-1])
    pairs[table[0, 0], 0, 0, 3] = 0x7e00
    out2, lse2 = run()
    assert bool(out2.isnan().all()) and bool(lse2.isnan().all())
