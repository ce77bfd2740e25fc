"""Value scales that differ by far inside a row: what a probability times its
token's scale is held to goes by the products, not by the scales alone.  Against
the 64-bit oracle, with the bound that each form of the attention keeps (22
bits where rows are few, one rounding to binary16 where they are many)."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_kv4_gpu import f64, filled

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16
FEW, MANY = 2.0 ** -22, 2.0 ** -11


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def check(tq2, cache, table, q, ctx, kept, window=0, scale=0.125):
    T, Hq, D = q.shape
    out, lse = torch.empty((T, Hq, D), dtype=q.dtype, device=DEV), torch.empty((T, Hq), device=DEV)
    tq2.tq2_kv4_attn(q.to(DEV), torch.from_numpy(cache.bytes).to(DEV), torch.from_numpy(table).to(DEV),
                     torch.tensor([ctx], dtype=torch.int32, device=DEV), scale=scale, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    want, wl, tol, ltol = ref.attention(f64(q), cache, table, [ctx], [0, T], np.float64(np.float32(scale)), window,
                                        torch.finfo(q.dtype).eps, kept=kept)
    worst = np.abs(f64(out) - want) / tol
    assert np.all(worst <= 1), (float(worst.max()), np.unravel_index(worst.argmax(), worst.shape))
    assert np.all(np.abs(f64(lse) - wl) <= ltol)


def unequal(seed, D, tokens, small, large, at, below, P=32):
    """A cache of one key head whose value scales are near `small`, with middles
    of zero, and `large` at the tokens `at`, whose scores are about `below` less."""
    pages = -(-tokens // P)
    cache, g = filled(seed, pages, 1, P, D, kscale=0.02)
    pairs = cache.bytes[..., P * D:].view(np.float16).reshape(pages, 1, 2, P, 2)
    pairs[:, :, :, :, 1] = 0
    pairs[:, :, 1, :, 0] = (small * np.exp2(g.uniform(0, 1, (pages, 1, P)))).astype(np.float16)
    for t in at:
        pairs[t // P, 0, 1, t % P, 0] = large
        pairs[t // P, 0, 0, t % P, 1] = -below / (0.125 * D)
    return cache, g


def queries(g, T, heads, D, dtype):
    """A sum of about D a head, so that a key's middle moves its score by scale * D times itself."""
    return torch.from_numpy(1 + 0.3 * g.standard_normal((T, heads, D))).to(dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("small,large", [(1e-3, 2000), (1e-4, 2000), (1e-4, 4000)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_large_scale_of_no_weight(tq2, D, small, large, dtype):
    """One token with a large scale and a weight of 2^-60, in the first tile, in the middle and at the end."""
    for at in ([3], [70], [199], [5, 100, 198]):
        cache, g = unequal(D, D, 200, small, large, at, 42.0)
        check(tq2, cache, np.arange(7, dtype=np.int32)[None], queries(g, 1, 16, D, dtype), 200, FEW)


def test_a_large_scale_where_tokens_are_split(tq2):
    cache, g = unequal(3, 64, 4000, 1e-3, 2000, [1, 1777, 3999], 42.0)
    table = np.arange(125, dtype=np.int32)[None]
    check(tq2, cache, table, queries(g, 1, 8, 64, F16), 4000, FEW)
    check(tq2, cache, table, queries(g, 5, 7, 64, F16), 4000, FEW)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_large_scale_in_a_prompt(tq2, D, dtype):
    """The form for many rows (260 new tokens of 16 heads, a table of 300 tiles)."""
    for at in ([3], [5, 100, 290]):
        cache, g = unequal(D, D, 300, 1e-4, 4000, at, 42.0)
        table = np.full((1, 300), -1, np.int32)
        table[0, :10] = np.arange(10)
        check(tq2, cache, table, queries(g, 260, 16, D, dtype), 300, MANY)


@pytest.mark.parametrize("below", [0.0, 5.0, 16.0, 24.0])
def test_a_large_scale_of_some_weight(tq2, below):
    """From the one that decides the output to one that just adds to it."""
    cache, g = unequal(5, 64, 150, 1e-3, 2000, [90], below)
    check(tq2, cache, np.arange(5, dtype=np.int32)[None], queries(g, 2, 8, 64, F16), 150, FEW)


def test_scales_of_nothing_and_of_the_least(tq2):
    """Tokens without spread (scale 0) hold the largest scores; what is left of the others counts still."""
    cache, g = unequal(6, 64, 320, 0.0, 0.5, [40, 200, 300], 9.0)
    table = np.arange(10, dtype=np.int32)[None]
    check(tq2, cache, table, queries(g, 1, 8, 64, F16), 320, FEW)
    cache, g = unequal(7, 64, 320, 2.0 ** -24, 2.0 ** -14, [40, 200, 300], 3.0)
    check(tq2, cache, table, queries(g, 1, 8, 64, BF16), 320, FEW)


def test_rising_scores_and_falling_scales(tq2):
    """Every tile's scores pass the last one's, its scales fall below them, and the other way round."""
    for sign in (1, -1):
        cache, g = unequal(8, 64, 640, 1.0, 1.0, [], 0.0)
        pairs = cache.bytes[..., 32 * 64:].view(np.float16).reshape(20, 1, 2, 32, 2)
        tile = np.arange(20).reshape(20, 1, 1) * sign
        pairs[:, :, 0, :, 1] = (tile * 0.7 / (0.125 * 64) * 5).astype(np.float16)
        pairs[:, :, 1, :, 0] = np.exp2(-tile * 0.9 - (9 if sign < 0 else 0)).astype(np.float16)
        check(tq2, cache, np.arange(20, dtype=np.int32)[None], queries(g, 1, 4, 64, F16), 640, FEW)


def test_rows_do_not_move_each_other(tq2):
    """A row's bits do not depend on what the other rows of the call look like."""
    cache, g = unequal(9, 64, 400, 1e-3, 2000, [9, 133], 42.0)
    table = torch.arange(13, dtype=torch.int32, device=DEV)[None]
    c, ctx = torch.from_numpy(cache.bytes).to(DEV), torch.tensor([400], dtype=torch.int32, device=DEV)
    q = queries(g, 1, 16, 64, F16).to(DEV)
    a = tq2.tq2_kv4_attn(q, c, table, ctx)
    q2 = q.clone()
    q2[:, 1::2] *= -8
    assert torch.equal(a[:, ::2], tq2.tq2_kv4_attn(q2, c, table, ctx)[:, ::2])
