"""Sizes at the ends of what the attention half's calls take: places next to
2^31 and the most tokens of a call, against the same work at small places and
in pieces."""
import numpy as np
import pytest

from tests.test_kv4_gpu import filled

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


@pytest.mark.parametrize("S,G", [(260, 16), (600, 7), (1, 16), (5, 16)])
def test_places_next_to_two_gibi(tq2, S, G):
    """A table of the greatest width, its pages over and over; windows that end in
    an odd and an even number of tiles."""
    D, P, near = 64, 32, 300
    most = 2 ** 26 - 1
    cache, g = filled(1, 300, 1, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    small = torch.from_numpy(g.permutation(300).astype(np.int32)).to(DEV)[None]
    far = torch.zeros((1, most), dtype=torch.int32, device=DEV)
    far[:, most - near:] = small
    q = torch.from_numpy(g.standard_normal((S, G, D))).to(F16).to(DEV)

    def run(table, width, short, window):
        lse = torch.zeros((S, G), device=DEV)
        ctx = torch.tensor([width * P - short], dtype=torch.int32, device=DEV)
        return tq2.tq2_kv4_attn(q, c, table, ctx, window=window, lse=lse), lse

    for window in (40, 70, 100, 170):
        for short in (0, 1, 33):
            a, al = run(small, near, short, window)
            b, bl = run(far, most, short, window)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(a).all()) and torch.equal(al, bl) and torch.equal(a, b), (window, short)


@pytest.mark.parametrize("T", [2 ** 25 + 1, 2 ** 26 - 3, 2 ** 26])
def test_the_most_tokens_of_a_rotation(tq2, T):
    """The same bits as in pieces."""
    D = 16
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, 1, D), generator=g, device=DEV, dtype=F16)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    inv, w = torch.rand(D // 2, generator=g, device=DEV), torch.rand(D, generator=g, device=DEV)
    none = x[:, :0]
    y, _ = tq2.tq2_qk_norm_rope(x, none, pos, inv, w)
    for t in range(0, T, 2 ** 24):
        e = min(T, t + 2 ** 24)
        z, _ = tq2.tq2_qk_norm_rope(x[t:e], none[t:e], pos[t:e], inv, w)
        assert torch.equal(y[t:e], z), t
    del x, y, z
    torch.cuda.empty_cache()
