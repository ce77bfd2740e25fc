"""How near the attention half's calls come to 64 bits where a bound per
element is wide: statistics over many outputs, with what each rounding adds."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_kv4_gpu import f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("start", [0, 1000000])
def test_angles_are_held_beyond_32_bits(tq2, inter, start):
    """fp32 in, fp32 out, no norm.  A rounding to fp32 is off by 0.42 * 2^-24 in
    the mean square.  An output takes the sum's (0.42), one product's on half of
    the weight (0.30) and its sine's and cosine's, each within one rounding more
    than the right one (0.60): 0.79 * 2^-24 together.  An angle rounded to 32
    bits of a turn's fraction would add 0.69, to 1.05."""
    T, H, D = 1024, 12, 128
    x = torch.randn((T, H, D), generator=torch.Generator().manual_seed(start + inter))
    pos = (start + torch.arange(T) * 3).int()
    inv = (10000.0 ** (-torch.arange(0, D, 2).double() / D)).float()
    y, _ = tq2.tq2_qk_norm_rope(x.to(DEV), x[:, :0].to(DEV), pos.to(DEV), inv.to(DEV), interleaved=inter)
    want, _ = ref.norm_rope(f64(x), None, 0.0, pos.numpy(), inv.numpy(), inter)
    off = np.sqrt(np.mean((f64(y) - want) ** 2) / np.mean(want ** 2))
    assert off <= 0.8 * 2.0 ** -24, off * 2 ** 24


@pytest.mark.parametrize("start", [2 ** 24, 2 ** 28 + 1, 2 ** 31 - 1024, -2 ** 31])
def test_angles_of_the_farthest_positions(tq2, start):
    """As above, of any position: products of 31 by 24 bits and hundreds of
    millions of turns.  The reference reduces in an extended type: 2^-64 of
    2^29 turns is 2^-35 of one, far below an fp32 rounding."""
    if np.finfo(np.longdouble).nmant < 63:
        pytest.skip("needs an extended type")
    T, H, D = 1024, 4, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H, D), generator=g)
    pos = torch.from_numpy(start + np.arange(T)).int()
    inv = 0.5 + 0.5 * torch.rand(D // 2, generator=g)
    y, _ = tq2.tq2_qk_norm_rope(x.to(DEV), x[:, :0].to(DEV), pos.to(DEV), inv.to(DEV))
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    a = np.fmod(pos.numpy().astype(np.longdouble)[:, None] * inv.numpy().astype(np.longdouble), two_pi).astype(np.float64)[:, None]
    u, v = f64(x)[..., :D // 2], f64(x)[..., D // 2:]
    want = np.concatenate([u * np.cos(a) - v * np.sin(a), v * np.cos(a) + u * np.sin(a)], -1)
    off = np.sqrt(np.mean((f64(y) - want) ** 2) / np.mean(want ** 2))
    assert off <= 0.8 * 2.0 ** -24, off * 2 ** 24
