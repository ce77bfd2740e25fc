"""The gated projections' epilogue: silu(g) * u of sums that are exact."""
import numpy as np
import pytest

from oracle import step as ref
from tests.test_step_gpu import DEV, f64, tq2  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Half steps of the value: the exponential and the reciprocal are off by a unit
# each (two half steps each), the sum under the reciprocal is rounded twice, the
# product with g once and that with u once.  What t = -g log2 e loses is put back,
# so |g| is not in it.
HALF_STEPS = 8.01


def weights(N, K):
    """Gate rows that take place 0, up rows that take place 1, as they are."""
    gate, up = (torch.full((N, K // 4), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))  # zeros
    gate[:, 0], up[:, 0] = 0x56, 0x59
    one = torch.ones((N, K // 256), dtype=torch.float16, device=DEV)
    return gate, one, up, one


def close(h, g, u):
    want = (ref.silu(g) * u)[:, None]
    assert np.all(np.abs(f64(h) - want) <= HALF_STEPS * 2.0 ** -24 * np.abs(want))


# one token, few, and every form for many
@pytest.mark.parametrize("M,N", [(1, 40), (2, 40), (16, 16400), (30, 40), (64, 9000), (100, 700), (129, 8100), (300, 9000)])
def test_fp16(tq2, M, N):  # noqa: F811
    w = weights(N, 512)
    for turn in range(400 // min(M, 20)):
        rng = np.random.default_rng(turn)
        x = torch.zeros((M, 512), dtype=torch.float16)
        x[:, 0] = torch.from_numpy(rng.uniform(-86.9, 86.9, M))
        x[:, 1] = torch.from_numpy(rng.uniform(0.5, 2.0, M))
        h = tq2.tq2_gemm_gate_up_silu(*w, x.to(DEV), out_dtype=torch.float32)
        close(h, x[:, 0].double().numpy(), x[:, 1].double().numpy())


@pytest.mark.parametrize("M,N", [(1, 40), (16, 16400), (30, 40), (33, 40), (300, 9000)])
def test_int8(tq2, M, N):  # noqa: F811
    w = weights(N, 512)
    s = 0.6875  # times 127 and less: exact
    for turn in range(400 // min(M, 20)):
        rng = np.random.default_rng(turn)
        x = torch.zeros((M, 512), dtype=torch.int8)
        x[:, 0] = torch.from_numpy(rng.integers(-126, 128, M))
        x[:, 1] = torch.from_numpy(rng.integers(1, 128, M))
        h = tq2.tq2_gemm_i8q_gate_up_silu(*w, x.to(DEV), s, out_dtype=torch.float32)
        close(h, s * x[:, 0].double().numpy(), s * x[:, 1].double().numpy())


@pytest.mark.parametrize("M", [1, 16, 140])
def test_ends_of_silu(tq2, M):  # noqa: F811
    """Zero, numbers beyond the exponential's range, infinities and NaN as the formula has them."""
    w = weights(64, 512)
    for g, want in ((0.0, 0.0), (-0.0, 0.0), (120.5, 120.5 * 3), (65504.0, 65504.0 * 3), (-104.0, 0.0), (-121.0, 0.0), (-65504.0, 0.0)):
        x = torch.zeros((M, 512), dtype=torch.float16, device=DEV)
        x[:, 0], x[:, 1] = g, 3.0
        h = tq2.tq2_gemm_gate_up_silu(*w, x, out_dtype=torch.float32)
        assert torch.allclose(h, torch.full_like(h, want), rtol=2.0 ** -21, atol=2.0 ** -118)
    # (infinite activations where no weight is 0)
    plus = torch.full((64, 64), 0xAA, dtype=torch.uint8, device=DEV)
    one = torch.ones((64, 1), dtype=torch.float16, device=DEV)
    x = torch.zeros((M, 256), dtype=torch.float16, device=DEV)
    x[0, 5] = torch.inf
    assert bool((tq2.tq2_gemm_gate_up_silu(plus, one, plus, one, x)[0] == torch.inf).all())
    x[0, 5] = -torch.inf
    assert bool(tq2.tq2_gemm_gate_up_silu(plus, one, plus, one, x)[0].isnan().all())
    x[0, 5] = torch.nan
    assert bool(tq2.tq2_gemm_gate_up_silu(plus, one, plus, one, x)[0].isnan().all())
