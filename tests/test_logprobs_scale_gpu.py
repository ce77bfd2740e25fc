"""Log probabilities of scaled logits: the distances from a row's largest logit
are scaled, so nothing passes fp32's range, the largest token's own distance is
0, and the error does not grow with the logits."""
import numpy as np
import pytest

from oracle import step as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = (torch.float16, torch.bfloat16, torch.float32)


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def logits(T, V, dtype, seed, size=4.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn((T, V), generator=g)).to(dtype).to(DEV)


def against_64_bits(tq2, x, tok, scale):
    """The distance d of a logit from the largest is off by half a step, the
    rate and their product by half a step each, the power by a unit: the mean of
    3 |d| over p, and a lane's V/256 sums, the lanes', waves' and parts' on top.
    Outside the sum: half a step of the distance and of the result, a unit and a
    half of the logarithm.  |d| and the logarithm are at most |log p|.  Below
    e^-87 a term may be 0."""
    T, V = x.shape
    lp64, H64 = ref.logprobs(x.double().cpu().numpy(), scale)
    lp, H, tt, tl = tq2.tq2_token_logprobs(x, tok, top=min(V, 7), scale=scale, want_entropy=True)
    at = ref.top_tokens(x.double().cpu().numpy(), min(V, 7))
    assert np.array_equal(tt.cpu().numpy(), at)
    p, far = np.exp(lp64), np.where(np.isfinite(lp64), -lp64, 0)
    mean = (p * far).sum(-1)
    term = (3 * mean + V / 256 + 80) * 2.0 ** -24
    for got, want in ((lp[:, None], np.take_along_axis(lp64, tok.cpu().numpy()[:, None], 1)), (tl, np.take_along_axis(lp64, at, 1))):
        got = got.cpu().double().numpy()
        with np.errstate(over="ignore"):  # log probabilities beyond fp32's range are -inf there
            low = np.isneginf(want.astype(np.float32))
        assert np.isneginf(got[low]).all()
        err = np.abs(np.where(low, 0, got) - np.where(low, 0, want))
        assert np.all(err <= term[:, None] + 5 * 2.0 ** -24 * np.abs(np.where(low, 0, want)))
    assert np.all(np.abs(H.cpu().double().numpy() - H64) <= 2 * term + 2 * term * mean + 4 * 2.0 ** -24 * np.abs(H64))


# one workgroup a row, and rows shared by workgroups
@pytest.mark.parametrize("T,V", [(4, 200), (3, 9001), (600, 3001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [25.0, 2.0, float(np.finfo(np.float32).max)])
def test_products_beyond_fp32(tq2, T, V, dtype, scale):
    """Finite logits whose product with the scale is not: far above the others,
    all masked by the type's lowest number, some masked so."""
    low = torch.finfo(dtype).min
    x = logits(T, V, dtype, 1)
    x[0, V // 2] = 3e38
    x[1] = low
    x[2, ::3] = low
    tok = torch.full((T,), V // 2, device=DEV)
    tok[2] = 3
    against_64_bits(tq2, x, tok, scale)
    lp, H, _, _ = tq2.tq2_token_logprobs(x, tok, scale=scale, want_entropy=True)
    assert lp[0] == 0 and H[0] == 0 and lp[2] == -torch.inf
    assert abs(float(lp[1]) + np.log(V)) < 1e-5 and abs(float(H[1]) - np.log(V)) < 1e-5


@pytest.mark.parametrize("T,V", [(1, 300), (1, 50000), (600, 2000)])
@pytest.mark.parametrize("scale", [33.33, 1.7, 0.3, 1.0])
def test_certain_token(tq2, T, V, scale):
    """A token far above the others has log probability 0 where the others lie
    more than 104 below (e^-104 is less than half of fp32's least number)."""
    for value in (30.1, 77.77, 401.3, 1009.0 + 1 / 3):
        x = torch.full((T, V), value - 110 / scale, device=DEV)
        x[:, V - 2] = value
        tok = torch.full((T,), V - 2, device=DEV)
        lp, H, tt, tl = tq2.tq2_token_logprobs(x, tok, top=2, scale=scale, want_entropy=True)
        assert bool((lp == 0).all()) and bool((tl[:, 0] == 0).all()) and bool((tt[:, 0] == V - 2).all())
        assert bool((H == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1.0, 0.7, 3.3, 25.0])
@pytest.mark.parametrize("T,V", [(2, 500), (3, 20001), (700, 2500)])
def test_one_token_one_value(tq2, T, V, dtype, scale):
    """A token's log probability is at most 0 and the same bits by either name."""
    x = logits(T, V, dtype, T + V)
    _, _, tt, tl = tq2.tq2_token_logprobs(x, top=9, scale=scale)
    assert bool((tl <= 0).all())
    for j in range(9):
        lp, _, _, _ = tq2.tq2_token_logprobs(x, tt[:, j].contiguous(), scale=scale)
        assert torch.equal(lp, tl[:, j])


@pytest.mark.parametrize("scale", [0.01, 1.0, 1.7, 33.33])
@pytest.mark.parametrize("far", [0.0, 5000.0, -5000.0])
@pytest.mark.parametrize("T,V", [(2, 500), (2, 20001), (600, 2500)])
def test_error_goes_by_distances(tq2, T, V, scale, far):
    x = logits(T, V, torch.float32, 5 + T, 9.0) + far
    tok = torch.randint(V, (T,), generator=torch.Generator().manual_seed(3)).to(DEV)
    against_64_bits(tq2, x, tok, float(np.float32(scale)))
