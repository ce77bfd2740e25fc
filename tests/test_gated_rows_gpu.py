"""One token through more rows than its own form's grid holds."""
import numpy as np
import pytest

from oracle import step as ref
from tests.test_step_gpu import DEV, F16, f64, gated_tol, magnitudes, tq2  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_one_token_through_most_rows(tq2):  # noqa: F811
    """2^25 rows of 8448 (71 GB of codes, gate and up one matrix): rows at both ends and between."""
    N, K = 1 << 25, 8448
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = torch.full((N, K // 4), 0x55, dtype=torch.uint8, device=DEV)   # weights of 0
    scales = torch.full((N, K // 256), 0.01, dtype=F16, device=DEV)
    at = torch.tensor([0, 1, 31, 32, 4097, N // 2 - 1, N // 2, N - 33, N - 2, N - 1], device=DEV)
    some = torch.randint(0, 256, (len(at), K // 4), generator=g, device=DEV, dtype=torch.uint8)
    codes[at] = some & ~((some >> 1) & some & 0x55) & 0xFF                 # code 3 becomes 2
    x = torch.randn((1, K), generator=g, device=DEV).half()
    h = tq2.tq2_gemm_gate_up_silu(codes, scales, codes, scales, x, out_dtype=torch.float32)
    got = f64(h[0, at])
    w = ref.dense(codes[at].cpu().numpy(), scales[at].cpu().numpy())
    want, gs, us, *_ = ref.gated(w, w, f64(x))
    a = magnitudes(w, f64(x))
    assert np.all(np.abs(got - want[0]) <= gated_tol(gs, us, a, a, want, K, torch.float32)[0])
    assert int((h != 0).sum()) == int((h[0, at] != 0).sum()) == len(at)
