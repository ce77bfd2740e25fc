"""The norm on columns of one matrix, the sum in place between them."""
import pytest

from tests.test_step_gpu import BF16, DEV, F16, F32, tq2  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("T,D", [(1, 72), (5, 72), (7, 4096), (600, 1000), (3, 16392)])
def test_sum_between_columns(tq2, T, D, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(T + D)
    whole = torch.randn((T, 3 * D), generator=g).to(dtype).to(DEV)
    x, r = whole[:, 2 * D:].clone(), whole[:, :D].clone()
    w = torch.randn(D, generator=g).to(DEV)
    out, h = tq2.tq2_add_rms_norm(x, r, w)
    q, s, _ = tq2.tq2_add_rms_norm_i8(x, r, w)
    for at in (0, D):  # in place of the residual, or between it and x
        for i8 in (False, True):
            a = whole.clone()
            kw = dict(weight=w, h_out=a[:, at:at + D])
            if i8:
                got_q, got_s, got = tq2.tq2_add_rms_norm_i8(a[:, 2 * D:], a[:, :D], **kw)
                assert torch.equal(got_q, q) and torch.equal(got_s, s)
            else:
                got_out, got = tq2.tq2_add_rms_norm(a[:, 2 * D:], a[:, :D], **kw)
                assert torch.equal(got_out, out)
            assert torch.equal(got, h)
            want = whole.clone()
            want[:, at:at + D] = h
            assert torch.equal(a, want)
