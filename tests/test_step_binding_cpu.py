"""The calls of the feed-forward half and the answer without a GPU: the
workspaces, the current device, and the binding without its native part."""
import ctypes
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from ternary_packed_weight_amd import build

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device addresses are only safe to pass where no GPU exists")
ROOT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..")
A, M = 1 << 40, 1 << 32  # fake, aligned, never dereferenced
BAD = 2 ** 64 - 1


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def test_gated_workspace_sizes(tq2):
    for M_ in (1, 16, 17, 33, 600, 65536):
        assert tq2.tq2_gemm_gate_up_silu_workspace_bytes(4096, 4096, M_) == 0
    size = tq2.tq2_gemm_i8q_gate_up_silu_workspace_bytes
    assert size(4096, 4096, 1) == size(4096, 4096, 32) == 0
    assert size(4096, 4096, 33) == 128 * 4096 * 3 // 2       # 12 bits an activation, whole groups of 128 tokens
    assert size(4096, 4096, 129) == 256 * 4096 * 3 // 2
    assert size(1, 256, 33) == 128 * 256 * 3 // 2
    for K in (256, 4096, 65280):
        assert 0 < size(64, K, 65536) <= 48 << 20
    for N, K, m in ((0, 256, 1), (1, 255, 1), (1, 65536, 1), (1, 256, 0), (1, 256, 65537), ((1 << 26) + 1, 256, 1)):
        assert size(N, K, m) == BAD


@no_gpu
def test_gated_workspace_refusals(tq2):
    lib = tq2.lib()

    def f(m=600, N=100, K=4096, ws=A + 6 * M, less=0):
        need = lib.tq2_gemm_i8q_gate_up_silu_workspace_bytes(N, K, m)
        p = [ctypes.c_void_p(a) for a in (A, A + M, A + 2 * M, A + 3 * M, A + 4 * M, A + 5 * M, ws)]
        return lib.tq2_gemm_i8q_gate_up_silu(*p[:4], N, K, p[4], m, 0.5, None, p[5], 0, p[6], need - less, None)

    assert f(ws=0) == 4 and f(less=1) == 4 and f(ws=A + 6 * M + 128) == 4
    for at in (A, A + M, A + 2 * M, A + 3 * M, A + 4 * M, A + 5 * M):
        assert f(ws=at) == 4                                 # in an input or in the output


def test_tensors_of_another_device(tq2, monkeypatch):
    """The checks that every one of these calls makes last, on stand-ins."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 1))
    b = SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0))
    with pytest.raises(ValueError, match="on cuda:1, the current device is cuda:0"):
        tq2._here(None, x=a, out=a)
    with pytest.raises(ValueError, match="on one device"):
        tq2._here(None, x=a, out=b)
    assert tq2._here(SimpleNamespace(cuda_stream=7), x=b, out=None).value == 7


WITHOUT = r"""
import sys
sys.modules["ternary_packed_weight_amd._tq2call"] = None   # what an import of a module that is not there meets
import torch
from ternary_packed_weight_amd import tq2

def refused(match, fn, *a, **kw):
    try:
        fn(*a, **kw)
    except ValueError as e:
        assert match in str(e), e
    else:
        raise AssertionError(match)

c, s = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.float16)
x, h = torch.zeros((3, 256), dtype=torch.float16), torch.zeros((3, 8), dtype=torch.float16)
refused("device tensor", tq2.tq2_add_rms_norm, x, x, h_out=x, out=torch.zeros_like(x))
refused("device tensor", tq2.tq2_add_rms_norm_i8, x, x, h_out=x, x_q=x.to(torch.int8), x_scales=torch.zeros(3))
refused("device tensor", tq2.tq2_gemm_gate_up_silu, c, s, c, s, x, h=h)
refused("device tensor", tq2.tq2_gemm_i8q_gate_up_silu, c, s, c, s, x.to(torch.int8), 0.5, h=h)
refused("device tensor", tq2.tq2_token_logprobs, x, torch.zeros(3, dtype=torch.int64), logprobs=torch.zeros(3))
refused("weight must hold 256", tq2.tq2_add_rms_norm, x, weight=torch.ones(255))
print("all calls")
"""


def test_calls_without_the_native_part():
    if not os.path.exists(build.LIB):
        build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all calls" in r.stdout, r.stderr
