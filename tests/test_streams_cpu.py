"""What a call on a given stream allocates is allocated under that stream, for
every call of the binding: seen through torch's allocation and stream calls,
without a GPU (the tensors' placement is refused afterwards)."""
import os

import pytest
import torch

from ternary_packed_weight_amd import build


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


class Side:
    cuda_stream = 0


def calls(tq2):
    """name -> (call that allocates everything it can, tensors that it allocates)"""
    N, K, M = 512, 1024, 3
    W = torch.zeros((N, K))
    m = (torch.zeros((N, K // 4), dtype=torch.uint8), torch.zeros((N, K // 256), dtype=torch.float16))
    x, xq = torch.zeros(K, dtype=torch.float16), torch.zeros(K, dtype=torch.int8)
    X, XQ = torch.zeros((M, K), dtype=torch.float16), torch.zeros((M, K), dtype=torch.int8)
    big = tuple(torch.zeros((1024, n), dtype=t) for n, t in ((1024, torch.uint8), (16, torch.float16)))
    XQ16 = torch.zeros((16, 4096), dtype=torch.int8)
    ws = lambda n: int(n > 0)
    h = torch.zeros((2, 3, 128))
    pos, inv, slots = torch.zeros(2, dtype=torch.int32), torch.zeros(64), torch.zeros(2, dtype=torch.int64)
    cache, table = torch.zeros((9, 3, 32 * 136), dtype=torch.uint8), torch.zeros((2, 900), dtype=torch.int32)
    need = tq2.tq2_kv4_attn_workspace_bytes(2, 3, 3, 128, 32, 900, 2, 1)
    assert need > 0 and min(f(1024, 4096, 16) for f in (tq2.tq2_gemm_workspace_bytes,
                                                       tq2.tq2_gemm_i8q_workspace_bytes)) > 0
    return {
        "pack": (lambda s: tq2.tq2_pack(W, stream=s), 3),
        "dequant": (lambda s: tq2.tq2_dequant(*m, stream=s), 1),
        "gemv": (lambda s: tq2.tq2_gemv(*m, x, stream=s), 1),
        "gate_up": (lambda s: tq2.tq2_gemv_gate_up(*m, *m, x, stream=s), 1),
        "quantize": (lambda s: tq2.tq2_quantize_i8(x, 0.5, stream=s), 1),
        "gemv_i8q": (lambda s: tq2.tq2_gemv_i8q(*m, xq, 0.5, stream=s), 1 + ws(tq2.tq2_workspace_bytes(tq2.TQ2_OP_GEMV_I8Q, N, K))),
        "gemv_i8": (lambda s: tq2.tq2_gemv_i8(*m, x, 0.5, stream=s), 1 + ws(tq2.tq2_workspace_bytes(tq2.TQ2_OP_GEMV_I8, N, K))),
        "fused": (lambda s: tq2.tq2_gemv_fused([m, m], x, stream=s), 1),
        "i8_fused": (lambda s: tq2.tq2_gemv_i8_fused([m, m], x, 0.5, stream=s), 1),
        "silu": (lambda s: tq2.tq2_gemv_gate_up_silu(*m, *m, x, stream=s), 1),
        "requant": (lambda s: tq2.tq2_gemv_i8_requant(*m, x, 0.5, 0.5, stream=s), 2),
        "gemm": (lambda s: tq2.tq2_gemm(*m, X, stream=s), 1 + ws(tq2.tq2_gemm_workspace_bytes(N, K, M))),
        "gemm_i8q": (lambda s: tq2.tq2_gemm_i8q(*m, XQ, 0.5, stream=s), 1 + ws(tq2.tq2_gemm_i8q_workspace_bytes(N, K, M))),
        "gemm_i8q_ws": (lambda s: tq2.tq2_gemm_i8q(*big, XQ16, 0.5, stream=s), 2),
        "gemm_ws": (lambda s: tq2.tq2_gemm(*big, XQ16.half(), stream=s), 2),
        "noalloc": (lambda s: tq2.tq2_gemm_noalloc(*m, X, stream=s), 1),
        "rope": (lambda s: tq2.tq2_qk_norm_rope(h, h, pos, inv, stream=s), 2),
        "load": (lambda s: tq2.tq2_kv4_load(cache, slots, 128, stream=s), 2),
        "attn": (lambda s: tq2.tq2_kv4_attn(h.half(), cache, table, pos, stream=s), 2),
    }


@pytest.mark.parametrize("name", ["pack", "dequant", "gemv", "gate_up", "quantize", "gemv_i8q", "gemv_i8", "fused", "i8_fused",
                                  "silu", "requant", "gemm", "gemm_i8q", "gemm_i8q_ws", "gemm_ws", "noalloc", "rope", "load", "attn"])
def test_allocations_belong_to_the_given_stream(tq2, monkeypatch, name):
    call, count = calls(tq2)[name]
    under, made = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            under.append(self.stream)

        def __exit__(self, *a):
            under.pop()

    empty = torch.empty

    def recorded(*a, **kw):
        made.append(under[-1] if under else None)
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch, "empty", recorded)
    for side in (Side(), None):
        made.clear()
        with pytest.raises(ValueError, match="device tensor"):
            call(side)
        assert made == [side] * count
