"""The limits that the header names, from both sides, without a GPU."""
import ctypes
import os

import pytest
import torch

from ternary_packed_weight_amd import build

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device addresses are only safe to pass where no GPU exists")
BAD = ctypes.c_size_t(-1).value
A, M = 1 << 44, 1 << 40
SHAPE, HIP = 2, 6  # HIP: every check passed, and there is no GPU to launch on


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def attn(tq2, T, Hq, Hk, B, mq, D=64, P=32, w=1, ts=None, qs=A + 9 * M):
    p = ctypes.c_void_p
    return tq2.lib().tq2_kv4_attn(p(A), Hq * D, D, T, Hq, 0, p(A + M), 9, P, Hk, D, p(A + 16 * M), w if ts is None else ts, w,
                                  p(A + 3 * M), p(qs), B, mq, 0.1, 0, p(A + 4 * M), p(0), p(A + 6 * M), 1 << 30, None)


@no_gpu
def test_attention_limits(tq2):
    ws = lambda T, Hq, Hk, B, mq, D=64, P=32, w=1: tq2.tq2_kv4_attn_workspace_bytes(T, Hq, Hk, D, P, w, B, mq)
    # rows outside every sequence: as many as B * max_q leaves
    assert attn(tq2, 6, 8, 2, 3, 2) == HIP and attn(tq2, 7, 8, 2, 3, 2) == SHAPE
    assert ws(6, 8, 2, 3, 2) == 0 and ws(7, 8, 2, 3, 2) == BAD
    # B * max_q * Hq
    assert attn(tq2, 5, 1, 1, 1, 2 ** 31 - 129) == HIP and attn(tq2, 5, 2, 1, 1, 2 ** 30) == SHAPE
    assert attn(tq2, 5, 65536, 1, 5, 1) == HIP and attn(tq2, 5, 65537, 1, 5, 1) == SHAPE
    assert attn(tq2, 5, 4096, 4096, 5, 1) == HIP and attn(tq2, 5, 4097, 4097, 5, 1) == SHAPE
    # the table
    assert attn(tq2, 2, 1, 1, 2, 1, w=2 ** 26 - 1) == HIP and attn(tq2, 2, 1, 1, 2, 1, w=2 ** 26) == SHAPE
    assert attn(tq2, 2, 1, 1, 2, 1, ts=2 ** 39) == HIP and attn(tq2, 2, 1, 1, 2, 1, ts=2 ** 39 + 1) == SHAPE
    # workgroups
    n = 2 ** 24
    assert attn(tq2, n - 513, 1, 1, n - 513, 1) == HIP and attn(tq2, n, 1, 1, n, 1) == SHAPE
    assert ws(n - 513, 1, 1, n - 513, 1) == 0 and ws(n, 1, 1, n, 1) == BAD
    # tokens
    assert attn(tq2, 2 ** 26, 1, 1, 2 ** 14, 2 ** 14) == HIP and attn(tq2, 2 ** 26 + 1, 1, 1, 2 ** 14, 2 ** 14) == SHAPE


@no_gpu
def test_rotation_and_cache_limits(tq2):
    p = ctypes.c_void_p

    def rope(T):
        return tq2.lib().tq2_qk_norm_rope(p(A), 16, 16, 1, p(0), 0, 0, 0, 0, T, 16, p(0), p(0), 0.0, p(A + M), p(A + 2 * M), 16, 0,
                                          p(A + 3 * M), p(0), 0, None)

    def store(T, Hk):
        return tq2.lib().tq2_kv4_store(p(A), 9, 32, Hk, 64, p(A + M), Hk * 64, 64, p(A + 2 * M), Hk * 64, 64, 0, p(A + 3 * M), T, None)

    assert rope(2 ** 26) == HIP and rope(2 ** 26 + 1) == SHAPE
    assert store(2 ** 26, 1) == HIP and store(2 ** 26 + 1, 1) == SHAPE
    assert store(2 ** 14, 4096) == HIP and store(2 ** 14 + 1, 4096) == SHAPE
