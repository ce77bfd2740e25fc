"""Columns of one matrix as a norm's tensors: the sum may stand between the
rows of what it does not touch.  Without a GPU."""
import ctypes
import os

import pytest
import torch

from ternary_packed_weight_amd import build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses are only safe to pass where no GPU exists")
A, M = 1 << 40, 1 << 32
ARG, HIP = 1, 6  # HIP: every check passed, and there is no GPU to launch on


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def norm(tq2, x, r, h, xs, rs=None, T=4, D=64, xd=2, rd=2, i8=False):
    p = ctypes.c_void_p
    head = (p(x), xs, xd, p(r), xs if rs is None else rs, rd, p(h), T, D, None, 1e-6)
    if i8:
        return tq2.lib().tq2_add_rms_norm_i8(*head, 0.5, p(A + M), None, None)
    return tq2.lib().tq2_add_rms_norm(*head, p(A + M), 0, None)


@pytest.mark.parametrize("i8", [False, True])
def test_columns_of_one_matrix(tq2, i8):
    f = lambda x, r, h, *a, **kw: norm(tq2, A + x, A + r, A + h, *a, i8=i8, **kw)  # noqa: E731
    row = 64 * 4
    # x beside the residual that the sum replaces, on either side; with columns between; all three
    assert f(row, 0, 0, 128) == HIP and f(0, row, row, 128) == HIP
    assert f(2 * row, 0, 0, 256) == HIP and f(2 * row, 0, row, 192) == HIP and f(0, 2 * row, row, 192) == HIP
    # rows of x that begin before or end behind those of the sum
    assert f(3 * row, 0, 0, 128) == HIP and f(0, 3 * row, 3 * row, 128) == HIP
    # some of their elements are one
    assert f(row - 16, 0, 0, 128) == ARG and f(row + 16, 0, 0, 128) == ARG and f(0, row - 16, row - 16, 128) == ARG
    assert f(0, row + 16, row + 16, 128) == ARG and f(0, 0, 0, 128) == ARG
    assert f(2 * row, 0, row - 16, 192) == ARG and f(2 * row, 0, row + 16, 192) == ARG
    # other strides: rows that drift into each other
    assert f(row, 0, 0, 132, rs=128) == ARG and f(row, 0, 0, 128, rs=132) == ARG and f(row, 0, 0, 0, rs=128) == ARG
    # the same in elements, not in bytes
    assert f(row, 0, 0, 128, xd=0) == ARG
    # one row: its stride says nothing
    assert f(row, 0, 0, 128, T=1) == HIP and f(row - 16, 0, 0, 128, T=1) == ARG
