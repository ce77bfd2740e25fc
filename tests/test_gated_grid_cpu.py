"""One token's grid, from the launches' own header: what the header of the
library takes as rows has to find room in one."""
import ctypes
import functools
import os
import subprocess
import tempfile

import pytest

from ternary_packed_weight_amd import build

SOURCE = r'''
#include "tq2_step.h"
extern "C" {
int fits(int64_t N, int64_t K) { return tq2::gated_one_fits(N, K); }
int64_t threads(int64_t N, int64_t K) { return tq2::gated_one_groups(N, K) * tq2::kGatedOneThreads; }
int rows(int64_t K) { return tq2::kGatedOneRows * 4 / tq2::gated_one_waves(K); }
}
'''


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "grid.cpp"), os.path.join(d, "grid.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        rocm = os.path.join(os.path.dirname(os.path.dirname(build.HIPCC)), "include")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", rocm, "-I", build.CSRC,
                        src, "-o", so], check=True)
        so = ctypes.CDLL(so)
        for f in (so.fits, so.threads):
            f.argtypes = [ctypes.c_int64, ctypes.c_int64]
        so.threads.restype = ctypes.c_int64
        so.rows.argtypes = [ctypes.c_int64]
        return so


@pytest.mark.parametrize("K,rows,most", [(256, 16, 1 << 26), (4096, 16, 1 << 26), (4352, 8, (1 << 26) - 8), (8192, 8, (1 << 26) - 8),
                                         (8448, 4, (1 << 25) - 4), (16384, 4, (1 << 25) - 4)])
def test_rows_of_one_token(K, rows, most):
    """`most` rows are the last that fit: one workgroup of 512 threads for every
    `rows` of them makes (2^32 - 512) / 512 workgroups, or N ends at 2^26."""
    g = lib()
    assert g.rows(K) == rows
    for N in (1, rows, rows + 1, 16384, 1 << 24, most - 1, most, most + 1, 1 << 25, 1 << 26):
        threads = (N + rows - 1) // rows * 512
        assert g.threads(N, K) == threads
        assert bool(g.fits(N, K)) == (N <= most) == (threads < 1 << 32) or N > 1 << 26
    # what takes the rest: 32 rows a workgroup of 512 threads
    assert (1 << 26) // 32 * 512 < 1 << 32
