"""How the attention's work is dealt to workgroups, and the store's quotient,
on the host: the dealing from the kernels' own header, the quotient by its
steps."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from ternary_packed_weight_amd import build

HARNESS = r'''
#include "tq2_kv4.h"
extern "C" {
int tiles(int64_t s0, int64_t s1, int ctx, int64_t T, int max_q, int64_t most, int G, int row0, int rows, int window, int* o) {
  const tq2::Kv4Seq q = tq2::kv4_seq(s0, s1, ctx, T, max_q, most);
  o[0] = (int)q.q0, o[1] = q.n, o[2] = q.c;
  return tq2::kv4_tiles(q, G, row0, rows, window, o + 3);
}
uint32_t units(int tiles, int grain) { return tq2::kv4_units(tiles, grain); }
uint32_t share(uint32_t units, int Hk, uint32_t budget, uint32_t least) { return tq2::kv4_share(units, Hk, budget, least); }
void take(uint32_t units, int Hk, uint32_t share, uint32_t* o) {
  const tq2::Kv4Take t = tq2::kv4_take(units, Hk, share);
  o[0] = t.wgs, o[1] = t.slots, o[2] = t.splits;
}
}
'''


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4work")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", build.CSRC, str(d / "h.cpp"),
                    "-o", str(d / "h.so")], check=True)
    lib = ctypes.CDLL(str(d / "h.so"))
    lib.share.restype = lib.units.restype = ctypes.c_uint32
    lib.tiles.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                          ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    return lib


def test_dealt_work_fits_its_workspace(work):
    """Workgroups, slots and joined groups stay inside what a call reserves:
    budget + items, 2 * budget, min(items, budget)."""
    g = np.random.default_rng(1)
    out = (ctypes.c_uint32 * 3)()
    for _ in range(3000):
        entries, Hk = int(g.integers(1, 200)), int(g.choice([1, 2, 3, 8]))
        budget, least = int(g.choice([1, 128, 256, 490, 512])), int(g.choice([1, 8, 16, 48]))
        u = np.floor(np.exp(g.uniform(0, 12, entries))).astype(int) * (g.random(entries) < 0.9)
        share = work.share(int(u.sum()), Hk, budget, least)
        wgs = slots = splits = 0
        for x in u:
            work.take(int(x), Hk, share, out)
            assert out[0] * share >= x * Hk and (x == 0) == (out[0] == 0)
            assert out[1] in (0, out[0]) and (out[1] > 0) == (x > share) and out[2] == (Hk if x > share else 0)
            wgs, slots, splits = wgs + out[0], slots + out[1], splits + out[2]
        assert wgs <= budget + entries * Hk and slots <= 2 * budget and splits <= min(budget, entries * Hk)


def test_parts_cover_the_tiles_once():
    """A part takes ceil(n / parts) tiles, rounded up to whole steps; the last ones may be left with none."""
    for step in (1, 2):
        for n in list(range(1, 70)) + [157, 4094, 4095]:
            for parts in list(range(1, 40)) + [512]:
                chunk = -(-(-(-n // parts)) // step) * step
                seen = []
                for p in range(parts):
                    seen += range(chunk * p, min(chunk * p + chunk, n))
                assert seen == list(range(n))


def test_tiles_of_a_row_tile(work):
    o = (ctypes.c_int * 4)()
    t = lambda *a: work.tiles(*a, o)
    # 10 new tokens of 4 heads, 100 cached: rows 0..15 are tokens 0..3, which see up to 94 tokens
    assert t(5, 15, 100, 20, 16, 1000, 4, 0, 16, 0) == 3 and list(o) == [5, 10, 100, 0]
    assert t(5, 15, 100, 20, 16, 1000, 4, 32, 16, 0) == 4
    assert t(5, 15, 100, 20, 16, 1000, 4, 48, 16, 0) == 0          # no row there
    assert t(5, 15, 100, 20, 16, 1000, 4, 32, 16, 10) == 2 and o[3] == 2  # places 89-9 .. 99
    assert t(5, 15, 0, 20, 16, 1000, 4, 0, 16, 0) == 1             # rows that see nothing are written once
    assert t(5, 5, 100, 20, 16, 1000, 4, 0, 16, 0) == 0            # no new token
    # held inside the call's sizes
    assert t(-3, 1 << 40, 1 << 30, 20, 16, 1000, 4, 0, 16, 0) > 0 and list(o)[:3] == [0, 16, 1000]
    assert t(30, 40, -7, 20, 16, 1000, 4, 0, 16, 0) == 0 and list(o)[:3] == [20, 0, 0]


def test_units_of_many_tiles(work):
    assert [work.units(t, 0) for t in (0, 1, 7)] == [0, 1, 7] and [work.units(t, 3) for t in (0, 1, 8, 9)] == [0, 1, 1, 2]


def f32(x):
    return np.asarray(x).astype(np.float32)


@pytest.mark.parametrize("off", [-1, 0, 1])
def test_quotient_is_the_division(off):
    """q = a r, q + (a - q b) r, each one fp32 rounding, is a / b for every
    binary16 b and a reciprocal within one last place; numerators around whole
    and half quotients, where a code's border is."""
    if np.finfo(np.longdouble).nmant < 60:
        pytest.skip("needs an extended type for the fma")
    g = np.random.default_rng(2)
    b = np.concatenate([np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32), np.full(64, 15, np.float32)])
    r = (np.float32(1) / b).view(np.int32)
    r = (r + off).view(np.float32)
    L = np.longdouble
    for it in range(24):
        if it % 3 == 0:
            a = f32(g.uniform(-9, 9, b.shape)) * b
        else:
            near = g.integers(-9, 9, b.shape) + (0.5 if it % 3 == 2 else 0.0)
            a = f32(near * b.astype(np.float64) * (1 + g.integers(-3, 4, b.shape) * 2.0 ** -24))
        q = a * r
        q = f32(L(q) + L(f32(L(a) - L(q) * L(b))) * L(r))
        assert np.array_equal(q, a / b)


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses are only safe to pass where no GPU exists")
def test_workspace_is_enough_for_every_window():
    """The workspace that a call asks for does not know of a window: no window may need more."""
    from ternary_packed_weight_amd import tq2
    P = ctypes.c_void_p
    M = 1 << 40

    def status(B, mq, Hk, G, D, PP, width, window, need):
        T, Hq = B * mq, Hk * G
        return tq2.lib().tq2_kv4_attn(P(M), Hq * D, D, T, Hq, 0, P(2 * M), 1 << 20, PP, Hk, D, P(3 * M), width, width, P(4 * M),
                                      P(0), B, mq, 0.1, window, P(5 * M), P(0), P(6 * M), need, None)

    g = np.random.default_rng(3)
    for _ in range(400):
        B, mq = int(np.exp(g.uniform(0, 5))), int(np.exp(g.uniform(0, 7)))
        Hk, G, D = int(g.choice([1, 2, 8])), int(g.choice([1, 4, 16])), int(g.choice([64, 128, 256]))
        width = int(np.exp(g.uniform(0, 8)))
        need = tq2.tq2_kv4_attn_workspace_bytes(B * mq, Hk * G, Hk, D, 64, width, B, mq)
        assert need != 2 ** 64 - 1
        for window in (0, 1, 100, 700, 2500, 20000, 2 ** 31 - 1):
            assert status(B, mq, Hk, G, D, 64, width, window, need) == 6, (B, mq, Hk, G, D, width, window)  # the launch: no GPU here
