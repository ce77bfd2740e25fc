"""The attention half of a decode step without a GPU: refusals of the C ABI
and of the binding, the cache's addresses and a call's split of the tokens
(compiled for the host from the kernels' own header), and pins of the
oracles."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import attention as ref
from ternary_packed_weight_amd import build

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device addresses are only safe to pass where no GPU exists")
A = 1 << 40  # fake, aligned, never dereferenced
BAD = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def tq2():
    if not os.path.exists(build.LIB):
        build.build()
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def P(addr):
    return ctypes.c_void_p(addr)


# ---- refusals of the C ABI ----

@no_gpu
def test_rope_refusals(tq2):
    M = 1 << 32

    def f(q=A, qts=2304, qhs=128, Hq=16, k=A + M, kts=2304, khs=128, Hk=2, idt=0, T=4, D=128, qw=0, kw=0, eps=1e-6,
          pos=A + 2 * M, inv=A + 3 * M, rot=128, il=0, qo=A + 4 * M, ko=A + 5 * M, odt=0):
        return tq2.lib().tq2_qk_norm_rope(P(q), qts, qhs, Hq, P(k), kts, khs, Hk, idt, T, D, P(qw), P(kw), eps, P(pos),
                                          P(inv), rot, il, P(qo), P(ko), odt, None)

    assert f(T=0) == 0 and f(T=-1) == 1
    assert f(Hq=0, Hk=0) == 1 and f(Hq=-1) == 1 and f(q=0) == 1 and f(k=0) == 1 and f(qo=0) == 1 and f(ko=0) == 1
    assert f(pos=0) == 1 and f(inv=0) == 1 and f(il=2) == 1
    assert f(idt=3) == 1 and f(odt=-1) == 1
    assert f(eps=-1.0) == 1 and f(eps=float("nan")) == 1 and f(eps=float("inf")) == 1
    assert f(D=8) == 2 and f(D=120) == 2 and f(D=528) == 2 and f(rot=144) == 2 and f(rot=8) == 2 and f(rot=-16) == 2
    assert f(qts=-1) == 1 and f(qts=1 << 41) == 2
    assert f(q=A + 8) == 3 and f(qts=2305) == 3 and f(khs=132) == 3 and f(qo=A + 4 * M + 8) == 3 and f(qw=A + 2) == 3
    assert f(qo=A + 16) == 1 and f(ko=A + 4 * M + 1024) == 1 and f(qo=A + 2 * M) == 1  # overlaps


def _store(tq2, cache=A, pages=8, PP=32, Hk=2, D=64, k=A + (1 << 32), kts=128, khs=64, v=A + (2 << 32), vts=128, vhs=64,
           dt=0, slots=A + (3 << 32), T=5):
    return tq2.lib().tq2_kv4_store(P(cache), pages, PP, Hk, D, P(k), kts, khs, P(v), vts, vhs, dt, P(slots), T, None)


@no_gpu
def test_store_and_load_refusals(tq2):
    f = lambda **kw: _store(tq2, **kw)
    assert f(T=0) == 0 and f(T=-1) == 1 and f(pages=0) == 1 and f(Hk=0) == 1 and f(dt=3) == 1
    assert f(cache=0) == 1 and f(k=0) == 1 and f(v=0) == 1 and f(slots=0) == 1
    assert f(PP=16) == 2 and f(PP=48) == 2 and f(PP=8192) == 2 and f(D=32) == 2 and f(D=96) == 2 and f(D=512) == 2
    assert f(pages=1 << 40) == 2 and f(T=1 << 31) == 2
    assert f(cache=A + 8) == 3 and f(k=A + (1 << 32) + 2) == 3 and f(slots=A + (3 << 32) + 4) == 3 and f(vhs=60) == 3
    assert f(k=A + 64) == 1 and f(slots=A + 8) == 1  # inside the cache

    def g(cache=A, pages=8, PP=32, Hk=2, D=64, slots=A + (3 << 32), T=5, k=A + (1 << 32), v=A + (2 << 32), dt=2):
        return tq2.lib().tq2_kv4_load(P(cache), pages, PP, Hk, D, P(slots), T, P(k), P(v), dt, None)

    assert g(T=0) == 0 and g(T=-1) == 1 and g(k=0, v=0) == 1 and g(cache=0) == 1 and g(slots=0) == 1 and g(dt=-1) == 1
    assert g(D=100) == 2 and g(PP=31) == 2 and g(k=A + (1 << 32) + 8) == 3
    assert g(k=A + 16) == 1 and g(v=A + (1 << 32)) == 1
    assert tq2.tq2_kv4_page_bytes(64, 2, 128) == 2 * 64 * 136 and tq2.tq2_kv4_page_bytes(33, 2, 128) == 0
    assert tq2.tq2_kv4_page_bytes(64, 0, 128) == 0


@no_gpu
def test_attn_refusals(tq2):
    M = 1 << 34

    def f(q=A, qts=512, qhs=64, T=3, Hq=8, dt=0, cache=A + M, pages=9, PP=32, Hk=2, D=64, table=A + 2 * M, ts=4, w=4,
          ctx=A + 3 * M, qs=0, B=3, mq=1, scale=0.1, window=0, out=A + 4 * M, lse=0, ws=A + 5 * M, wb=1 << 26):
        return tq2.lib().tq2_kv4_attn(P(q), qts, qhs, T, Hq, dt, P(cache), pages, PP, Hk, D, P(table), ts, w, P(ctx),
                                      P(qs), B, mq, scale, window, P(out), P(lse), P(ws), wb, None)

    assert f(T=0, mq=1) == 0 and f(T=-1) == 1
    assert f(B=0) == 1 and f(mq=0) == 1 and f(w=0) == 1 and f(window=-1) == 1 and f(Hq=9) == 1 and f(Hq=0) == 1
    assert f(dt=2) == 1 and f(dt=-1) == 1 and f(pages=0) == 1
    assert f(scale=float("nan")) == 5 and f(scale=float("inf")) == 5
    assert f(D=96) == 2 and f(PP=33) == 2 and f(T=4) == 2 and f(T=2) == 2 and f(w=1 << 30) == 2 and f(ts=-4) == 2
    assert f(B=1 << 28, mq=8, T=1 << 31) == 2
    assert f(q=0) == 1 and f(cache=0) == 1 and f(table=0) == 1 and f(ctx=0) == 1 and f(out=0) == 1
    assert f(q=A + 8) == 3 and f(qhs=65) == 3 and f(out=A + 4 * M + 4) == 3 and f(lse=A + 6 * M + 2) == 3
    assert f(out=A + 64) == 1 and f(out=A + M) == 1 and f(lse=A + 4 * M) == 1 and f(out=A + 2 * M) == 1
    need = tq2.tq2_kv4_attn_workspace_bytes(3, 8, 2, 64, 32, 64, 3, 1)
    assert 0 < need < 1 << 24
    assert f(w=64, ws=0) == 4 and f(w=64, wb=need - 1) == 4 and f(w=64, ws=A + 5 * M + 64) == 4
    assert f(w=64, ws=A + 4 * M) == 4 and f(w=64, ws=A + M) == 4
    ws = tq2.tq2_kv4_attn_workspace_bytes
    assert ws(3, 8, 2, 64, 32, 1, 3, 1) == 0                  # one tile of tokens: nothing to split
    assert ws(3, 8, 3, 64, 32, 1, 3, 1) == BAD and ws(3, 8, 2, 65, 32, 1, 3, 1) == BAD
    assert ws(3, 8, 2, 64, 32, 0, 3, 1) == BAD and ws(3, 8, 2, 64, 32, 1, 0, 1) == BAD and ws(7, 8, 2, 64, 32, 1, 3, 2) == BAD


def test_attn_workspace_stays_small(tq2):
    worst = 0
    for B in (1, 2, 7, 64, 300):
        for mq in (1, 5, 40, 700):
            for Hk, G in ((1, 1), (2, 16), (8, 4), (3, 33)):
                for D in (64, 128, 256):
                    for w in (1, 10, 4096):
                        worst = max(worst, tq2.tq2_kv4_attn_workspace_bytes(B * mq, Hk * G, Hk, D, 64, w, B, mq))
    assert 0 < worst <= 64 << 20


# ---- refusals of the binding (CPU tensors: none reaches the library) ----

def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_refusals(tq2):
    q, k = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64))
    pos, inv = torch.zeros(3, dtype=torch.int32), torch.zeros(32)
    rope = tq2.tq2_qk_norm_rope
    _raises("q must be a", rope, q[0], k, pos, inv)
    _raises("q must have dtype", rope, q.double(), k.double(), pos, inv)
    _raises("same tokens", rope, q, k[:2], pos, inv)
    _raises("same tokens", rope, q, k.half(), pos, inv)
    _raises("contiguous", rope, q.transpose(1, 2), k, pos, inv)
    _raises("positions must have dtype", rope, q, k, pos.long(), inv)
    _raises("positions must hold 3", rope, q, k, pos[:2], inv)
    _raises("inv_freq must have dtype", rope, q, k, pos, inv.double())
    _raises("q_weight must hold 64", rope, q, k, pos, inv, q_weight=torch.zeros(32))
    _raises("out_dtype", rope, q, k, pos, inv, out_dtype=torch.int8)
    _raises("k_out must hold", rope, q, k, pos, inv, k_out=torch.zeros(3))
    _raises("device tensor", rope, q, k, pos, inv)
    cache, slots = torch.zeros((4, 2, 32 * 72), dtype=torch.uint8), torch.zeros(3, dtype=torch.int64)
    _raises("cache must be", tq2.tq2_kv4_store, cache[0], k, k, slots)
    _raises("cache must have dtype", tq2.tq2_kv4_store, cache.to(torch.int8), k, k, slots)
    _raises("no whole number", tq2.tq2_kv4_store, cache[..., :100].contiguous(), k, k, slots)
    _raises("heads", tq2.tq2_kv4_store, cache, q, q, slots)
    _raises("same shape", tq2.tq2_kv4_store, cache, k, q, slots)
    _raises("slots must have dtype", tq2.tq2_kv4_store, cache, k, k, slots.int())
    _raises("slots must hold 3", tq2.tq2_kv4_store, cache, k, k, slots[:1])
    _raises("device tensor", tq2.tq2_kv4_store, cache, k, k, slots)
    _raises("dtype must be", tq2.tq2_kv4_load, cache, slots, 64, dtype=torch.float64)
    _raises("k_out must hold", tq2.tq2_kv4_load, cache, slots, 64, k_out=torch.zeros(5))
    _raises("v_out must have dtype", tq2.tq2_kv4_load, cache, slots, 64, dtype=torch.float16, v_out=torch.zeros(384))
    h, table, ctx = q.half(), torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    attn = tq2.tq2_kv4_attn
    _raises("q must have dtype", attn, q, cache, table, ctx)
    _raises("table must be", attn, h, cache, table.long(), ctx)
    _raises("rows of table", attn, h, cache, table.t().contiguous().t(), ctx)
    _raises("ctx_len must hold 3", attn, h, cache, table, ctx[:2])
    _raises("q_start must hold 4", attn, h, cache, table, ctx, q_start=ctx, max_q=1)
    _raises("needs max_q", attn, h, cache, table, ctx, q_start=torch.zeros(4, dtype=torch.int32))
    _raises("not max_q tokens", attn, h, cache, table, ctx, max_q=2)
    _raises("out must have dtype", attn, h, cache, table, ctx, out=torch.zeros_like(q))
    _raises("lse must hold", attn, h, cache, table, ctx, lse=torch.zeros(3))
    _raises("device tensor", attn, h, cache, table, ctx)


# ---- addresses, bad pages and splits, from the kernels' own header ----

HARNESS = r'''
#include "tq2_kv4.h"
extern "C" {
int64_t unit_at(int P, int D, int t, int u) { return tq2::kv4_value_unit_at(P, D, t, u); }
int64_t key_at(int D, int t) { return tq2::kv4_key_at(D, t); }
int64_t kpair_at(int P, int D, int t) { return tq2::kv4_key_pair_at(P, D, t); }
int64_t vpair_at(int P, int D, int t) { return tq2::kv4_value_pair_at(P, D, t); }
int64_t slot_block(int64_t s, int64_t n, int H, int P, int D, int h, int* t) { return tq2::kv4_slot_block(s, n, H, P, D, h, t); }
int64_t page_block(int32_t p, int64_t n, int H, int P, int D, int h) { return tq2::kv4_page_block(p, n, H, P, D, h); }
void range(int n, int c, int G, int row0, int rows, int window, int ns, int waves, int* o) {
  tq2::Kv4Range r = tq2::kv4_range(n, c, G, row0, rows, window, ns, waves);
  o[0] = r.first, o[1] = r.last, o[2] = r.chunk, o[3] = r.splits;
}
}
'''


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4")
    (d / "h.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", build.CSRC, str(d / "h.cpp"),
                    "-o", str(d / "h.so")], check=True)
    lib = ctypes.CDLL(str(d / "h.so"))
    for f in ("unit_at", "key_at", "kpair_at", "vpair_at", "slot_block", "page_block"):
        getattr(lib, f).restype = ctypes.c_int64
    return lib


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("PP", [32, 64])
def test_every_byte_of_a_block_has_one_owner(layout, D, PP):
    seen = np.zeros(PP * (D + 8), int)
    for t in range(PP):
        seen[layout.key_at(D, t):layout.key_at(D, t) + D // 2] += 1
        for u in range(D // 4):
            at = layout.unit_at(PP, D, t, u)
            assert at == ref.Cache(1, 1, PP, D)._value_byte(t, 4 * u)
            seen[at:at + 2] += 1
        for at in (layout.kpair_at(PP, D, t), layout.vpair_at(PP, D, t)):
            assert at % 4 == 0
            seen[at:at + 4] += 1
    assert np.all(seen == 1)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_loads_stay_in_a_block(layout, D):
    """The loads of a wave for a tile: per lane D/8 bytes of a key in two
    tokens, D/4 bytes of value codes, 32 bytes of pairs each."""
    for PP in (32, 128, 4096):
        whole = PP * (D + 8)
        for t32 in (0, PP - 32):
            keys, values = set(), set()
            for lane in range(64):
                col, g = lane % 16, lane // 16
                for u in (0, 4):
                    at = layout.key_at(D, t32 + (col >> 2) * 8 + (col & 3) + u) + g * (D // 8)
                    assert at % min(16, D // 8) == 0 and 0 <= at and at + D // 8 <= PP * D // 2
                    keys.add(at)
                at = layout.unit_at(PP, D, t32, 0) + lane * (D // 4)
                assert at % 16 == 0 and at + D // 4 <= PP * D
                values.add(at)
                for f in (layout.kpair_at, layout.vpair_at):
                    at = f(PP, D, t32 + g * 8)
                    assert at % 16 == 0 and at + 32 <= whole
            assert len(keys) == 128 and len(values) == 64  # each byte of the tile once


def test_slots_and_pages_that_are_not_there(layout):
    t = ctypes.c_int(-1)
    slot = lambda s, pages=6: layout.slot_block(ctypes.c_int64(s), ctypes.c_int64(pages), 2, 32, 64, 1, ctypes.byref(t))
    assert slot(0) == 32 * 72 and t.value == 0
    assert slot(6 * 32 - 1) == 11 * 32 * 72 and t.value == 31
    for s in (-1, -32, -33, 6 * 32, 1 << 40, -(1 << 63), (1 << 63) - 1):
        assert slot(s) == -1, s
    page = lambda p, pages=6: layout.page_block(ctypes.c_int32(p), ctypes.c_int64(pages), 2, 32, 64, 1)
    assert page(5) == 11 * 32 * 72
    for p in (-1, 6, 2 ** 31 - 1, -2 ** 31):
        assert page(p) == -1
    far = layout.slot_block(ctypes.c_int64((1 << 33) + 5), ctypes.c_int64(1 << 29), 2, 32, 128, 0, ctypes.byref(t))
    assert far == (1 << 28) * 2 * 32 * 136 and t.value == 5  # past 32 bits


def test_splits_cover_what_rows_see_once(layout):
    g = np.random.default_rng(0)
    out = (ctypes.c_int * 4)()
    for _ in range(4000):
        n, G = int(g.integers(1, 40)), int(g.integers(1, 20))
        c = int(g.integers(0, 3000)) if g.random() < 0.8 else int(g.integers(0, 40))
        rows = int(g.choice([16, 32, 64]))
        row0 = rows * int(g.integers(0, -(-n * G // rows)))
        window = 0 if g.random() < 0.5 else int(g.choice([1, 7, 32, 500, 2 ** 31 - 1]))
        ns, waves = int(g.integers(1, 65)), 4
        layout.range(n, c, G, row0, rows, window, ns, waves, out)
        first, last, chunk, splits = out
        i = np.arange(row0 // G, min(n - 1, (row0 + rows - 1) // G) + 1)
        p = c - n + i
        lo = np.maximum(0, p - window + 1) if window else np.zeros_like(p)
        some = (p >= lo) & (p >= 0)
        assert 0 <= splits <= ns
        if not some.any():
            assert splits == 0 or last > first  # an empty range, or tiles that no row sees
            continue
        assert first * 32 <= lo[some].min() and last * 32 > p.max() and last <= -(-c // 32)
        assert chunk % waves == 0 and (splits - 1) * chunk < last - first <= splits * chunk


# ---- the oracles ----

def test_oracle_quantizer():
    x = np.zeros((1, 64), np.float32)
    x[0, :16] = np.arange(16) - 7.5
    c, s, z = ref.quantize(x)
    assert s[0] == 1 and z[0] == 0
    assert list(c[0, :16]) == list(range(16)) and np.all(c[0, 16:] == 8)  # 7.5 ties to 8
    assert np.array_equal(ref.held(c, s, z)[0, :16], x[0, :16].astype(np.float64))
    c, s, z = ref.quantize(np.full((2, 64), 0.375, np.float32))
    assert np.all(c == 0) and np.all(ref.held(c, s, z) == 0.375)
    g = np.random.default_rng(1)
    x = g.standard_normal((50, 128)).astype(np.float32)
    c, s, z = ref.quantize(x)
    # off by half a step, and what rounding s and z to binary16 moves
    assert np.all(np.abs(ref.held(c, s, z) - x) <= (s.astype(np.float64) * (0.5 + 15 * 2.0 ** -11) + 2.0 ** -11)[:, None])


def test_oracle_cache_round_trip():
    g = np.random.default_rng(2)
    cache = ref.Cache(3, 2, 32, 64, fill=0x5a)
    k, v = g.standard_normal((2, 5, 2, 64)).astype(np.float32)
    slots = [95, 0, 40, 33, -1]
    cache.store(k, v, slots)
    for h in range(2):
        for value, x in ((0, k), (1, v)):
            got = cache.tokens(slots[:4], h)[value]
            for a, b in zip(got, ref.quantize(x[:4, h])):
                assert np.array_equal(a, b)
    assert (cache.bytes != 0x5a).sum() <= 4 * 2 * 2 * (32 + 4)


def test_oracle_attention_by_hand():
    cache = ref.Cache(1, 1, 32, 64)
    k, v = np.zeros((2, 3, 1, 64), np.float32)
    k[:, 0, 0], k[:, 0, 1] = [0, 1, 2], [-1, -2, -3]
    v[:, 0, :] = np.array([1, 2, 4])[:, None]
    cache.store(k, v, [0, 1, 2])
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = 1
    kk = ref.held(*cache.tokens([0, 1, 2], 0)[0])[:, 0]
    out, lse, tol, _ = ref.attention(q, cache, np.zeros((1, 1), np.int32), [3], [0, 2], 0.5, 0, 2.0 ** -10)
    for i, n in ((0, 2), (1, 3)):
        w = np.exp(0.5 * kk[:n])
        assert np.allclose(out[i, 0], (w @ [1, 2, 4][:n]) / w.sum(), atol=1e-12) and np.isclose(lse[i, 0], np.log(w.sum()))
    assert np.all(tol > 0)
    out, lse, _, _ = ref.attention(q, cache, np.zeros((1, 1), np.int32), [1], [0, 2], 0.5, 0, 2.0 ** -10)
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and np.allclose(out[1], 1)
    out, _, _, _ = ref.attention(q, cache, np.zeros((1, 1), np.int32), [3], [0, 2], 0.5, 1, 2.0 ** -10)
    assert np.allclose(out[0, 0], 2) and np.allclose(out[1, 0], 4)


def test_oracle_rotation():
    g = np.random.default_rng(3)
    x, inv = g.standard_normal((4, 2, 32)), np.array([1.0, 0.5, 0.25, 0.125] * 2, np.float32)
    for inter in (False, True):
        y, _ = ref.norm_rope(x, None, 0.0, [0, 3, 10, 10 ** 6], inv, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[0], x[0])
        assert np.array_equal(y[..., 16:], x[..., 16:])
        back, _ = ref.norm_rope(y, None, 0.0, [0, -3, -10, -10 ** 6], inv, inter)
        assert np.allclose(back, x)
    y, _ = ref.norm_rope(x, np.full(32, 2.0), 0.0, [0] * 4, inv, False)
    assert np.allclose((y ** 2).mean(-1), 4)
