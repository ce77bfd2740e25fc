"""The feed-forward half of a decode step and the answer without a GPU:
refusals of the C ABI and of the binding, and pins of the oracles."""
import ctypes
import math
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import step as ref
from ternary_packed_weight_amd import build

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device addresses are only safe to pass where no GPU exists")
A = 1 << 40  # fake, aligned, never dereferenced
M = 1 << 32
BAD = 2 ** 64 - 1


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
def test_norm_refusals(tq2):
    def f(x=A, xs=4096, xd=2, r=A + M, rs=4096, rd=1, h=A + 2 * M, T=4, D=4096, w=A + 3 * M, eps=1e-6, out=A + 4 * M, od=0):
        return tq2.lib().tq2_add_rms_norm(P(x), xs, xd, P(r), rs, rd, P(h), T, D, P(w), eps, P(out), od, None)

    assert f(T=0) == 0 and f(T=-1) == 1
    assert f(x=0) == 1 and f(out=0) == 1 and f(r=0) == 1  # a sum without a residual
    assert f(xd=3) == 1 and f(xd=-1) == 1 and f(rd=3) == 1 and f(od=3) == 1 and f(od=-1) == 1
    assert f(eps=-1.0) == 1 and f(eps=math.nan) == 1 and f(eps=math.inf) == 1
    assert f(D=0) == 2 and f(D=4) == 2 and f(D=100) == 2 and f(D=65544) == 2 and f(T=(1 << 26) + 1) == 2
    assert f(xs=-1) == 1 and f(rs=-16) == 1 and f(xs=1 << 41) == 2 and f(rs=1 << 41) == 2
    assert f(x=A + 8) == 3 and f(r=A + M + 2) == 3 and f(h=A + 2 * M + 8) == 3 and f(out=A + 4 * M + 4) == 3
    assert f(w=A + 3 * M + 8) == 3 and f(xs=4098) == 3 and f(rs=4100) == 3
    assert f(rs=4088) == 1                                   # rows of the sum in each other
    assert f(h=A + M + 16) == 1 and f(h=A) == 1              # the sum over a part of the residual, over x
    assert f(out=A) == 1 and f(out=A + M) == 1 and f(out=A + 2 * M + 4096) == 1 and f(out=A + 3 * M) == 1
    assert f(out=A - 4 * 4096 * 2 + 16) == 1 and f(w=A + 2 * M) == 1


@no_gpu
def test_norm_i8_refusals(tq2):
    def f(x=A, r=0, h=0, T=4, D=64, s=0.5, q=A + 4 * M, sc=0, w=0, eps=1e-6):
        return tq2.lib().tq2_add_rms_norm_i8(P(x), 64, 0, P(r), 64, 0, P(h), T, D, P(w), eps, s, P(q), P(sc), None)

    assert f(s=0.0) == 5 and f(s=-1.0) == 5 and f(s=math.inf) == 5 and f(s=math.nan) == 5
    assert f(s=0.5, sc=A + M) == 1                           # one scale, or one a row
    assert f(T=0) == 0 and f(q=0) == 1 and f(q=A + 4 * M + 8) == 3 and f(s=0.0, sc=A + M + 2) == 3
    assert f(h=A + M) == 1                                   # a sum without a residual
    assert f(s=0.0, sc=A) == 1 and f(s=0.0, sc=A + 4 * M + 252) == 1 and f(q=A + 256) == 1
    assert f(D=12) == 2 and f(eps=-0.5) == 1


@no_gpu
@pytest.mark.parametrize("i8", [False, True])
def test_gated_refusals(tq2, i8):
    lib = tq2.lib()

    def f(cg=A, sg=A + M, cu=A + 2 * M, su=A + 3 * M, N=64, K=512, x=A + 4 * M, m=5, s=0.5, xs=0, h=A + 5 * M, hd=0, ws=0, wb=0):
        if i8:
            return lib.tq2_gemm_i8q_gate_up_silu(P(cg), P(sg), P(cu), P(su), N, K, P(x), m, s, P(xs), P(h), hd, P(ws), wb, None)
        return lib.tq2_gemm_gate_up_silu(P(cg), P(sg), P(cu), P(su), N, K, P(x), m, P(h), hd, P(ws), wb, None)

    size = lib.tq2_gemm_i8q_gate_up_silu_workspace_bytes if i8 else lib.tq2_gemm_gate_up_silu_workspace_bytes
    most = 65280 if i8 else 65536
    assert f(N=0) == 1 and f(m=0) == 1 and f(N=-1) == 1
    assert f(K=0) == 2 and f(K=128) == 2 and f(K=300) == 2 and f(K=most + 256) == 2 and f(m=65537) == 2
    assert f(N=(1 << 26) + 1, K=256) == 2 and f(N=1 << 26, K=65280) == 2 and f(N=1 << 26, K=256, m=65536) == 2
    for name in ("cg", "sg", "cu", "su", "x", "h"):
        assert f(**{name: 0}) == 1
    assert f(hd=3) == 1 and f(hd=-1) == 1
    assert f(cg=A + 8) == 3 and f(cu=A + 2 * M + 4) == 3 and f(sg=A + M + 1) == 3 and f(x=A + 4 * M + 8) == 3 and f(h=A + 5 * M + 8) == 3
    for at in (A, A + M, A + 2 * M, A + 3 * M, A + 4 * M):
        assert f(h=at) == 1
    if i8:
        assert f(s=0.0) == 5 and f(s=-2.0) == 5 and f(s=math.nan) == 5 and f(s=0.5, xs=A + 6 * M) == 1
        assert f(s=0.0, xs=A + 6 * M + 2) == 3 and f(s=0.0, xs=A + 5 * M) == 1
    assert size(0, 256, 1) == BAD and size(1, 100, 1) == BAD and size(1, most + 256, 1) == BAD and size(1, 256, 0) == BAD
    assert size(64, 512, 5) != BAD


@no_gpu
def test_logprobs_refusals(tq2):
    def f(x=A, st=5000, dt=2, T=600, V=5000, scale=1.0, tok=A + M, lp=A + 2 * M, H=A + 3 * M, top=4, tt=A + 4 * M, tl=A + 5 * M,
          ws=0, wb=0):
        return tq2.lib().tq2_token_logprobs(P(x), st, dt, T, V, scale, P(tok), P(lp), P(H), top, P(tt), P(tl), P(ws), wb, None)

    assert f(T=0) == 0 and f(T=-1) == 1 and f(V=0) == 1 and f(top=-1) == 1 and f(st=-1) == 1 and f(dt=3) == 1
    assert f(scale=0.0) == 5 and f(scale=-1.0) == 5 and f(scale=math.inf) == 5 and f(scale=math.nan) == 5
    assert f(top=65) == 2 and f(V=3, top=4) == 2 and f(V=(1 << 24) + 1) == 2 and f(T=(1 << 22) + 1) == 2 and f(st=1 << 41) == 2
    assert f(x=0) == 1 and f(tok=0) == 1 and f(lp=0) == 1 and f(tt=0) == 1 and f(tl=0) == 1
    assert f(top=0) == 1 and f(top=0, tt=0) == 1             # places for tokens that are not asked for
    assert f(tok=0, lp=0, H=0, top=0, tt=0, tl=0) == 1       # nothing asked for
    assert f(x=A + 2) == 3 and f(tok=A + M + 4) == 3 and f(lp=A + 2 * M + 2) == 3 and f(tt=A + 4 * M + 4) == 3
    assert f(lp=A) == 1 and f(H=A + 2 * M) == 1 and f(tl=A + 4 * M + 8) == 1 and f(tt=A + M) == 1
    need = tq2.tq2_token_logprobs_workspace_bytes(1, 100000, 4)
    assert 0 < need < BAD
    one = dict(T=1, V=100000, ws=A + 6 * M, wb=need)
    assert f(**{**one, "ws": 0}) == 4 and f(**{**one, "wb": need - 1}) == 4 and f(**{**one, "ws": A + 6 * M + 16}) == 4
    assert f(**{**one, "ws": A}) == 4 and f(**{**one, "ws": A + 2 * M}) == 4


def test_logprobs_workspace(tq2):
    size = tq2.tq2_token_logprobs_workspace_bytes
    assert size(0, 100, 1) == 0 and size(512, 100000, 64) == 0 and size(1, 100, 1) == 0
    assert size(1, 0, 0) == BAD and size(-1, 100, 0) == BAD and size(1, 100, 65) == BAD and size(1, 10, 11) == BAD
    for T in (1, 7, 511):  # enough for `top` more keys of every part
        assert size(T, 200000, 64) > size(T, 200000, 1) > size(T, 200000, 0) > 0


# ---- refusals of the binding ----

def refused(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_binding_refusals_norm(tq2):
    x, w = torch.zeros((3, 64)), torch.ones(64)
    for f in (tq2.tq2_add_rms_norm, tq2.tq2_add_rms_norm_i8):
        refused("device tensor", f, x)
        refused(r"x must be a \[T, D\]", f, x[0])
        refused("x must have dtype", f, x.double())
        refused("contiguous", f, torch.zeros((64, 3)).t())
        refused("residual must be", f, x, torch.zeros((3, 72)))
        refused("residual must hold 3 rows", f, x, torch.zeros((2, 64)))
        refused("weight must hold 64", f, x, None, torch.ones(63))
        refused("weight must have dtype", f, x, None, w.half())
        refused("h_out needs a residual", f, x, h_out=torch.zeros_like(x))
        refused("h_out must have the shape and dtype", f, x, x, h_out=x.half())
        refused("row stride of the residual", f, x, x, h_out=torch.zeros((3, 72))[:, :64])
        refused("strided rows", f, x, torch.zeros((3, 72))[:, :64])
    refused("out must have dtype", tq2.tq2_add_rms_norm, x, out=torch.zeros((3, 64)), out_dtype=torch.float16)
    refused("out_dtype", tq2.tq2_add_rms_norm, x, out_dtype=torch.int8)
    refused("x_q must have dtype", tq2.tq2_add_rms_norm_i8, x, x_q=torch.zeros((3, 64)))
    refused("x_scales must hold 3", tq2.tq2_add_rms_norm_i8, x, x_scales=torch.zeros(2))
    refused("x_scales is written", tq2.tq2_add_rms_norm_i8, x, s=0.5, x_scales=torch.zeros(3))
    for s in (0.0, -1.0, math.nan):
        with pytest.raises(tq2.Tq2Error):
            tq2.tq2_add_rms_norm_i8(x, s=s)


def test_binding_refusals_gated(tq2):
    c, s = torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.float16)
    x, q = torch.zeros((3, 256), dtype=torch.float16), torch.zeros((3, 256), dtype=torch.int8)
    f, i = tq2.tq2_gemm_gate_up_silu, tq2.tq2_gemm_i8q_gate_up_silu
    refused("device tensor", f, c, s, c, s, x)
    refused("device tensor", i, c, s, c, s, q, 0.5)
    refused("same shape", f, c, s, c[:4].contiguous(), s[:4].contiguous(), x)
    refused(r"x must be a \[M, 256\]", f, c, s, c, s, x[:, :128])
    refused("x must have dtype", f, c, s, c, s, x.float())
    refused("x must have dtype", i, c, s, c, s, x, 0.5)
    refused("contiguous", f, c, s, c, s, torch.zeros((256, 3), dtype=torch.float16).t())
    refused("h must hold 24", f, c, s, c, s, x, h=torch.zeros((3, 7)))
    refused("h must have dtype", f, c, s, c, s, x, h=torch.zeros((3, 8)), out_dtype=torch.float16)
    refused("out_dtype", f, c, s, c, s, x, out_dtype=torch.int8)
    refused("s must hold 3", i, c, s, c, s, q, torch.zeros(4))
    refused("s must have dtype", i, c, s, c, s, q, torch.zeros(3, dtype=torch.float64))
    refused("s must be a number", i, c, s, c, s, q, None)


def test_binding_refusals_logprobs(tq2):
    f, x, t = tq2.tq2_token_logprobs, torch.zeros((3, 100)), torch.zeros(3, dtype=torch.int64)
    refused("device tensor", f, x, t)
    refused("logits must be", f, x[0])
    refused("logits must have dtype", f, x.double())
    refused("contiguous", f, torch.zeros((100, 3)).t())
    refused("tokens must hold 3", f, x, t[:2])
    refused("tokens must have dtype", f, x, t.int())
    refused("logprobs needs tokens", f, x, logprobs=torch.zeros(3))
    refused("top_tokens and top_logprobs need top", f, x, t, top_tokens=torch.zeros((3, 1), dtype=torch.int64))
    refused("top_tokens must hold 6", f, x, t, top=2, top_tokens=torch.zeros((3, 1), dtype=torch.int64))
    refused("top_tokens must have dtype", f, x, t, top=2, top_tokens=torch.zeros((3, 2), dtype=torch.int32))
    refused("entropy must hold 3", f, x, t, entropy=torch.zeros(4))


# ---- pins of the oracles ----

def test_oracle_norm_against_rationals():
    x = np.array([[3.0, -4.0, 12.0, 0.0]], np.float32)
    y = ref.rms_norm(x, [1.0, 2.0, 1.0, 1.0], 0.0)   # root of 169/4: 6.5
    assert np.allclose(y[0], [3 / 6.5, -8 / 6.5, 12 / 6.5, 0], rtol=1e-15)
    assert np.allclose(ref.rms_norm_steps(x, None, 0.0), y / [1, 2, 1, 1], rtol=3 * 2.0 ** -24)
    h = ref.norm_sum([[1.0, 2.0 ** -30]], [[1.0, 1.0]], lambda a: a.astype(np.float16).astype(np.float32))
    assert h.tolist() == [[2.0, 1.0]] and ref.norm_sum([[0.5]], None, None).tolist() == [[0.5]]


def test_oracle_codes():
    y = np.array([[0.5, -0.5, 1.5, -1.5, 2.5, 126.5, -127.0, 127.0]], np.float32)
    c, s = ref.codes8(y)
    assert s[0] == 1 and c[0].tolist() == [0, 0, 2, -2, 2, 126, -127, 127]  # ties to even
    assert ref.codes8(y * 2, 1.0)[0][0].tolist() == [1, -1, 3, -3, 5, 127, -128, 127]
    c, s = ref.codes8(np.zeros((2, 4), np.float32))
    assert not c.any() and not s.any()


def test_oracle_gated_against_rationals():
    g = np.random.default_rng(3)
    codes, scales = g.integers(0, 256, (2, 64), dtype=np.uint8), g.random((2, 1)).astype(np.float16)
    w = ref.dense(codes, scales)
    for n in range(2):
        for k in (0, 1, 2, 3, 77, 255):
            q = int(codes[n, k // 4]) >> (2 * (k % 4)) & 3
            assert Fraction(float(w[n, k])) == Fraction(float(scales[n, 0])) * (q - 1)
    x = g.standard_normal((1, 256))
    h, a, u, ma, mu = ref.gated(w[:1], w[1:], x)
    ax = sum(Fraction(float(p)) * Fraction(float(q)) for p, q in zip(w[0], x[0]))
    ux = sum(Fraction(float(p)) * Fraction(float(q)) for p, q in zip(w[1], x[0]))
    assert abs(a[0, 0] - float(ax)) < 1e-13 and abs(u[0, 0] - float(ux)) < 1e-13
    assert math.isclose(h[0, 0], float(ax) / (1 + math.exp(-float(ax))) * float(ux), rel_tol=1e-12)
    assert ma[0, 0] >= abs(a[0, 0]) and ref.silu(np.array([0.0, 800.0, -800.0])).tolist() == [0, 800, 0]


def test_oracle_logprobs():
    lp, H = ref.logprobs([[0.0, 0.0, 0.0, 0.0], [math.log(3), 0.0, -math.inf, -math.inf]])
    assert np.allclose(lp[0], -math.log(4)) and math.isclose(H[0], math.log(4))
    assert np.allclose(lp[1][:2], [math.log(0.75), math.log(0.25)]) and np.isneginf(lp[1][2:]).all()
    assert math.isclose(H[1], -0.75 * math.log(0.75) - 0.25 * math.log(0.25))
    lp, H = ref.logprobs([[-math.inf] * 3, [0.0, math.inf, 1.0], [math.nan, 0.0, 1.0]])
    assert np.isneginf(lp[0]).all() and H[0] == 0 and np.isnan(lp[1:]).all() and np.isnan(H[1:]).all()
    half, _ = ref.logprobs([[2.0, 0.0]], 0.5)
    assert math.isclose(half[0, 1], -math.log(1 + math.e))
    assert ref.top_tokens([[1.0, 3.0, 3.0, -1.0, 0.0], [0.0, -0.0, 0.0, -math.inf, -math.inf]], 4).tolist() == [[1, 2, 0, 4], [0, 1, 2, 3]]
    assert ref.top_tokens([[math.nan, 1.0]], 1).tolist() == [[-1]]
