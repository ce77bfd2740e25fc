"""Calls on a stream that the caller gives, while that stream is behind and the
current one goes on: every call's outputs and workspace are its own until its
kernels have run."""
import numpy as np
import pytest

from tests.test_kv4_gpu import filled, layer_inputs, layer_step, set_place

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
F16 = torch.float16


@pytest.fixture(scope="module")
def tq2():
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import tq2 as mod
    return mod


def behind(stream):
    """A few milliseconds of products on the stream."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        a = torch.ones((4096, 4096), device=DEV)
        for _ in range(8):
            a = a @ a * 2.0 ** -12


def tread(*sizes):
    """The current stream takes memory of these sizes, as often as it likes, and writes all of it."""
    for n in sizes:
        for _ in range(4):
            torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("handle", ["long", "short"])
def test_step_on_a_given_stream(tq2, handle):
    """All four calls with stream=: the short way (outputs and workspace given) and the long one."""
    s, e = layer_inputs(2), layer_inputs(2)
    for x in (s, e):
        set_place(x, 4)
    layer_step(tq2, e)
    want = tq2.tq2_kv4_load(e["cache"], e["slots"], e["D"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    behind(side)
    if handle == "short":
        s["v"].copy_(s["qkv"][:, s["Hq"] + s["Hk"]:])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):       # the copy inside the step
            layer_step(tq2, s, stream=side)
        got = tq2.tq2_kv4_load(s["cache"], s["slots"], s["D"], k_out=torch.empty_like(s["k"]),
                               v_out=torch.empty_like(s["v"]), stream=side)
        out = s["out"]
    else:
        Hq, Hk = s["Hq"], s["Hk"]
        q, k = tq2.tq2_qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hk], s["pos"], s["inv"], out_dtype=F16, stream=side)
        with torch.cuda.stream(side):
            v = s["qkv"][:, Hq + Hk:].half()
        tq2.tq2_kv4_store(s["cache"], k, v, s["slots"], stream=side)
        out = tq2.tq2_kv4_attn(q, s["cache"], s["table"], s["ctx"], stream=side)
        got = tq2.tq2_kv4_load(s["cache"], s["slots"], s["D"], stream=side)
    tread(out.nbytes, got[0].nbytes)
    torch.cuda.synchronize()
    assert torch.equal(out, e["out"]) and torch.equal(s["cache"], e["cache"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("B,S,G,width", [(3, 1, 16, 600), (2, 130, 16, 300)])
def test_attention_workspace_of_a_given_stream(tq2, B, S, G, width):
    """A workspace that the call allocates (part sums, groups and a list for
    many rows) holds until the stream has come to it, and the current stream's
    next tensors are others."""
    Hk, D, P = 1, 64, 32
    cache, g = filled(3, 700, Hk, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    table = torch.from_numpy(g.integers(0, 700, (B, width)).astype(np.int32)).to(DEV)
    ctx = torch.tensor([width * P - 7 * b for b in range(B)], dtype=torch.int32, device=DEV)
    q = torch.from_numpy(g.standard_normal((B * S, G * Hk, D))).to(F16).to(DEV)
    need = tq2.tq2_kv4_attn_workspace_bytes(B * S, G * Hk, Hk, D, P, width, B, S)
    assert need > 0
    want = tq2.tq2_kv4_attn(q, c, table, ctx)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        behind(side)
        out = tq2.tq2_kv4_attn(q, c, table, ctx, stream=side)
        tread(need, out.nbytes)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_batched_product_workspace_of_a_given_stream(tq2):
    N, K, M = 1024, 4096, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    m = tq2.tq2_pack(torch.randint(-1, 2, (N, K), generator=g, device=DEV).float())[:2]
    x = torch.randn((M, K), generator=g, device=DEV).half()
    xq = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    runs = [(lambda s: tq2.tq2_gemm(*m, x, stream=s), tq2.tq2_gemm_workspace_bytes(N, K, M)),
            (lambda s: tq2.tq2_gemm_i8q(*m, xq, 0.05, stream=s), tq2.tq2_gemm_i8q_workspace_bytes(N, K, M))]
    side = torch.cuda.Stream()
    for run, need in runs:
        assert need > 0
        want = run(None)
        torch.cuda.synchronize()
        behind(side)
        y = run(side)
        tread(need, y.nbytes)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_calls_on_the_stream_of_a_capture(tq2):
    """A graph captured on a stream that the calls are given too, outputs and
    workspace allocated inside; replays against eager calls."""
    Hk, G, D, P, width = 2, 8, 64, 32, 60
    cache, g = filled(5, 130, Hk, P, D)
    c = torch.from_numpy(cache.bytes).to(DEV)
    table = torch.from_numpy(g.integers(0, 130, (2, width)).astype(np.int32)).to(DEV)
    ctx = torch.tensor([1, 1], dtype=torch.int32, device=DEV)
    x = torch.zeros((2, Hk * G + Hk, D), device=DEV)
    pos, inv = torch.zeros(2, dtype=torch.int32, device=DEV), torch.rand(D // 2, device=DEV)

    def step(stream):
        q, k = tq2.tq2_qk_norm_rope(x[:, :Hk * G], x[:, Hk * G:], pos, inv, out_dtype=F16, stream=stream)
        return tq2.tq2_kv4_attn(q, c, table, ctx, stream=stream), k

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, k = step(side)
    for it in range(5):
        x.copy_(torch.from_numpy(g.standard_normal(x.shape)))
        pos.fill_(it)
        ctx.copy_(torch.tensor([width * P - 3 * it, 40 + it]))
        graph.replay()
        torch.cuda.synchronize()
        want, wk = step(None)
        tread(out.nbytes, 1 << 20)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(k, wk), it
