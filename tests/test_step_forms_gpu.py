"""The gated projections at the sizes that each form takes (by tokens, by the
workgroups that the GPU holds at once, by the workspace), and the calls of the
feed-forward half on streams, in graphs and with places of their own."""
import numpy as np
import pytest

from oracle import step as ref
from tests.test_step_gpu import BF16, DEV, F16, F32, f32, f64, feed_forward, gated_tol, layer, magnitudes, tq2  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def drawn(N, K, g):
    """Packed weights on the device, a row's least and largest scales far apart."""
    codes = torch.randint(0, 256, (N, K // 4), generator=g, device=DEV, dtype=torch.uint8)
    codes &= ~((codes >> 1) & codes & 0x55) & 0xFF  # code 3 becomes 2
    scales = (0.002 + 0.06 * torch.rand((N, K // 256), generator=g, device=DEV)).half()
    return codes, scales


def some(n, most, g):
    """All of 0 .. n - 1, or `most` of them: both ends, and others between."""
    if n <= most:
        return np.arange(n)
    ends = most // 3
    return np.unique(np.concatenate([np.arange(ends), np.arange(n - ends, n), g.integers(0, n, ends)]))


def check(tq2, M, N, K, i8, dst):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(M + N + K)
    gate, up = drawn(N, K, g), drawn(N, K, g)
    x = torch.randn((M, K), generator=g, device=DEV)
    x[:, ::97] *= 10
    out = torch.full((M * N + 64,), 7.0, dtype=dst, device=DEV)
    h = out[:M * N].view(M, N)
    n, m = (some(k, most, np.random.default_rng(K)) for k, most in ((N, 240), (M, 72)))
    if i8:
        s = (x.abs().amax(-1) / 127).float() if i8 == "token" else torch.full((M,), 0.02, device=DEV)
        x = (x / s[:, None]).round().clamp(-128, 127).to(torch.int8)
        x[0, 0] = -128
        tq2.tq2_gemm_i8q_gate_up_silu(*gate, *up, x, s if i8 == "token" else 0.02, h=h)
        unit = f64(s)[m, None] if i8 == "token" else float(np.float32(0.02))
    else:
        x = x.half()
        tq2.tq2_gemm_gate_up_silu(*gate, *up, x, h=h)
        unit = 1.0
    torch.cuda.synchronize()
    assert bool((out[M * N:] == 7.0).all())
    x64 = f64(x[torch.from_numpy(m).to(DEV)])
    at = torch.from_numpy(n).to(DEV)
    wg, wu = (ref.dense(c[at].cpu().numpy(), s[at].cpu().numpy()) for c, s in (gate, up))
    want, gs, us, *_ = ref.gated(wg, wu, x64 * unit)
    tol = gated_tol(gs, us, magnitudes(wg, x64) * unit, magnitudes(wu, x64) * unit, want, K, dst)
    err = np.abs(f64(h[torch.from_numpy(m).to(DEV)][:, at]) - want)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(~(err <= tol))[:5])


# rows that fill the GPU with 64, 32 and 16 of them a workgroup; K with more
# scales than are asked for ahead; 32, 64 and 128 tokens a workgroup whose waves
# share K, and more workgroups than run at once
@pytest.mark.parametrize("M,N,K,dst", [
    (1, 12400, 768, F16), (16, 12305, 1024, F32), (5, 6200, 2560, BF16), (13, 12300, 8704, F16), (2, 12300, 65536, F32),
    (9, 6150, 33024, F32), (24, 16400, 768, F16), (32, 5000, 256, F32), (100, 9000, 1024, F32), (300, 4000, 768, BF16),
    (129, 8100, 256, F16), (600, 4100, 1280, F32), (257, 8203, 256, F16), (130, 16500, 512, BF16), (700, 8200, 2304, F16)])
def test_gated_forms(tq2, M, N, K, dst):  # noqa: F811
    check(tq2, M, N, K, None, dst)


# 64 rows and the longest K whose scales find room beside their codes, and the
# next; rows' last blocks alone; one token over one, two and four waves a row and more than once around
@pytest.mark.parametrize("M,N,K,dst", [
    (14, 12300, 32768, F32), (48, 16400, 768, F32), (33, 33000, 256, F16), (64, 8192, 512, F32), (61, 700, 16640, F32), (30, 33000, 256, F32), (16, 12300, 33024, F16), (13, 12290, 4352, F32), (3, 6146, 2304, F32), (2, 300, 16640, F32),
    (1, 6150, 4352, F32), (1, 999, 8448, F16), (1, 1000, 12544, F32), (1, 35, 33024, BF16), (1, 17, 65536, F32)])
def test_gated_few_tokens_and_long_rows(tq2, M, N, K, dst):  # noqa: F811
    check(tq2, M, N, K, None, dst)


@pytest.mark.parametrize("kind", ["static", "token"])
@pytest.mark.parametrize("M,N,K,dst", [
    (1, 12400, 768, F16), (16, 12305, 8704, F32), (20, 6200, 1024, BF16), (32, 6150, 33024, F32), (9, 6150, 512, F16),
    (17, 3000, 256, F32), (33, 16400, 768, F16), (600, 8300, 512, F32), (520, 8301, 256, BF16), (64, 33000, 1280, F16)])
def test_gated_forms_i8(tq2, M, N, K, dst, kind):  # noqa: F811
    check(tq2, M, N, K, kind, dst)


@pytest.mark.parametrize("kind", ["static", "token"])
@pytest.mark.parametrize("M,N,K", [(700, 100, 65280), (1030, 8300, 33280)])
def test_gated_i8_in_parts_of_the_workspace(tq2, M, N, K, kind):  # noqa: F811
    """More tokens than their pieces find room for at once."""
    need = tq2.tq2_gemm_i8q_gate_up_silu_workspace_bytes(N, K, M)
    assert need <= 48 << 20 and M * K * 3 // 2 > need
    check(tq2, M, N, K, kind, F32)


def test_one_matrix_as_gate_and_up(tq2):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(3)
    m = drawn(200, 512, g)
    for M in (1, 40, 200):
        x = torch.randn((M, 512), generator=g, device=DEV).half()
        h = tq2.tq2_gemm_gate_up_silu(*m, *m, x, out_dtype=F32)
        y = x.double() @ torch.from_numpy(ref.dense(*(t.cpu().numpy() for t in m))).to(DEV).T
        want = torch.nn.functional.silu(y) * y
        assert torch.allclose(h.double(), want, rtol=1e-4, atol=1e-4)


# ---- streams, graphs, places ----

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


def inputs(M, i8, D=512, N=1280, V=70000, seed=0):
    g = torch.Generator().manual_seed(seed + M)
    w = layer(g, D, N, V)
    return {"w": w, "i8": i8, "M": M, "N": N, "o": torch.randn((M, D), generator=g).to(DEV),
            "h": (2 * torch.randn((M, D), generator=g)).to(BF16).to(DEV), "tokens": torch.randint(V, (M,), generator=g).to(DEV),
            "logits": (4 * torch.randn((M, V), generator=g)).to(DEV), "top": 6, "V": V, "D": D}


def places(tq2, e):  # noqa: F811
    M, D, N = e["M"], e["D"], e["N"]

    def bytes_of(n):
        return torch.empty(n, dtype=torch.uint8, device=DEV) if n else None

    size = tq2.tq2_gemm_i8q_gate_up_silu_workspace_bytes if e["i8"] else tq2.tq2_gemm_gate_up_silu_workspace_bytes
    return {"y": torch.empty((M, D), dtype=torch.int8 if e["i8"] else F16, device=DEV), "s": torch.empty(M, device=DEV),
            "h": torch.empty_like(e["h"]), "a": torch.empty((M, N), dtype=F16, device=DEV), "gws": bytes_of(size(N, D, M)),
            "lp": torch.empty(M, device=DEV), "H": torch.empty(M, device=DEV),
            "tt": torch.empty((M, e["top"]), dtype=torch.int64, device=DEV), "tl": torch.empty((M, e["top"]), device=DEV),
            "lws": bytes_of(tq2.tq2_token_logprobs_workspace_bytes(M, e["V"], e["top"]))}


def calls(tq2, e, stream=None, p=None):  # noqa: F811
    """The calls one after another, into the places p or into new ones."""
    w, p = e["w"], p or dict.fromkeys(("y", "s", "h", "a", "gws", "lp", "H", "tt", "tl", "lws"))
    if e["i8"]:
        y, s, h = tq2.tq2_add_rms_norm_i8(e["o"], e["h"], w["w1"], h_out=p["h"], x_q=p["y"], x_scales=p["s"], stream=stream)
        a = tq2.tq2_gemm_i8q_gate_up_silu(*w["gate"], *w["up"], y, s, h=p["a"], ws=p["gws"], stream=stream)
    else:
        y, h = tq2.tq2_add_rms_norm(e["o"], e["h"], w["w1"], h_out=p["h"], out=p["y"], stream=stream)
        a = tq2.tq2_gemm_gate_up_silu(*w["gate"], *w["up"], y, h=p["a"], ws=p["gws"], stream=stream)
    return [y, h, a, *tq2.tq2_token_logprobs(e["logits"], e["tokens"], top=e["top"], want_entropy=True, logprobs=p["lp"],
                                             entropy=p["H"], top_tokens=p["tt"], top_logprobs=p["tl"], ws=p["lws"],
                                             stream=stream)]


CASES = [(1, False), (1, True), (24, False), (40, True), (140, False), (520, True)]


@pytest.mark.parametrize("M,i8", CASES)
def test_given_places_are_the_same_call(tq2, M, i8):  # noqa: F811
    e = inputs(M, i8)
    want = calls(tq2, e)
    for _ in range(2):
        p = places(tq2, e)
        got = calls(tq2, e, None, p)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert got[0] is p["y"] and got[2] is p["a"] and got[4] is p["H"] and got[6] is p["tl"]


@pytest.mark.parametrize("M,i8", CASES)
def test_calls_on_a_given_stream(tq2, M, i8):  # noqa: F811
    e = inputs(M, i8, seed=1)
    want = calls(tq2, e)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for p in (None, places(tq2, e)):
        behind(side)
        got = calls(tq2, e, side, p)
        tread(*(t.nbytes for t in got), 1 << 20)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("i8", [False, True])
def test_two_streams_at_once(tq2, i8):  # noqa: F811
    """Each with outputs and workspaces of its own."""
    each = [inputs(M, i8, seed=2) for M in (90, 200)]
    want = [calls(tq2, e) for e in each]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in each]
    put = [places(tq2, e) for e in each]
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for e, side, p in zip(each, sides, put):
            calls(tq2, e, side, p)
    got = [calls(tq2, e, side, p) for e, side, p in zip(each, sides, put)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("M,i8", CASES)
def test_two_graphs_that_share_places(tq2, M, i8):  # noqa: F811
    """Captured on a stream that the calls are given too; one set of outputs and
    workspaces for both, replayed in turn."""
    e = [inputs(M, i8, seed=s) for s in (3, 4)]
    p = places(tq2, e[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in e]
    for one, graph in zip(e, graphs):
        with torch.cuda.graph(graph, stream=side):
            got = calls(tq2, one, side, p)
    g = torch.Generator().manual_seed(9)
    for it in range(4):
        for one, graph in zip(e, graphs):
            one["o"].copy_(torch.randn(one["o"].shape, generator=g))
            one["logits"].mul_(-0.9)
            one["tokens"].add_(1)
            graph.replay()
            torch.cuda.synchronize()
            have = [t.clone() for t in got]
            want = calls(tq2, one)
            tread(1 << 22)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(have, want)), it


@pytest.mark.parametrize("i8", [False, True])
def test_the_chain_after_a_graph_of_itself(tq2, i8):  # noqa: F811
    """A graph captured with new places inside, eager chains before and after it unchanged."""
    e = inputs(33, i8, V=1000, seed=5)
    before = feed_forward(tq2, e["w"], e["o"], e["h"], e["tokens"], i8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = feed_forward(tq2, e["w"], e["o"], e["h"], e["tokens"], i8)
    for _ in range(3):
        graph.replay()
        after = feed_forward(tq2, e["w"], e["o"], e["h"], e["tokens"], i8)
        torch.cuda.synchronize()
        for a, b, c in zip(before, inside, after):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_rows_behind_the_last_stay(tq2):  # noqa: F811
    """Outputs of T rows in larger tensors: what lies behind them is left."""
    g = torch.Generator().manual_seed(6)
    for T, D, V in ((1, 72, 100), (3, 4096, 70000), (600, 264, 3001)):
        x = torch.randn((T, D), generator=g).to(DEV)
        out, h = torch.full((T + 1, D), 9.0, device=DEV), torch.full((T + 1, D), 9.0, device=DEV)
        tq2.tq2_add_rms_norm(x, x, h_out=h[:T], out=out[:T])
        q, s = torch.full((T + 1, D), 99, dtype=torch.int8, device=DEV), torch.full((T + 1,), 9.0, device=DEV)
        tq2.tq2_add_rms_norm_i8(x, x_q=q[:T], x_scales=s[:T])
        lg = torch.randn((T, V), generator=g).to(DEV)
        lp, H = torch.full((T + 1,), 9.0, device=DEV), torch.full((T + 1,), 9.0, device=DEV)
        tt, tl = torch.full((T + 1, 3), -7, device=DEV), torch.full((T + 1, 3), 9.0, device=DEV)
        tq2.tq2_token_logprobs(lg, torch.zeros(T, dtype=torch.int64, device=DEV), top=3, logprobs=lp[:T], entropy=H[:T],
                               top_tokens=tt[:T], top_logprobs=tl[:T])
        torch.cuda.synchronize()
        for t in (out, h, s, lp, H, tl):
            assert bool((t[T:] == 9.0).all()) and not bool((t[:T] == 9.0).all())
        assert bool((q[T:] == 99).all()) and bool((tt[T:] == -7).all())
        assert np.array_equal(tt[:T].cpu().numpy(), ref.top_tokens(f32(lg), 3))
