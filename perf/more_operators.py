"""The feed-forward half of a decode step and the model's answer, operator by operator: what is measured.

Three operators stand around the ternary projections of a layer that follow
its attention, and behind the last layer:

  norm     the residual's addition and RMS norm, in floating point or in 8
           bits with one scale, or a scale a token (what the projections read)
  gated    the gate and up projections, SiLU and the product, for any number
           of tokens, with fp16 or 8-bit activations (what the down
           projection reads)
  answer   log probabilities of given tokens, the entropy, and the likeliest
           tokens of rows of logits

With `own` false `run` computes the plain form in elementary torch operations
(32 bits; 64 where a code's border needs them; one rounding at the end); with
`own` true it makes the library's calls.  `exact` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "i8": 1}
BLOCK = 256  # weights that share a scale


# ---- the cases ----

def _norm(T, D, src, res, dst, scale="none", weight=True):
    """T tokens of D channels in `src`, a residual of type `res` ("none":
    without one), into `dst`; "i8" with scale "static" (one for all) or "token"."""
    return {"op": "norm", "T": T, "D": D, "src": src, "res": res, "dst": dst, "scale": scale, "weight": weight}


def _gated(M, N, K, src, dst, scale="none"):
    """M tokens of K channels in `src` through two ternary matrices of N
    rows; "i8" with scale "static" or "token"."""
    return {"op": "gated", "M": M, "N": N, "K": K, "src": src, "dst": dst, "scale": scale}


def _answer(T, V, src, top, given=True, entropy=True):
    """T rows of V logits; the `top` likeliest of each."""
    return {"op": "answer", "T": T, "V": V, "src": src, "top": top, "given": given, "entropy": entropy}


def listed():
    return [
        # one token between attention and the gate and up projections of the 8B stack
        {"name": "norm one token", **_norm(1, 4096, "f32", "f32", "f16")},
        # a prompt at the same place
        {"name": "norm prompt 4096", **_norm(4096, 4096, "f32", "bf16", "f16")},
        # a decoding batch for the int8 projections, whose scale is fixed
        {"name": "norm i8 64 tokens", **_norm(64, 4096, "f32", "f32", "i8", "static")},
        # an odd batch of another width, a scale for each token
        {"name": "norm i8 1001 tokens", **_norm(1001, 5000, "bf16", "bf16", "i8", "token")},
        # one token through the 8B stack's gate and up
        {"name": "gated one token", **_gated(1, 16384, 4096, "f16", "f16")},
        # a decoding batch
        {"name": "gated 16 tokens", **_gated(16, 16384, 4096, "f16", "f16")},
        # an odd batch of drafts through an odd number of rows
        {"name": "gated 77 odd", **_gated(77, 5461, 2560, "f16", "f32")},
        # a prompt chunk
        {"name": "gated prompt 4096", **_gated(4096, 16384, 4096, "f16", "f16")},
        # a decoding batch in 8 bits
        {"name": "gated i8 32 tokens", **_gated(32, 16384, 4096, "i8", "f16", "static")},
        # a prompt in 8 bits, a scale for each token
        {"name": "gated i8 prompt 1500", **_gated(1500, 16384, 4096, "i8", "bf16", "token")},
        # one row after the output projection, its likeliest tokens
        {"name": "answer one row", **_answer(1, 131072, "f32", 20)},
        # a prompt's log probabilities over an odd vocabulary
        {"name": "answer prompt 2048", **_answer(2048, 65537, "f32", 5)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("norm", "gated", "gated", "answer"))
    if op == "norm":
        D = 8 * _log(rng, 8, 2048)
        T = _log(rng, 1, max(1, 4096 * 4096 // D))
        dst, scale = rng.choice((("f16", "none"), ("bf16", "none"), ("f32", "none"), ("i8", "static"), ("i8", "token")))
        return _norm(T, D, rng.choice(("f16", "bf16", "f32")), rng.choice(("none", "f16", "bf16", "f32")), dst, scale,
                     rng.random() < 0.8)
    if op == "gated":
        K, N = BLOCK * _log(rng, 1, 64), _log(rng, 1, 20000)
        M = _log(rng, 1, max(1, min(6000, 4096 * 16384 * 4096 // (N * K))))
        src, scale = rng.choice((("f16", "none"), ("f16", "none"), ("i8", "static"), ("i8", "token")))
        return _gated(M, N, K, src, rng.choice(("f16", "bf16", "f32")), scale)
    V = _log(rng, 100, 262144)
    T = _log(rng, 1, max(1, 2048 * 65537 // V))
    top, given = rng.choice((0, 1, rng.randint(2, 32))), rng.random() < 0.8
    return _answer(T, V, rng.choice(("f16", "bf16", "f32")), top, given, not (given or top) or rng.random() < 0.6)


def work(case):
    if case["op"] == "norm":
        T, n = case["T"], case["T"] * case["D"]
        moved = n * (SIZE[case["src"]] + SIZE[case["dst"]]) + 4 * case["D"] * case["weight"]
        if case["res"] != "none":
            moved += 2 * n * SIZE[case["res"]]
        return {"bytes": moved + (4 * T if case["scale"] == "token" else 0), "flops": 6 * n}
    if case["op"] == "gated":
        M, N, K = case["M"], case["N"], case["K"]
        moved = 2 * N * K * 66 // 256 + M * (K * SIZE[case["src"]] + N * SIZE[case["dst"]])
        return {"bytes": moved + (4 * M if case["scale"] == "token" else 0), "flops": 4 * M * N * K}
    T, V = case["T"], case["V"]
    moved = T * V * SIZE[case["src"]] + T * (12 * case["given"] + 4 * case["entropy"] + 12 * case["top"])
    return {"bytes": moved, "flops": 4 * T * V}


# ---- inputs ----

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _channels(g, T, D):
    """Activations: a spread of sizes over the channels, a few of them far larger."""
    spread = torch.exp(0.3 * _normal(g, D))
    spread = torch.where(torch.rand(D, generator=g, device=DEV) < 0.005, 12 * spread, spread)
    return _normal(g, T, D) * spread


def _matrix(g, N, K):
    """Packed ternary weights: codes 0, 1, 2 with shares 0.3, 0.4, 0.3, four a byte, and fp16 scales of blocks."""
    u = torch.rand((N, K), generator=g, device=DEV)
    q = ((u >= 0.3).to(torch.uint8) + (u >= 0.7).to(torch.uint8)).view(N, K // 4, 4)
    codes = q[..., 0] | (q[..., 1] << 2) | (q[..., 2] << 4) | (q[..., 3] << 6)
    return codes, (0.005 + 0.045 * torch.rand((N, K // BLOCK), generator=g, device=DEV)).half()


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        state = {"case": case, "x": _channels(g, T, D).to(TYPES[case["src"]]), "residual": None, "h": None,
                 "weight": 1 + 0.2 * _normal(g, D) if case["weight"] else None, "s": None, "scales": None}
        if case["res"] != "none":
            # a stream that many layers have added to; the sum goes to a buffer of its own, so that a call can be made again
            state["residual"] = (4 * _channels(g, T, D)).to(TYPES[case["res"]])
            state["h"] = torch.empty_like(state["residual"])
        if case["dst"] == "i8":
            state["out"] = torch.empty((T, D), dtype=torch.int8, device=DEV)
            if case["scale"] == "static":
                state["s"] = 4.0 / 127  # a learned range that clips the far channels
            else:
                state["scales"] = torch.empty(T, device=DEV)
        else:
            state["out"] = torch.empty((T, D), dtype=TYPES[case["dst"]], device=DEV)
        return state
    if case["op"] == "gated":
        M, N, K = case["M"], case["N"], case["K"]
        gate, up = _matrix(g, N, K), _matrix(g, N, K)
        x = _channels(g, M, K)
        state = {"case": case, "gate": gate, "up": up, "s": None,
                 "h": torch.empty((M, N), dtype=TYPES[case["dst"]], device=DEV),
                 # scratch that a program keeps for all its layers
                 "ws": torch.empty(64 << 20, dtype=torch.uint8, device=DEV)}
        if case["src"] == "i8":
            token = x.abs().amax(-1) / 127
            state["s"] = 4.0 / 127 if case["scale"] == "static" else token
            s = state["s"] if case["scale"] == "static" else token[:, None]
            state["x"] = (x / s).round().clamp(-128, 127).to(torch.int8)
        else:
            state["x"] = x.half()
        return state
    T, V, top = case["T"], case["V"], case["top"]
    # logits: a body, and some tokens that stand out in each row
    x = 2 * _normal(g, T, V)
    at = torch.randint(V, (T, 8), generator=g, device=DEV)
    x.scatter_(1, at, 8 + 3 * _normal(g, T, 8))
    tokens = torch.where(torch.rand(T, generator=g, device=DEV) < 0.7, at[:, 0],
                         torch.randint(V, (T,), generator=g, device=DEV))
    return {"case": case, "logits": x.to(TYPES[case["src"]]), "tokens": tokens if case["given"] else None,
            "logprobs": torch.empty(T, device=DEV) if case["given"] else None,
            "entropy": torch.empty(T, device=DEV) if case["entropy"] else None,
            "top_tokens": torch.empty((T, top), dtype=torch.int64, device=DEV) if top else None,
            "top_logprobs": torch.empty((T, top), device=DEV) if top else None,
            "ws": torch.empty(16 << 20, dtype=torch.uint8, device=DEV)}


# ---- plain forms ----

def _ratio(a, b):
    """a / b as one division in 32 bits: through 64, whose second rounding does not show."""
    return (a.double() / b).float()


def _held(codes, scale):
    """The values that 8-bit codes stand for."""
    return codes * scale


def _plain_norm(state):
    case, h = state["case"], state["x"].float()
    if state["residual"] is not None:
        state["h"].copy_(state["residual"].float() + h)
        h = state["h"].float()
    eight = case["dst"] == "i8"
    # codes lie next to borders: their root is that of a sum in 64 bits
    sq = h.double() if eight else h
    y = h * (1 / torch.sqrt((sq * sq).mean(-1, keepdim=True) + 1e-6)).float()
    if state["weight"] is not None:
        y = y * state["weight"]
    if not eight:
        state["out"].copy_(y)
        return _found(state["out"], state["h"])
    if state["s"] is not None:
        s = torch.full((1, 1), state["s"], device=DEV)
    else:
        s = _ratio(y.abs().amax(-1, keepdim=True), 127.0)
        state["scales"].copy_(s[:, 0])
    q = _ratio(y, torch.where(s == 0, 1, s).double()).round().clamp(-128, 127)
    state["out"].copy_(q)
    return _found(_held(state["out"], s), state["scales"], state["h"])


def _dense(codes, scales):
    """The fp32 matrix that packed weights stand for."""
    N = codes.shape[0]
    q = torch.stack((codes & 3, (codes >> 2) & 3, (codes >> 4) & 3, codes >> 6), -1)
    return ((q.view(N, -1, BLOCK).float() - 1) * scales.float()[..., None]).view(N, -1)


def _plain_gated(state):
    x = state["x"].float()
    if state["s"] is not None:
        x = x * (state["s"] if isinstance(state["s"], float) else state["s"][:, None])
    a, b = x @ _dense(*state["gate"]).T, x @ _dense(*state["up"]).T
    state["h"].copy_(a / (1 + torch.exp(-a)) * b)
    return state["h"]


def _plain_answer(state):
    case, x = state["case"], state["logits"].float()
    m = x.amax(-1, keepdim=True)
    t = x - m
    e = torch.exp(t)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    if state["tokens"] is not None:
        state["logprobs"].copy_((torch.gather(x, 1, state["tokens"][:, None]) - lse)[:, 0])
    if state["entropy"] is not None:
        state["entropy"].copy_(torch.log(z[:, 0]) - (e * t).sum(-1) / z[:, 0])
    if case["top"]:
        # the largest values, of equal ones the first: both in one whole number
        b = (x + 0.0).view(torch.int32)
        key = (b ^ ((b >> 31) & 0x7fffffff)).long() * (1 << 32) + (case["V"] - torch.arange(case["V"], device=DEV))
        at = case["V"] - (torch.topk(key, case["top"], -1).values & 0xffffffff)
        state["top_tokens"].copy_(at)
        state["top_logprobs"].copy_(torch.gather(x, 1, at) - lse)
    return _found(state["logprobs"], state["entropy"], state["top_tokens"], state["top_logprobs"])


def _found(*outputs):
    return [o for o in outputs if o is not None]


def run(state):
    case = state["case"]
    if not own:
        return {"norm": _plain_norm, "gated": _plain_gated, "answer": _plain_answer}[case["op"]](state)
    from ternary_packed_weight_amd import tq2
    if case["op"] == "norm":
        if case["dst"] != "i8":
            tq2.tq2_add_rms_norm(state["x"], state["residual"], state["weight"], eps=1e-6, h_out=state["h"],
                                 out=state["out"])
            return _found(state["out"], state["h"])
        tq2.tq2_add_rms_norm_i8(state["x"], state["residual"], state["weight"], eps=1e-6, s=state["s"],
                                h_out=state["h"], x_q=state["out"], x_scales=state["scales"])
        held = _held(state["out"], state["s"] if state["s"] is not None else state["scales"][:, None])
        return _found(held, state["scales"], state["h"])
    if case["op"] == "gated":
        if case["src"] == "i8":
            return tq2.tq2_gemm_i8q_gate_up_silu(*state["gate"], *state["up"], state["x"], state["s"], h=state["h"],
                                                 ws=state["ws"])
        return tq2.tq2_gemm_gate_up_silu(*state["gate"], *state["up"], state["x"], h=state["h"], ws=state["ws"])
    tq2.tq2_token_logprobs(state["logits"], state["tokens"], top=case["top"], logprobs=state["logprobs"],
                           entropy=state["entropy"], top_tokens=state["top_tokens"],
                           top_logprobs=state["top_logprobs"], ws=state["ws"])
    return _found(state["logprobs"], state["entropy"], state["top_tokens"], state["top_logprobs"])


# ---- the definitions in 64 bits ----

def _exact_norm(state):
    case = state["case"]

    def f32(t):
        return t.to(torch.float32).to(torch.float64)

    total = state["x"].double()
    if state["residual"] is not None:  # a sum in fp32, held in the residual's type
        total = f32(total + state["residual"].double()).to(TYPES[case["res"]]).double()
    h = total if state["residual"] is not None else None
    root = torch.rsqrt(total.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6)
    w = 1.0 if state["weight"] is None else state["weight"].double()
    if case["dst"] != "i8":
        return _found(total * root * w, h)
    # the steps that are fp32 are rounded one by one, so that codes are those of the definition
    y = f32(f32(total * f32(root)) * w)
    if case["scale"] == "static":
        s = f32(torch.tensor([[state["s"]]], dtype=torch.float64, device=DEV))
        scales = None
    else:
        s = f32(y.abs().max(-1, keepdim=True).values / 127)
        scales = s[:, 0]
    q = torch.where(s == 0, 0, torch.round(f32(y / torch.where(s == 0, 1.0, s)))).clamp(-128, 127)
    return _found(q * s, scales, h)


def _exact_gated(state):
    case, x = state["case"], state["x"].double()
    if case["scale"] == "token":
        x *= state["s"].double()[:, None]
    elif case["scale"] == "static":
        x *= torch.tensor(state["s"], dtype=torch.float32).item()
    out = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // case["K"])
    place = torch.arange(case["K"], device=DEV)
    for n in range(0, case["N"], step):
        y = []
        for codes, scales in (state["gate"], state["up"]):
            q = (codes[n:n + step][:, place // 4].int() >> (2 * (place % 4))) & 3
            w = (q - 1).double() * torch.repeat_interleave(scales[n:n + step].double(), BLOCK, dim=1)
            y.append(torch.mm(x, w.t().contiguous()))
        out[:, n:n + step] = y[0] * torch.special.expit(y[0]) * y[1]
    return out


def _exact_answer(state):
    case, T = state["case"], state["logits"].shape[0]
    outs = {name: torch.empty(state[name].shape, dtype=torch.float64, device=DEV)
            for name in ("logprobs", "entropy", "top_logprobs") if state[name] is not None}
    top = torch.empty((T, case["top"]), dtype=torch.int64, device=DEV)
    step = max(1, (1 << 25) // case["V"])
    for t in range(0, T, step):
        some = slice(t, min(T, t + step))
        logp = torch.log_softmax(state["logits"][some].double(), -1)
        if case["given"]:
            rows = torch.arange(logp.shape[0], device=DEV)
            outs["logprobs"][some] = logp[rows, state["tokens"][some]]
        if case["entropy"]:
            outs["entropy"][some] = torch.special.entr(logp.exp()).sum(-1)
        if case["top"]:
            order = torch.argsort(state["logits"][some].double(), dim=-1, descending=True, stable=True)
            top[some] = order[:, :case["top"]]
            outs["top_logprobs"][some] = torch.take_along_dim(logp, top[some], 1)
    return _found(outs.get("logprobs"), outs.get("entropy"), top if case["top"] else None, outs.get("top_logprobs"))


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "gated": _exact_gated, "answer": _exact_answer}[case["op"]](state)
