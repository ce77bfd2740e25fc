"""The attention half of one decoder layer, from the ternary projections to the
residual stream, over a 4-bit cache.

A batch of prompts of unequal length goes through in one call each (q/k/v
product, head norms and rotation, store, attention, output product); then one
token of every sequence a step, as one HIP graph that a decode loop replays:
what moves from step to step (positions, slots, lengths) lives on the device
and is advanced inside the graph.

    python examples/decode_layer.py [--batch 8] [--prompt 1024] [--steps 32]

Random weights of the 8B decode stack's layer: 4096 wide, 32 query and 2 key
heads of 128.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from ternary_packed_weight_amd import tq2  # noqa: E402

WIDTH, HQ, HK, D, PAGE = 4096, 32, 2, 128, 64
DEV = "cuda"


def ternary(n, k, g):
    """A random ternary matrix [n][k] of about unit gain, packed."""
    w = torch.randint(-1, 2, (n, k), generator=g, device=DEV).float() * (1.2 * k ** -0.5)
    codes, scales, bad = tq2.tq2_pack(w)
    return codes, scales


class Layer:
    def __init__(self, batch, longest, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.qkv, self.o = ternary((HQ + 2 * HK) * D, WIDTH, g), ternary(WIDTH, HQ * D, g)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(D, generator=g, device=DEV) for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)).float()
        # pages of all sequences, dealt in an order of their own
        self.width = -(-longest // PAGE)
        pages = batch * self.width
        self.table = torch.randperm(pages, generator=g, device=DEV).int().view(batch, self.width)
        self.cache = torch.zeros((pages, HK, PAGE * (D + 8)), dtype=torch.uint8, device=DEV)

    def slots(self, sequence, place):
        return self.table[sequence, place // PAGE].long() * PAGE + place % PAGE

    def buffers(self, tokens, batch, longest_new):
        new = dict(dtype=torch.float16, device=DEV)
        need = max(tq2.tq2_kv4_attn_workspace_bytes(tokens, HQ, HK, D, PAGE, self.width, batch, longest_new), 1)
        return dict(q=torch.empty((tokens, HQ, D), **new), k=torch.empty((tokens, HK, D), **new),
                    v=torch.empty((tokens, HK, D), **new), out=torch.empty((tokens, HQ, D), **new),
                    ws=torch.empty(need, dtype=torch.uint8, device=DEV))

    def forward(self, x, positions, slots, lengths, b, starts=None, longest_new=None):
        """x [tokens][WIDTH] fp16 -> the same; b: buffers for as many tokens."""
        y = tq2.tq2_gemm(*self.qkv, x).view(len(x), HQ + 2 * HK, D)
        tq2.tq2_qk_norm_rope(y[:, :HQ], y[:, HQ:HQ + HK], positions, self.inv_freq, self.q_norm, self.k_norm,
                             q_out=b["q"], k_out=b["k"])
        b["v"].copy_(y[:, HQ + HK:])
        tq2.tq2_kv4_store(self.cache, b["k"], b["v"], slots)
        tq2.tq2_kv4_attn(b["q"], self.cache, self.table, lengths, q_start=starts, max_q=longest_new, out=b["out"], ws=b["ws"])
        return x + tq2.tq2_gemm(*self.o, b["out"].view(len(x), HQ * D)).half()


def plain(layer, x, qkv, kept, lengths, place):
    """The same token in plain 64-bit operations, over keys and values as the cache gives them back."""
    out = []
    for s in range(len(x)):
        k, v = (t.double() for t in kept[s])
        q = qkv[s, :HQ].double()
        q = q / torch.sqrt(q.pow(2).mean(-1, keepdim=True) + 1e-6) * layer.q_norm.double()
        a = float(place[s]) * layer.inv_freq.double()
        u, w = q[:, :D // 2], q[:, D // 2:]
        q = torch.cat((u * a.cos() - w * a.sin(), w * a.cos() + u * a.sin()), -1).half().double()
        p = torch.stack([torch.softmax(k[:, h // (HQ // HK)] @ q[h] * D ** -0.5, -1) for h in range(HQ)])
        out.append(torch.stack([p[h] @ v[:, h // (HQ // HK)] for h in range(HQ)]))
    return torch.stack(out)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args(argv)
    g = torch.Generator(device=DEV).manual_seed(1)
    layer = Layer(a.batch, a.prompt + a.steps + 1)

    # prompts of unequal length, one call for all of them
    n = [max(1, a.prompt * (i + 1) // a.batch) for i in range(a.batch)]
    sequence = torch.repeat_interleave(torch.arange(a.batch), torch.tensor(n)).to(DEV)
    place = torch.cat([torch.arange(m) for m in n]).to(DEV)
    lengths = torch.tensor(n, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    x = torch.randn((sum(n), WIDTH), generator=g, device=DEV).half()
    b = layer.buffers(len(x), a.batch, max(n))
    y = layer.forward(x, place.int(), layer.slots(sequence, place), lengths, b, starts, max(n))

    # then a token of each a step, captured once
    b = layer.buffers(a.batch, a.batch, 1)
    token, at = y[starts[1:].long() - 1].clone(), lengths.clone()
    every = torch.arange(a.batch, device=DEV)

    def step():
        lengths.add_(1)
        token.copy_(layer.forward(token, at, layer.slots(every, at.long()), lengths, b))
        at.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps - 2):
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, a.steps - 2)

    # the last step once more in plain operations
    last = token.clone()
    graph.replay()
    torch.cuda.synchronize()
    qkv = tq2.tq2_gemm(*layer.qkv, last).view(a.batch, HQ + 2 * HK, D)
    kept = [tq2.tq2_kv4_load(layer.cache, layer.slots(s, torch.arange(int(lengths[s]), device=DEV)), D, dtype=torch.float32)
            for s in range(a.batch)]
    want = plain(layer, last, qkv, kept, lengths, at - 1)
    off = float((b["out"].double() - want).norm() / want.norm())
    print(f"{sum(n)} prompt tokens of {a.batch} sequences, {a.steps} tokens each: {t * 1e6:.1f} us a layer and step, "
          f"attention off by {off:.1e} from 64 bits")
    return off


if __name__ == "__main__":
    main()
