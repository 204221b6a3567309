#!/usr/bin/env python3
"""One verify (or draft) step of a 4-bit decoder, from the residual stream to drawn tokens.

Every layer runs
    rms_norm -> qkv gemm -> rotary positions -> kv_write -> paged_attention -> o gemm
    -> rms_norm (+ residual) -> gate_up gemm -> silu(gate) * up -> down gemm
and the step ends with rms_norm (+ residual) -> lm_head gemm -> sample. The rotary positions
and the gate are torch operations; everything else is this library's. Weights are seeded random
4-bit codes of a Qwen2.5-7B-shaped layer by default, the cache is 8-bit.

    python examples/decoder_step.py [--batch 1] [--tokens 5] [--context 2000] [--layers 4] [--steps 20]

captures the step in a HIP graph and prints its time.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_weight_only_gemm_amd as w4  # noqa: E402


@dataclass
class Shape:
    hidden: int = 3584
    heads: int = 28
    kv_heads: int = 4
    head_dim: int = 128
    ffn: int = 18944
    vocab: int = 152064
    layers: int = 4
    page: int = 64
    eps: float = 1e-6
    base: float = 1e6


class Linear:
    """Random 4-bit weights in the storage format, scaled to keep a unit-variance input near unit variance."""

    def __init__(self, k, n, gen):
        self.q = torch.randint(-2 ** 31, 2 ** 31, (k // 8, n), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)
        self.s = ((0.75 + 0.5 * torch.rand(k // 128, n, generator=gen, device="cuda")) * (0.2 / k ** 0.5)).half()
        self.z = torch.randint(6, 10, (k // 128, n), generator=gen, device="cuda", dtype=torch.uint8)

    def __call__(self, a):
        return w4.gemm(a, self.q, self.s, self.z)


class Decoder:
    def __init__(self, shape: Shape, pages: int, seed: int = 0):
        self.shape = s = shape
        gen = torch.Generator(device="cuda").manual_seed(seed)
        norm = lambda: (1 + 0.1 * torch.randn(s.hidden, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.layers = []
        for _ in range(s.layers):
            cache = (pages, s.kv_heads, s.page, s.head_dim)
            self.layers.append(dict(
                norm1=norm(), norm2=norm(),
                qkv=Linear(s.hidden, (s.heads + 2 * s.kv_heads) * s.head_dim, gen),
                o=Linear(s.heads * s.head_dim, s.hidden, gen),
                gate_up=Linear(s.hidden, 2 * s.ffn, gen), down=Linear(s.ffn, s.hidden, gen),
                k=torch.zeros(cache, dtype=torch.int8, device="cuda"), v=torch.zeros(cache, dtype=torch.int8, device="cuda"),
                ks=torch.zeros(cache[:3], device="cuda"), vs=torch.zeros(cache[:3], device="cuda")))
        self.norm, self.head = norm(), Linear(s.hidden, s.vocab, gen)
        # cosines and sines of every position's angles, from 64-bit angles
        freq = s.base ** (-torch.arange(0, s.head_dim, 2, device="cuda", dtype=torch.float64) / s.head_dim)
        angle = torch.arange(pages * s.page, device="cuda", dtype=torch.float64)[:, None] * freq
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def rotate(self, x, positions):
        """Rotary positions on [T, heads, D] (the two halves of a head form the pairs)."""
        c, s = self.cos[positions][:, None], self.sin[positions][:, None]
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def step(self, x, positions, slots, block_table, q_start, kv_len, max_q, max_kv, u, **sampling):
        """x: bfloat16 [T, hidden] embeddings of the new tokens. Returns (token, prob, logits) of each."""
        s, T = self.shape, x.shape[0]
        add = None  # a layer's output, added by the next norm
        for layer in self.layers:
            if add is None:
                a = w4.rms_norm(x, layer["norm1"], eps=s.eps)
            else:
                a, x = w4.rms_norm(add, layer["norm1"], residual=x, eps=s.eps)
            qkv = layer["qkv"](a).view(T, s.heads + 2 * s.kv_heads, s.head_dim)
            turned = self.rotate(qkv[:, :s.heads + s.kv_heads], positions)
            w4.kv_write(turned[:, s.heads:], qkv[:, s.heads + s.kv_heads:], slots, layer["k"], layer["v"], layer["ks"],
                        layer["vs"])
            o = w4.paged_attention(turned[:, :s.heads].to(torch.bfloat16), layer["k"], layer["v"], block_table, q_start,
                                   kv_len, max_q, max_kv, layer["ks"], layer["vs"])
            a, x = w4.rms_norm(layer["o"](o.view(T, -1)), layer["norm2"], residual=x, eps=s.eps)
            gate, up = layer["gate_up"](a).chunk(2, -1)
            add = layer["down"]((torch.nn.functional.silu(gate) * up).to(torch.bfloat16))
        a, x = w4.rms_norm(add, self.norm, residual=x, eps=s.eps)
        logits = self.head(a)
        token, prob = w4.sample(logits, u, **sampling)
        return token, prob, logits


def batch_of(decoder: Decoder, batch, tokens, context, seed=1):
    """The inputs of a step of `batch` sequences of `tokens` new tokens that end at `context`, their cache filled."""
    s = decoder.shape
    gen = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-context // s.page)
    table = torch.randperm(batch * per, generator=gen, device="cuda").view(batch, per)
    at = torch.arange(context - tokens, context, device="cuda")
    slots = (table[:, at // s.page] * s.page + at % s.page).reshape(-1)
    for layer in decoder.layers:
        layer["k"].random_(-127, 128, generator=gen)
        layer["v"].random_(-127, 128, generator=gen)
        layer["ks"].fill_(0.01)
        layer["vs"].fill_(0.01)
    T = batch * tokens
    return dict(x=torch.randn(T, s.hidden, generator=gen, device="cuda").to(torch.bfloat16), positions=at.repeat(batch),
                slots=slots, block_table=table.to(torch.int32),
                q_start=torch.arange(0, T + 1, tokens, dtype=torch.int32, device="cuda"),
                kv_len=torch.full((batch,), context, dtype=torch.int32, device="cuda"), max_q=tokens, max_kv=context,
                u=torch.rand(T, generator=gen, device="cuda"), temperature=torch.full((T,), 0.8, device="cuda"),
                top_k=torch.full((T,), 50, dtype=torch.int32, device="cuda"), top_p=torch.full((T,), 0.95, device="cuda"))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("batch", 1), ("tokens", 5), ("context", 2000), ("layers", 4), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    shape = Shape(layers=a.layers)
    decoder = Decoder(shape, a.batch * -(-a.context // shape.page))
    inputs = batch_of(decoder, a.batch, a.tokens, a.context)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        token, _, _ = decoder.step(**inputs)          # sizes the stream's workspace
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            drawn, prob, _ = decoder.step(**inputs)
        graph.replay()
        stream.synchronize()
        assert torch.equal(drawn, token), "a replay of the step differs from the eager one"
        begin, end = torch.cuda.Event(True), torch.cuda.Event(True)
        begin.record(stream)
        for _ in range(a.steps):
            graph.replay()
        end.record(stream)
        stream.synchronize()
    ms = begin.elapsed_time(end) / a.steps
    print(f"{a.batch} x {a.tokens} tokens over {a.context}, {a.layers} layers and the head: {ms:.3f} ms a step; "
          f"tokens {drawn.tolist()[:8]}, probabilities {[round(p, 4) for p in prob.tolist()[:8]]}")


if __name__ == "__main__":
    main()
