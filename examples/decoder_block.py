"""The attention block of a decoder layer on ternary projections, as a program
would run it: RMS norm, q/k/v projection, rotary append to the 8-bit cache,
attention, output projection, with the residual stream in fp32.

    python examples/decoder_block.py [--hidden 5120] [--prompt 2048] [--steps 32]

A prompt goes through in chunks (the projections' s8 rung, fed by the norm's
8-bit output), then tokens one at a time (their gemv rung, fed by its bf16
output), the decode step captured in a graph. Weights and inputs are random.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ternary_weight_linear_amd as tl  # noqa: E402


def ternary(rng, n, k, group=128):
    w = rng.choice(np.array([-1, 0, 1], np.int8), size=(n, k), p=(0.3, 0.4, 0.3))
    s = (rng.uniform(0.5, 1.5, (n, k // group)) / np.sqrt(0.6 * k)).astype(np.float16)
    return tl.TernaryWeights.from_host(w, s, device="cuda:0")


class DecoderBlock:
    """One block and the cache of `seqs` sequences of up to `most` tokens."""

    def __init__(self, hidden, q_heads, kv_heads, d, seqs, most, seed=0, sections=None):
        rng = np.random.default_rng(seed)
        self.hidden, self.hq, self.hkv, self.d, self.seqs, self.most = hidden, q_heads, kv_heads, d, seqs, most
        self.w_qkv = ternary(rng, (q_heads + 2 * kv_heads) * d, hidden)
        self.w_out = ternary(rng, hidden, q_heads * d)
        self.norm = torch.from_numpy(rng.uniform(0.8, 1.2, hidden).astype(np.float32)).to("cuda:0")
        pages = (most + tl.KV_PAGE - 1) // tl.KV_PAGE
        self.cache = tl.KVCache.empty(seqs * pages, kv_heads, d, "cuda:0")
        order = rng.permutation(seqs * pages).astype(np.int32).reshape(seqs, pages)
        self.table = torch.from_numpy(order).to("cuda:0")
        self.rope = tl.Rope.make(most, d // 2, 1e6, sections=sections, interleaved=True, device="cuda:0")
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device="cuda:0")

    def batch(self, n):
        """n new tokens of every sequence; the lengths are read when the kernels run."""
        begin = torch.arange(self.seqs + 1, dtype=torch.int32, device="cuda:0") * n
        return tl.KVBatch(begin, self.kv_len, self.table, max_q=n, max_kv=self.most)

    def forward(self, x, stream, positions, batch):
        """x: the layer before's output [T, hidden] fp32, added to the residual
        `stream` [T, hidden] in place. Returns the block's output [T, hidden] fp32
        and what it went through."""
        if tl.resolve_rung(x.shape[0]) == "s8":
            q8, scale = tl.rmsnorm_s8(x, self.norm, residual=stream, layout="operand_order")
            normed = (q8, scale)
            qkv = tl.linear_s8_q(q8, scale, self.w_qkv, layout="operand_order")
        else:
            normed = tl.rmsnorm(x, self.norm, residual=stream)
            qkv = tl.linear(normed, self.w_qkv)
        heads = qkv.unflatten(1, (self.hq + 2 * self.hkv, self.d))
        a, b = self.hq, self.hq + self.hkv
        q = tl.kv_append(self.cache, batch, heads[:, a:b], heads[:, b:], q=heads[:, :a], rope=self.rope, positions=positions)
        o = tl.kv_attn(q, self.cache, batch, self.d ** -0.5)
        y = tl.linear(o.flatten(1), self.w_out)
        return y, {"normed": normed, "qkv": qkv, "q": q, "o": o}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--chunk", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    d, hq = 128, a.hidden // 128
    hkv = max(1, hq // 5) if hq % 5 == 0 else 1
    block = DecoderBlock(a.hidden, hq, hkv, d, 1, a.prompt + a.steps + 64, sections=(16, 24, 24))
    gen = torch.Generator(device="cuda:0").manual_seed(1)

    def tokens(n):
        return torch.randn((n, a.hidden), device="cuda:0", generator=gen)

    def positions(first, n):  # text: the three axes agree
        return (first + torch.arange(n, dtype=torch.int32, device="cuda:0")).repeat(3, 1).contiguous()

    torch.cuda.synchronize()
    t = time.perf_counter()
    for first in range(0, a.prompt, a.chunk):
        n = min(a.chunk, a.prompt - first)
        block.kv_len += n
        y, _ = block.forward(tokens(n), torch.zeros((n, a.hidden), device="cuda:0"), positions(first, n), block.batch(n))
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt} tokens in chunks of {a.chunk}: {(time.perf_counter() - t) * 1e3:.2f} ms, first call included")

    x, stream, pos, batch = tokens(1), torch.zeros((1, a.hidden), device="cuda:0"), positions(a.prompt, 1), block.batch(1)

    def step():
        block.kv_len.add_(1)
        y, _ = block.forward(x, stream, pos, batch)
        x.copy_(y)
        pos.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warms up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"{a.steps} decode steps: {(time.perf_counter() - t) / a.steps * 1e6:.1f} us each, {int(block.kv_len)} tokens in the cache, "
          f"output finite: {bool(torch.isfinite(x).all())}")


if __name__ == "__main__":
    main()
