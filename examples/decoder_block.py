"""The attention block of a decoder layer on ternary projections, as a program
would run it: RMS norm, q/k/v projection, rotary append to the 8-bit cache,
attention, output projection, with the residual stream in fp32; with --hybrid, a
recurrent block in front of it: projection, causal convolution, state space
scan, gated norm, output projection, and the norm that leads to the next block.

    python examples/decoder_block.py [--hidden 5120] [--prompt 2048] [--steps 32] [--hybrid]

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
            normed = tl.rmsnorm_s8(x, self.norm, residual=stream, layout="operand_order")
        else:
            normed = tl.rmsnorm(x, self.norm, residual=stream)
        return self.mix(normed, positions, batch)

    def mix(self, normed, positions, batch):
        """The block behind its norm: `normed` as rmsnorm or rmsnorm_s8 (in operand order) returns it."""
        qkv = project(normed, self.w_qkv)
        heads = qkv.unflatten(1, (self.hq + 2 * self.hkv, self.d))
        a, b = self.hq, self.hq + self.hkv
        q = tl.kv_append(self.cache, batch, heads[:, a:b], heads[:, b:], q=heads[:, :a], rope=self.rope, positions=positions)
        o = tl.kv_attn(q, self.cache, batch, self.d ** -0.5)
        y = tl.linear(o.flatten(1), self.w_out)
        return y, {"normed": normed, "qkv": qkv, "q": q, "o": o}


def project(normed, w):
    """A projection of a norm's output: 8-bit codes with their scales, or bf16."""
    return tl.linear_s8_q(*normed, w, layout="operand_order") if isinstance(normed, tuple) else tl.linear(normed, w)


class RecurrentBlock:
    """A recurrent block and the states of `seqs` sequences, one slot each."""

    def __init__(self, hidden, heads, dim, groups, state_dim, seqs, width=4, seed=0):
        rng = np.random.default_rng(seed)
        self.heads, self.dim, self.groups, self.state_dim, self.seqs = heads, dim, groups, state_dim, seqs
        self.inner = heads * dim
        self.channels = self.inner + 2 * groups * state_dim  # x, B and C, which the convolution mixes
        n = (self.inner + self.channels + heads + 15) // 16 * 16  # z, those, dt
        self.w_in = ternary(rng, n, hidden)
        self.w_out = ternary(rng, hidden, self.inner)

        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0")

        self.norm, self.post = dev(rng.uniform(0.8, 1.2, hidden)), dev(rng.uniform(0.8, 1.2, hidden))
        self.gate_norm = dev(rng.uniform(0.8, 1.2, self.inner))
        self.conv, self.conv_bias = dev(rng.uniform(-0.5, 0.5, (self.channels, width))), dev(rng.uniform(-0.1, 0.1, self.channels))
        step = np.exp(rng.uniform(np.log(1e-3), np.log(0.1), heads))
        self.dt_bias, self.a = dev(step + np.log(-np.expm1(-step))), dev(-rng.uniform(1, 16, heads))
        self.d = dev(np.ones(heads))
        self.inputs = torch.zeros((seqs, width - 1, self.channels), device="cuda:0")
        self.states = torch.zeros((seqs, heads, state_dim, dim), device="cuda:0")
        self.slots = torch.arange(seqs, dtype=torch.int32, device="cuda:0")

    def batch(self, n):
        """n new tokens of every sequence."""
        begin = torch.arange(self.seqs + 1, dtype=torch.int32, device="cuda:0") * n
        return tl.StateBatch(begin, self.slots, self.slots, max_q=n)

    def forward(self, x, stream, batch, next_norm):
        """x as DecoderBlock.forward takes it; the block's own output goes into
        `stream` too, through its norm. Returns `next_norm` of the stream, and
        what the block went through."""
        wide = tl.resolve_rung(x.shape[0]) == "s8"
        if wide:
            normed = tl.rmsnorm_s8(x, self.norm, residual=stream, layout="operand_order")
        else:
            normed = tl.rmsnorm(x, self.norm, residual=stream)
        p = project(normed, self.w_in)
        i, c, g, n = self.inner, self.channels, self.groups, self.state_dim
        mixed = tl.causal_conv(p[:, i:i + c], self.conv, self.inputs, batch, bias=self.conv_bias)
        y = tl.scan(mixed[:, :i].unflatten(1, (self.heads, self.dim)), mixed[:, i:i + g * n].unflatten(1, (g, n)),
                    mixed[:, i + g * n:].unflatten(1, (g, n)), p[:, i + c:i + c + self.heads], self.a, self.states, batch,
                    d=self.d, dt_bias=self.dt_bias)
        if wide:
            gated = tl.rmsnorm_gated_s8(y.flatten(1), p[:, :i], self.gate_norm, group=i // g, layout="operand_order")
        else:
            gated = tl.rmsnorm_gated(y.flatten(1), p[:, :i], self.gate_norm, group=i // g)
        o = project(gated, self.w_out)
        if wide:
            out = tl.rmsnorm_post_s8(o, self.post, stream, next_norm, scale=0.5, layout="operand_order")
        else:
            out = tl.rmsnorm_post(o, self.post, stream, next_norm, scale=0.5)
        return out, {"normed": normed, "p": p, "mixed": mixed, "y": y, "gated": gated, "o": o}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--chunk", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--hybrid", action="store_true", help="a recurrent block in front of the attention block")
    a = ap.parse_args()
    d, hq = 128, a.hidden // 128
    hkv = max(1, hq // 5) if hq % 5 == 0 else 1
    block = DecoderBlock(a.hidden, hq, hkv, d, 1, a.prompt + a.steps + 64, sections=(16, 24, 24))
    before = RecurrentBlock(a.hidden, 2 * a.hidden // 64, 64, 8 if a.hidden % 1024 == 0 else 1, 128, 1) if a.hybrid else None
    gen = torch.Generator(device="cuda:0").manual_seed(1)

    def tokens(n):
        return torch.randn((n, a.hidden), device="cuda:0", generator=gen)

    def positions(first, n):  # text: the three axes agree
        return (first + torch.arange(n, dtype=torch.int32, device="cuda:0")).repeat(3, 1).contiguous()

    def layer(x, stream, pos, batch, states):
        if before is None:
            return block.forward(x, stream, pos, batch)[0]
        return block.mix(before.forward(x, stream, states, block.norm)[0], pos, batch)[0]

    torch.cuda.synchronize()
    t = time.perf_counter()
    for first in range(0, a.prompt, a.chunk):
        n = min(a.chunk, a.prompt - first)
        block.kv_len += n
        y = layer(tokens(n), torch.zeros((n, a.hidden), device="cuda:0"), positions(first, n), block.batch(n),
                  before and before.batch(n))
    torch.cuda.synchronize()
    print(f"prompt of {a.prompt} tokens in chunks of {a.chunk}: {(time.perf_counter() - t) * 1e3:.2f} ms, first call included")

    x, stream, pos, batch = tokens(1), torch.zeros((1, a.hidden), device="cuda:0"), positions(a.prompt, 1), block.batch(1)
    states = before and before.batch(1)

    def step():
        block.kv_len.add_(1)
        x.copy_(layer(x, stream, pos, batch, states))
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
