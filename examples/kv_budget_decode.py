"""Prompt and decode with a bounded KV cache: W4A16 projections, the paged 8-bit
cache with a scale per page and head, and eviction by accumulated attention weight.

    python examples/kv_budget_decode.py [--prompt 900] [--steps 200] [--budget 512] [--slack 128]

A stack of attention layers (random 4-bit weights, no checkpoint) reads a batch of
prompts in chunks and then decodes token by token.  Every layer's cache has room
for budget + slack tokens per sequence and never grows: whenever a chunk or a
token would not fit, each sequence is cut to its `budget` most used tokens, in
place, and the pages behind them fill up again.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a16_quantized_gemm_gb300 import binding  # noqa: E402


class Layer:
    """Weights and cache of one attention layer."""

    def __init__(self, hidden, Hq, Hkv, D, B, capacity, T, fmt, gen):
        g = 128
        self.Hq, self.Hkv, self.D = Hq, Hkv, D

        def packed(K, N):
            q = torch.randint(0, 16, (K, N), generator=gen, dtype=torch.uint8).cuda()
            z = torch.full((K // g, N), 8, dtype=torch.uint8, device="cuda")
            s = torch.full((K // g, N), 0.2 / K ** 0.5, dtype=torch.float16, device="cuda")
            return binding.pack(q, z, s, g), ((q.float() - 8) * s.repeat_interleave(g, 0).float())

        self.qkv, self.qkv_plain = packed(hidden, (Hq + 2 * Hkv) * D)
        self.o, self.o_plain = packed(Hq * D, hidden)
        pages = -(-capacity // T)
        self.blocks = binding.KVBlocks.empty(B * pages, Hkv, T, D, fmt)
        self.weights = torch.zeros(B, Hkv, pages * T, device="cuda")  # what each cached token drew so far


class Stack:
    def __init__(self, layers=2, hidden=1024, Hq=16, Hkv=4, D=64, B=4, budget=512, slack=128, T=64, fmt=torch.int8,
                 seed=0):
        gen = torch.Generator().manual_seed(seed)
        if budget < 1 or slack < 1:
            raise ValueError("budget and slack must be at least 1")
        self.B, self.budget, self.capacity = B, budget, budget + slack
        self.layers = [Layer(hidden, Hq, Hkv, D, B, self.capacity, T, fmt, gen) for _ in range(layers)]
        pages = -(-self.capacity // T)
        self.table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.held = [0] * B  # the same on the host, for the bounds
        self.evictions, self.graph = 0, None
        self.first, self.recent = min(4, budget // 2), min(64, budget // 2)

    def norm(self, x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).half()

    def make_room(self, new):
        """Every sequence to the budget where `new` tokens would not fit."""
        if max(self.held) + new <= self.capacity:
            return
        batch = binding.KVBatch(self.table, self.kv_len, max_len=self.capacity)
        for layer in self.layers:
            _, lengths = binding.kvb_evict(layer.blocks, batch, layer.weights, self.budget, first=self.first,
                                           recent=self.recent)
        self.kv_len.copy_(lengths)
        self.held = [min(n, self.budget) for n in self.held]
        self.evictions += 1

    def _forward(self, x, new):
        self.kv_len += new
        starts = None if new == 1 else torch.arange(0, self.B * new + 1, new, dtype=torch.int32, device="cuda")
        batch = binding.KVBatch(self.table, self.kv_len, q_start=starts, max_q=new, max_len=self.capacity)
        for layer in self.layers:
            heads = binding.gemm(self.norm(x), layer.qkv).view(self.B * new, -1, layer.D)
            k = heads[:, layer.Hq:layer.Hq + layer.Hkv]
            binding.kvb_append(layer.blocks, batch, k, heads[:, layer.Hq + layer.Hkv:], w=layer.weights)
            out = binding.kvb_attention(layer.blocks, batch, heads[:, :layer.Hq], w_in=layer.weights,
                                        w_out=layer.weights)
            x = x + binding.gemm(out.view(self.B * new, -1), layer.o)
        return x

    def step(self, x, new):
        """x [B * new][hidden]: `new` tokens of every sequence through the stack."""
        self.make_room(new)
        self.held = [n + new for n in self.held]
        return self._forward(x, new)

    def decode(self, x):
        """One token of every sequence, x [B][hidden], as a CUDA graph: lengths advance on the device."""
        self.make_room(1)
        self.held = [n + 1 for n in self.held]
        if self.graph is None:
            self.x, self.graph = x.clone(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.y = self._forward(self.x, 1)
        self.x.copy_(x)
        self.graph.replay()
        return self.y

    def prompt(self, x):
        """x [B][tokens][hidden], in chunks that fit behind the budget."""
        chunk, out = self.capacity - self.budget, []
        for at in range(0, x.shape[1], chunk):
            part = x[:, at:at + chunk]
            n = part.shape[1]
            out.append(self.step(part.reshape(self.B * n, -1).contiguous(), n).view(self.B, n, -1))
        return torch.cat(out, 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--prompt", type=int, default=900)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--budget", type=int, default=512)
    p.add_argument("--slack", type=int, default=128)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--format", choices=["int8", "e4m3"], default="int8")
    a = p.parse_args()
    fmt = torch.int8 if a.format == "int8" else torch.float8_e4m3fn
    stack = Stack(B=a.batch, budget=a.budget, slack=a.slack, fmt=fmt)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(a.batch, a.prompt, 1024, generator=gen, device="cuda").half()
    x = stack.prompt(x)[:, -1]
    x = stack.decode(stack.norm(x))  # captures the step
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        x = stack.decode(stack.norm(x))
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(a.steps, 1)
    size = sum(b.k.numel() * 2 + b.ks.numel() * 8 for b in (layer.blocks for layer in stack.layers))
    print(f"{a.batch} sequences, {a.prompt} prompt + {a.steps} decoded tokens in a cache of {stack.capacity} each "
          f"({size / 2 ** 20:.1f} MiB), {stack.evictions} evictions, {t * 1e6:.0f} us per decoded step")


if __name__ == "__main__":
    main()
