"""Greedy decoding with drafted trees and an adapter per request: W4A16 projections with low-rank adapters beside them,
keys rotated on the way into the paged 8-bit cache, attention for a tree of drafts, and the accepted path moved together.

    python examples/tree_decode.py [--prompt 300] [--steps 60] [--batch 4]

A stack of attention layers (random 4-bit weights, no checkpoint) over a toy vocabulary.  Each step guesses a small tree of
next tokens from the successors seen so far, runs all of its nodes at once, keeps the path on which every node is its
parent's most likely token, and learns the successors.  A step is one CUDA graph: nothing in it waits for the host.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w4a16_quantized_gemm_gb300 import binding  # noqa: E402

PARENTS = [-1, 0, 0, 1, 1, 2, 2, 3, 3]  # node 0 is certain; then two guesses after each of the first ones


def rope_table(positions, dims, base=10000.0):
    """Cosines and sines of every position, from angles in 64 bits."""
    half = dims // 2
    turn = base ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Layer:
    """Weights, adapters and cache of one attention layer."""

    def __init__(self, hidden, Hq, Hkv, D, B, pages, T, fmt, adapters, R, gen):
        g = 128
        self.Hq, self.Hkv, self.D = Hq, Hkv, D

        def packed(K, N):
            q = torch.randint(0, 16, (K, N), generator=gen, dtype=torch.uint8).cuda()
            z = torch.full((K // g, N), 8, dtype=torch.uint8, device="cuda")
            s = torch.full((K // g, N), 0.2 / K ** 0.5, dtype=torch.float16, device="cuda")
            a = (torch.randn(adapters, R, K, generator=gen) * K ** -0.5).half().cuda()
            b = (torch.randn(adapters, N, R, generator=gen) * 0.3 * R ** -0.5).half().cuda()
            return binding.pack(q, z, s, g), binding.Adapters(a, b), (q.float() - 8) * s.repeat_interleave(g, 0).float()

        self.qkv, self.qkv_lora, self.qkv_plain = packed(hidden, (Hq + 2 * Hkv) * D)
        self.o, self.o_lora, self.o_plain = packed(Hq * D, hidden)
        self.blocks = binding.KVBlocks.empty(B * pages, Hkv, T, D, fmt)


class Stack:
    def __init__(self, layers=2, hidden=1024, Hq=16, Hkv=4, D=64, B=4, room=512, T=64, fmt=torch.int8, vocab=256,
                 adapters=3, R=16, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.n, self.vocab = B, len(PARENTS), vocab
        pages = -(-room // T)
        self.room = pages * T
        self.layers = [Layer(hidden, Hq, Hkv, D, B, pages, T, fmt, adapters, R, gen) for _ in range(layers)]
        self.embed = (torch.randn(vocab, hidden, generator=gen)).half().cuda()
        self.rope = binding.Rope(rope_table(self.room + self.n, D).cuda())
        self.table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.new_len = torch.zeros_like(self.kv_len)
        # the last request has no adapter
        self.ids = torch.tensor([b % adapters if b + 1 < B else -1 for b in range(B)], dtype=torch.int32, device="cuda")
        depth = [0] * self.n
        for i, p in enumerate(PARENTS):
            depth[i] = depth[p] + 1 if p >= 0 else 0
        self.depth = torch.tensor(depth, dtype=torch.int32, device="cuda")
        self.mask = binding.tree_masks([PARENTS] * B).cuda()
        self.starts = torch.arange(0, B * self.n + 1, self.n, dtype=torch.int32, device="cuda")
        self.successors = torch.randint(0, vocab, (vocab, 2), generator=gen).cuda()  # guesses after each token
        self.token = torch.zeros(B, dtype=torch.long, device="cuda")                 # the next one, certain
        self.held, self.graph = 0, None                                              # what the fullest sequence may hold

    def norm(self, x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).half()

    def _forward(self, x, batch, starts, pos, tree):
        for layer in self.layers:
            y = self.norm(x)
            heads = binding.lora_add(binding.gemm(y, layer.qkv), y, layer.qkv_lora, self.ids, q_start=starts)
            heads = heads.view(x.shape[0], -1, layer.D)
            q, k = heads[:, :layer.Hq], heads[:, layer.Hq:layer.Hq + layer.Hkv]
            binding.kvb_append_rope(layer.blocks, batch, k, heads[:, layer.Hq + layer.Hkv:], self.rope, Q=q, q_out=q, pos=pos)
            if tree:
                out = binding.kvb_attention_tree(layer.blocks, batch, q, self.mask)
            else:
                out = binding.kvb_attention(layer.blocks, batch, q)
            out = out.view(x.shape[0], -1)
            x = x + binding.lora_add(binding.gemm(out, layer.o), out, layer.o_lora, self.ids, q_start=starts)
        return x

    def logits(self, x):
        return self.norm(x).float() @ self.embed.float().T

    def prompt(self, tokens):
        """tokens [B][n]: fills the cache; the most likely next token is certain to be kept."""
        B, n = tokens.shape
        if self.held + n > self.room:
            raise ValueError("the prompt does not fit the cache")
        self.held += n
        self.kv_len += n
        starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        batch = binding.KVBatch(self.table, self.kv_len, q_start=starts, max_q=n)
        x = self._forward(self.embed[tokens.flatten()], batch, starts, None, False)
        self.token.copy_(self.logits(x.view(B, n, -1)[:, -1]).argmax(1))
        return x.view(B, n, -1)

    def _step(self):
        B, n = self.B, self.n
        # the tree's tokens: child k of a node is guess k after its token
        tokens = [self.token]
        for i in range(1, n):
            tokens.append(self.successors[tokens[PARENTS[i]], (i - 1) % 2])
        tokens = torch.stack(tokens, 1)
        pos = (self.kv_len[:, None] + self.depth).flatten()
        self.kv_len += n
        batch = binding.KVBatch(self.table, self.kv_len, q_start=self.starts, max_q=n)
        x = self._forward(self.embed[tokens.flatten()], batch, self.starts, pos, True).view(B, n, -1)
        best = self.logits(x.view(B * n, -1)).argmax(1).view(B, n)
        # the path on which every node is what its parent found most likely (of equal guesses the first)
        kept = [torch.ones(B, dtype=torch.bool, device="cuda")]
        taken = [torch.zeros(B, dtype=torch.bool, device="cuda") for _ in range(n)]
        for i in range(1, n):
            p = PARENTS[i]
            kept.append(kept[p] & (tokens[:, i] == best[:, p]) & ~taken[p])
            taken[p] = taken[p] | kept[i]
        kept = torch.stack(kept, 1)
        count = kept.sum(1).to(torch.int32)
        path = torch.where(kept, torch.arange(n, device="cuda"), n).sort(1).values.to(torch.int32)
        for layer in self.layers:
            binding.kvb_accept(layer.blocks, batch, path, count, new_len=self.new_len)
        self.kv_len.copy_(self.new_len)
        last = path.long().gather(1, (count - 1).long()[:, None])
        self.token.copy_(best.gather(1, last)[:, 0])
        # what followed node 0 is the first guess next time, what was the first the second
        seen, follows = tokens[:, 0], best[:, 0]
        self.successors[seen, 1] = torch.where(self.successors[seen, 0] == follows, self.successors[seen, 1],
                                               self.successors[seen, 0])
        self.successors[seen, 0] = follows
        return tokens, kept, x

    def step(self):
        """One tree of every sequence.  Returns its tokens [B][n], which of them are kept, and their last hidden states."""
        if self.held + self.n > self.room:
            raise ValueError("the cache is full")
        if self.graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                self.out = self._step()
            self.graph = graph
        self.graph.replay()
        self.held += int(self.out[1].sum(1).max())  # for the bound alone; a program may bound it by the tree's depth
        return self.out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--format", choices=["int8", "e4m3"], default="int8")
    a = p.parse_args()
    fmt = torch.int8 if a.format == "int8" else torch.float8_e4m3fn
    stack = Stack(B=a.batch, room=a.prompt + (a.steps + 1) * len(PARENTS), fmt=fmt)
    gen = torch.Generator("cuda").manual_seed(1)
    stack.prompt(torch.randint(0, stack.vocab, (a.batch, a.prompt), generator=gen, device="cuda"))
    stack.step()  # captures the step
    torch.cuda.synchronize()
    t, tokens = time.perf_counter(), 0
    for _ in range(a.steps):
        tokens += int(stack.step()[1].sum())
    t = (time.perf_counter() - t) / max(a.steps, 1)
    print(f"{a.batch} sequences, {a.prompt} prompt tokens, {a.steps} steps of {len(PARENTS)} drafts: "
          f"{tokens / max(a.steps * a.batch, 1):.2f} tokens per step and sequence, {t * 1e6:.0f} us per step")


if __name__ == "__main__":
    main()
