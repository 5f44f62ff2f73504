"""Training adapters on layers of int8 weights: documents of different lengths packed into one row, attention with
its gradient, rotary positions, layer norms with parameters, low-rank adapters beside the frozen int8 linears,
and gradients clipped by their norm.

    python examples/adapter_training.py [--layers 2] [--steps 10] [--tokens 2000]

The model learns to give back the hidden states of a copy of itself with other norms. Weights and hidden states
are random.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_int8_amd as m8  # noqa: E402


class Block(torch.nn.Module):
    """x + attention(norm(x) and an adapter's part of it), frozen but for the norm and the adapter."""

    def __init__(self, hidden, q_heads, heads, dim, rank, rope, generator):
        super().__init__()
        new = lambda *shape: torch.randn(shape, device="cuda", generator=generator)  # noqa: E731
        self.weight = torch.nn.Parameter(torch.ones(hidden, device="cuda"))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, device="cuda"))
        self.down = torch.nn.Parameter(new(rank, hidden) / hidden ** 0.5)
        self.up = torch.nn.Parameter(torch.zeros(hidden, rank, device="cuda"))
        self.attention = m8.Int8SelfAttention((new((q_heads + 2 * heads) * dim, hidden) / hidden ** 0.5).bfloat16(),
                                              (new(hidden, q_heads * dim) / hidden ** 0.5).bfloat16(), q_heads, None,
                                              rope=rope, heads=heads, dim=dim)

    def forward(self, x, rows):
        h = m8.layer_norm(x, self.weight, self.bias)
        h = h + ((h.float() @ self.down.t()) @ self.up.t()).to(h.dtype)
        return x + self.attention.packed(h, rows)


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--tokens", type=int, default=2000, help="of a step, in documents of different lengths")
    p.add_argument("--q-heads", type=int, default=16)
    p.add_argument("--heads", type=int, default=4)
    p.add_argument("--dim", type=int, default=64)
    p.add_argument("--rank", type=int, default=8)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden = a.q_heads * a.dim
    rope = m8.llmint8_rope_table(m8.rope_frequencies(a.dim)[0], a.tokens)
    blocks = torch.nn.ModuleList(Block(hidden, a.q_heads, a.heads, a.dim, a.rank, rope, g) for _ in range(a.layers))
    lens = [a.tokens // 2, a.tokens // 3, a.tokens // 8]
    rows = m8.PackedRows.of(lens, rows=a.tokens)  # the rest of the rows is nobody's

    def run(x):
        for b in blocks:
            x = b(x, rows)
        return x

    x = torch.randn(a.tokens, hidden, device="cuda", generator=g).bfloat16()
    with torch.no_grad():
        kept = [p.clone() for p in blocks.parameters()]
        for b in blocks:
            b.weight.mul_(torch.rand(hidden, device="cuda", generator=g) + 0.5)
        target = run(x)
        for q, k in zip(blocks.parameters(), kept):
            q.copy_(k)
    optimizer = torch.optim.AdamW(blocks.parameters(), lr=1e-3, weight_decay=0.0)
    used = sum(lens)
    losses, norms, start = [], [], time.perf_counter()
    for _ in range(a.steps):
        optimizer.zero_grad(set_to_none=True)
        loss = (run(x)[:used].float() - target[:used].float()).square().mean()
        loss.backward()
        norms.append(m8.clip_grad_norm(blocks.parameters(), 0.1))
        optimizer.step()
        losses.append(loss.detach())
    torch.cuda.synchronize()
    ms = (time.perf_counter() - start) / a.steps * 1e3
    print(f"{a.steps} steps of {used} tokens: loss {float(losses[0]):.4f} to {float(losses[-1]):.4f}, "
          f"norm of the gradients {float(norms[0]):.3f} to {float(norms[-1]):.3f}, {ms:.2f} ms a step")
    return blocks, losses, norms


if __name__ == "__main__":
    main()
