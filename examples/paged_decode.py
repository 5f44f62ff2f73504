"""A server's attention on int8: int8 linears, the int8 key/value cache and the attention that reads it, run as
they would be for several users.

    python examples/paged_decode.py [--layers 2] [--users 4] [--steps 16]

Prompts of different lengths are written in one call, then every step adds a token to each user; half way one
user leaves, and the pages that this frees go to a new one. At the end the cache is read back and the last step
is checked against attention in 64 bits over what was read. Weights and hidden states are random.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_int8_amd as m8  # noqa: E402


def check(cache, seqs, ids, q, out):
    """The largest error of one new token's attention per user, in units of the largest value that it sees."""
    k, v = m8.llmint8_kv_gather(cache, seqs.whole(ids), q.dtype)
    worst, at, G = 0.0, 0, q.shape[1] // cache.heads
    for b, s in enumerate(ids):
        n = seqs.length(s)
        ks, vs = (x[at:at + n].double().cpu().repeat_interleave(G, 1).transpose(0, 1).contiguous() for x in (k, v))
        w = torch.softmax(ks @ q[b].double().cpu()[:, :, None] / cache.dim ** 0.5, 1)
        want = (w * vs).sum(1)
        worst = max(worst, float((out[b].double().cpu() - want).abs().max() / vs.abs().max()))
        at += n
    return worst


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--users", type=int, default=4)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--q-heads", type=int, default=32)
    p.add_argument("--heads", type=int, default=8)
    p.add_argument("--dim", type=int, default=128)
    p.add_argument("--context", type=int, default=2000, help="longest prompt")
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    hidden = a.q_heads * a.dim
    new = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731

    prompts = [max(1, a.context * (u + 1) // a.users) for u in range(a.users)]
    pages = sum(-(-(n + a.steps + 1) // 64) for n in prompts)
    freq, mag = m8.rope_frequencies(a.dim)
    rope = m8.llmint8_rope_table(freq, a.context + a.steps + 1, mag)
    caches = [m8.KVCache.empty(pages, a.heads, a.dim) for _ in range(a.layers)]
    layers = [m8.Int8SelfAttention((new((a.q_heads + 2 * a.heads) * a.dim, hidden) / hidden ** 0.5).half(),
                                   (new(hidden, hidden) / hidden ** 0.5).half(), a.q_heads, c, rope=rope)
              for c in caches]
    seqs = m8.PagedSequences(caches[0])  # the layers' caches have the same pages, and one table serves them all

    def step(ids, counts):
        batch = seqs.extend(ids, counts)
        x = new(sum(counts), hidden).half()
        for layer in layers:
            x = x + layer(x, batch)
        return x, batch

    ids = [seqs.add() for _ in prompts]
    step(ids, prompts)
    torch.cuda.synchronize()
    began = time.perf_counter()
    for i in range(a.steps):
        if i == a.steps // 2:
            seqs.release(ids.pop(0))
            ids.append(seqs.add())
            counts = [1] * (len(ids) - 1) + [prompts[0]]  # a prompt and the others' tokens in one call
        else:
            counts = [1] * len(ids)
        x, batch = step(ids, counts)
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    # one more token of every user, kept apart: q as it is written, what attention gives, and the cache read back
    batch = seqs.extend(ids, [1] * len(ids))
    n, c = len(ids), caches[0]
    k, v, q = (new(n, h, a.dim).half() for h in (a.heads, a.heads, a.q_heads))
    q = m8.llmint8_kv_append(c, batch, k, v, q=q, rope=rope)
    err = check(c, seqs, ids, q, m8.llmint8_kv_attention(c, batch, q))
    held = sum(seqs.length(s) for s in ids)
    print(f"{a.layers} layers, {n} users, {held} tokens in the cache: {c.memory_bytes() / c.pages / c.page:.0f} bytes "
          f"a token and layer ({4 * a.heads * a.dim} in 16 bits), {seqs.free_pages()} of {c.pages} pages free")
    print(f"{a.steps} steps, the new user's prompt among them: {took / a.steps * 1e3:.3f} ms a step")
    print(f"attention against 64 bits over the cache read back: {err:.1e} of the largest value")
    assert torch.isfinite(x).all() and err < 4e-3, err
    return err


if __name__ == "__main__":
    main()
