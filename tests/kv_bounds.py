"""Attention over the int8 key/value cache in 64 bits with a bound of the kernels' error for every output, and
data on which that bound is small against what any 64 tokens contribute.

Per row (query row and head), weights p_j = softmax_j, values v_j, o = sum_j p_j v_j, A = sum_j p_j |v_j|:
  |o' - o| <= u |o| + max(Q + S, F) + E A      u: unit roundoff of the output type
The 8-bit products hold q as integers of max|q| / 32639, h = half of one: with e (|e_c| <= h) the change of q,
  Q = h scale sum_c |sum_j p_j k_jc (v_j - o)| + 1.5 d^2 (A + |o|),  d = h scale max_j sum_c |k_jc|
to first order and (exp and the sum's own change) second; their weights are integers of 1 / 32639 of the largest of
their 64 tokens, V's scale (a per code) among them:
  S = sum over tiles (max_j p_j a_j) / 65278 sum_j |code_j|
The 16-bit products round each weight by 2^-11, those under 2^-14 to 2^-25 of 2^-8 of the row's largest: F = 2^-11 A
+ 2^-31 sum_j |code_j| max_j p_j a_j (q is exact, or to 2^-38 of its largest channel).
E, in units of 2^-24 and twice (the weight and the sum): a logit's scale and sum, eight roundings of |s| + |log2 a|;
its products' sum in fp32, a rounding of sum_c |q_c k_c| for every 16 channels and five more; exponentials,
logarithms, reciprocals of the hardware and the join, 24; the sums over a row's tokens, one for every 16 of them and
one a tile.
lse: h scale sum_c |sum_j p_j k_jc| + 1.5 d^2 + 2 E + 2^-23 |lse|.
"""
from __future__ import annotations

import math

import numpy as np

import oracle

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


class Data:
    """Cache, batch and q with logits of a few units and pages of like magnitudes: no 64 tokens outweigh the rest."""

    def __init__(self, seed, lens, counts, heads, q_heads, dim, page, dtype, dominant=0.0):
        import torch
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.counts, self.q_heads, self.dtype = list(lens), list(counts), q_heads, dtype
        need = [max(1, -(-n // page)) for n in lens]
        pages = sum(need) + 1
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        K = rng.integers(-127, 128, (pages, heads, page, dim), dtype=np.int8)
        V = rng.integers(-127, 128, (pages, heads, dim, page), dtype=np.int8)
        aK, aV = ((0.7 + 0.6 * rng.random((pages, heads))).astype(np.float32) for _ in range(2))
        self.ref = oracle.KVOracle(K, V, aK, aV)
        q = rng.standard_normal((self.rows, q_heads, dim)).astype(np.float32)
        if dominant:  # one channel of q far above the others, where the keys hold nearly nothing
            q[..., 3] = dominant * np.sign(q[..., 3])
            self.ref.K[..., 3] = rng.integers(-1, 2, K.shape[:-1], dtype=np.int8)
        self.q = torch.from_numpy(q).to(torch.float16 if dtype == "f16" else torch.bfloat16)

    def tokens(self, b, h):
        """(k, v, a per code of v, codes of v) of sequence b and head h, [tokens, dim] in 64 bits."""
        r, n = self.ref, self.lens[b]
        ids = self.table[b, :max(1, -(-n // r.page))]
        ak, av = r.aK[ids, h].astype(np.float64) / 127, r.aV[ids, h].astype(np.float64) / 127
        k = r.K[ids, h].astype(np.float64).reshape(-1, r.dim)[:n]
        c = r.V[ids, h].astype(np.float64).transpose(0, 2, 1).reshape(-1, r.dim)[:n]
        a = np.repeat(av, r.page)[:n, None]
        return k * np.repeat(ak, r.page)[:n, None], c * a, a, c

    def groups(self, scale=None, causal=True, window=0, sinks=0):
        """For every sequence and head with rows: (rows of the call, query heads, the rows' results), a row for
        each token and query head of the group."""
        r, G = self.ref, self.q_heads // self.ref.heads
        scale = 1.0 / math.sqrt(r.dim) if scale is None else scale
        q = self.q.double().numpy()
        for b, n in enumerate(self.counts):
            L = self.lens[b]
            if n == 0:
                continue
            pos, j = np.arange(L - n, L)[:, None], np.arange(L)
            see = (j <= pos) if causal else np.ones((n, L), bool)
            if window:
                see &= (j > pos - window) | (j < sinks)
            for h in range(r.heads):
                at, heads = slice(self.cu[b], self.cu[b + 1]), slice(h * G, h * G + G)
                yield at, heads, Rows(q[at, heads].reshape(n * G, r.dim), *self.tokens(b, h), see.repeat(G, 0), scale,
                                      U[self.dtype])


class Rows:
    """Results and bounds of rows that read the same tokens."""

    def __init__(self, q, k, v, a, codes, see, scale, u):
        s = np.where(see, scale * (q @ k.T), -np.inf)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        self.p = p = e / e.sum(1, keepdims=True)
        self.v, self.see = v, see
        self.o, self.lse = p @ v, (top + np.log(e.sum(1, keepdims=True)))[:, 0]
        A = p @ np.abs(v)
        h = np.abs(q).max(1, keepdims=True) / 65278
        # sum_c |sum_j p_j k_jc (v_jx - o_x)|, row by row
        cov = np.stack([np.abs(k.T @ (p[i][:, None] * v) - np.outer(k.T @ p[i], self.o[i])).sum(0) for i in range(len(q))])
        d = h * abs(scale) * np.where(see, np.abs(k).sum(1), 0).max(1, keepdims=True)
        Q = h * abs(scale) * cov + 1.5 * d * d * (A + np.abs(self.o))
        tiles = range(0, k.shape[0], 64)
        pa = p * a.T
        S = sum(pa[:, t:t + 64].max(1, keepdims=True) * np.abs(codes[t:t + 64]).sum(0) for t in tiles) / 65278
        F = 2.0 ** -11 * A + 2.0 ** -31 * pa.max(1, keepdims=True) * (see.astype(float) @ np.abs(codes))
        F += 2.0 ** -14 * Q  # q of the 16-bit products
        size = np.where(see, np.abs(s), 0).max(1, keepdims=True) + np.abs(np.log2(a)).max()
        whole = np.where(see, abs(scale) * (np.abs(q) @ np.abs(k).T), 0).max(1, keepdims=True)
        E = 2.0 ** -24 * (8 * size + (k.shape[1] / 16 + 5) * whole + 24 + 5 * len(tiles))
        self.exact_q_tol = u * np.abs(self.o) + F + 2 * E * A + 2.0 ** -25
        self.tol = u * np.abs(self.o) + np.maximum(Q + S, F) + 2 * E * A + 2.0 ** -25
        self.lse_tol = (h * abs(scale) * np.abs(p @ k).sum(1, keepdims=True) + 1.5 * d * d + 2 * E)[:, 0] + 2.0 ** -23 * np.abs(self.lse)

    def share(self, t):
        """What the 64 tokens from t on contribute to each row's output, and their weight."""
        return self.p[:, t:t + 64] @ self.v[t:t + 64], self.p[:, t:t + 64].sum(1, keepdims=True)


# lens, counts, heads, query heads, dim, page, dtype, options
CASES = [
    ([9000], [1], 1, 2, 64, 64, "f16", {}),                                       # single rows in parts, joined
    ([9000, 20], [4, 2], 1, 2, 64, 16, "bf16", {}),
    ([40] * 520 + [5000], [1] * 521, 1, 2, 64, 16, "bf16", {}),
    ([5000] + [30] * 99, [1] * 100, 1, 32, 32, 64, "f16", {}),                    # more than 2048 rows to join
    ([4000, 300], [1, 1], 2, 8, 128, 64, "f16", {}),
    ([3000, 2500], [5, 5], 2, 10, 96, 32, "bf16", {}),                            # two sixteens of rows
    ([2600, 700], [1, 1], 1, 4, 256, 128, "f16", {}),
    ([700, 650, 90], [1, 1, 1], 2, 4, 80, 16, "bf16", {}),                        # whole
    ([2600, 3, 4100], [9, 3, 7], 2, 4, 128, 16, "bf16", {"window": 2500, "sinks": 70}),
    ([5000], [200], 1, 1, 128, 64, "f16", {}),                                    # a prompt's tokens in parts
    ([5000], [150], 1, 1, 80, 16, "bf16", {}),
    ([3000, 1500], [40, 100], 1, 2, 256, 32, "f16", {}),
    ([1000, 300], [150, 300], 2, 2, 64, 64, "bf16", {}),                          # whole
    ([700], [130], 2, 2, 64, 128, "bf16", {"causal": False}),
    ([1500, 900], [130, 40], 1, 2, 64, 16, "f16", {"window": 600, "sinks": 64}),
    # single tokens and a prompt in one call, on either side of the average that chooses the kernel
    ([800, 1300, 400, 900, 600], [1, 1, 1, 1, 200], 2, 4, 128, 64, "bf16", {}),
    ([500] * 40 + [700], [1] * 40 + [150], 1, 4, 64, 16, "f16", {}),
]


def name(case):
    lens, counts, heads, q_heads, dim, page, dtype, kw = case
    return f"{len(lens)}x{max(lens)}-{max(counts)}-{q_heads}/{heads}-{dim}-{page}-{dtype}" + "".join(f"-{k}{v}" for k, v in kw.items())
