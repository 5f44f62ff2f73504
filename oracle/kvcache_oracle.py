"""Plain CPU form of the int8 key/value cache: codes and magnitudes in the fp32 operations of the
definition (bit for bit), attention in 64 bits. Sequence by sequence, page by page, head by head.

16-bit rows come in as float32 arrays holding their exact values.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["KVOracle", "rope_table"]

F32 = np.float32
TINY = F32(2.0 ** -64)


def rope_table(freq, rows, mag=1.0):
    """[rows, 2 len(freq)] fp32: mag cos(p f_i), then mag sin(p f_i), in 64 bits."""
    ang = np.arange(rows, dtype=np.float64)[:, None] * np.asarray(freq, np.float64)
    return np.concatenate([mag * np.cos(ang), mag * np.sin(ang)], 1).astype(np.float32)


class KVOracle:
    """K codes [pages, heads, page, dim], V codes [pages, heads, dim, page], aK, aV [pages, heads]."""

    def __init__(self, K, V, aK, aV):
        self.K, self.V = np.array(K), np.array(V)
        self.aK, self.aV = np.array(aK, F32), np.array(aV, F32)
        self.pages, self.heads, self.page, self.dim = self.K.shape

    @staticmethod
    def rotate(x, table, pos, interleaved):
        """x float32 [heads, dim] at position pos; every product and sum rounded to fp32."""
        if table is None:
            return x
        rot = table.shape[1]
        half = rot // 2
        row = table[min(max(pos, 0), table.shape[0] - 1)]
        c, s = row[:half], row[half:]
        y = x.copy()
        i1 = np.arange(0, rot, 2) if interleaved else np.arange(half)
        i2 = i1 + 1 if interleaved else i1 + half
        y[:, i1] = (x[:, i1] * c).astype(F32) - (x[:, i2] * s).astype(F32)
        y[:, i2] = (x[:, i2] * c).astype(F32) + (x[:, i1] * s).astype(F32)
        return y

    def _put(self, codes, amax, page, head, s0, x):
        """x float32 [n, dim] into slots s0.. of the page; codes is the [page, dim] view."""
        old = F32(0) if s0 == 0 else amax[page, head]
        a = max(old, F32(np.abs(x).max()) if x.size else F32(0))
        if a < TINY:
            a = F32(0)
        if s0 > 0 and a > old:
            r = F32(old / a)
            codes[:s0] = np.rint((codes[:s0].astype(F32) * r).astype(F32)).astype(np.int8)
        s = F32(F32(127) / a) if a > 0 else F32(0)
        codes[s0:s0 + len(x)] = np.rint((x * s).astype(F32)).astype(np.int8)
        amax[page, head] = a

    def page_of(self, table, b, j):
        e = j // self.page
        if e >= table.shape[1]:
            return -1
        p = int(table[b, e])
        return p if 0 <= p < self.pages else -1

    def append(self, cu, length, table, k, v, q=None, rope=None, interleaved=False):
        """k, v [rows, heads, dim], q [rows, q_heads, dim]; returns q rotated (float32, not rounded)."""
        q_out = None if q is None else np.array(q)
        for b in range(len(length)):
            n = int(cu[b + 1] - cu[b])
            first = int(length[b]) - n
            todo = {}
            for i in range(n):
                pos, row = first + i, int(cu[b]) + i
                if pos < 0:
                    continue
                todo.setdefault(pos // self.page, []).append((pos, row))
                if q is not None:
                    q_out[row] = self.rotate(q[row], rope, pos, interleaved)
            for e, tokens in todo.items():
                p = self.page_of(table, b, e * self.page)
                if p < 0:
                    continue
                s0 = tokens[0][0] % self.page
                rk = np.stack([self.rotate(k[row], rope, pos, interleaved) for pos, row in tokens])
                rv = np.stack([v[row] for _, row in tokens])
                for h in range(self.heads):
                    self._put(self.K[p, h], self.aK, p, h, s0, rk[:, h])
                    self._put(self.V[p, h].T, self.aV, p, h, s0, rv[:, h])
        return q_out

    def tokens(self, table, b, lo, hi):
        """(k, v, exists): float32 [hi - lo, heads, dim] values of tokens lo..hi-1 of sequence b."""
        n = max(hi - lo, 0)
        k = np.zeros((n, self.heads, self.dim), F32)
        v = np.zeros((n, self.heads, self.dim), F32)
        there = np.zeros(n, bool)
        for j in range(lo, hi):
            p = self.page_of(table, b, j)
            if p < 0:
                continue
            there[j - lo] = True
            s = j % self.page
            k[j - lo] = self.K[p, :, s].astype(F32) * (self.aK[p] / F32(127))[:, None]
            v[j - lo] = self.V[p, :, :, s].astype(F32) * (self.aV[p] / F32(127))[:, None]
        return k, v, there

    def attention(self, cu, length, table, q, scale=None, causal=True, window=0, sinks=0):
        """(out, lse, tol) in 64 bits, [rows, q_heads, dim], [rows, q_heads] and, for each row, the largest
        |v| it sees and the change of a logit that q held to 2^-16 of its largest channel can make."""
        rows, hq, D = q.shape
        G = hq // self.heads
        scale = 1.0 / math.sqrt(D) if scale is None else scale
        out = np.zeros((rows, hq, D))
        lse = np.full((rows, hq), -np.inf)
        vmax = np.zeros((rows, hq))
        dlogit = np.zeros((rows, hq))
        room = table.shape[1] * self.page
        for b in range(len(length)):
            n, whole = int(cu[b + 1] - cu[b]), int(length[b])
            L = min(whole, room)  # tokens past the table have no page
            if n == 0:
                continue
            k, v, there = self.tokens(table, b, 0, L)
            k, v = k.astype(np.float64), v.astype(np.float64)
            j = np.arange(L)
            for i in range(n):
                pos, row = whole - n + i, int(cu[b]) + i
                see = there.copy()
                if causal:
                    see &= j <= pos
                if window > 0:
                    see &= (j > pos - window) | (j < sinks)
                if not see.any():
                    continue
                for h in range(hq):
                    kk, vv, qq = k[see][:, h // G], v[see][:, h // G], q[row, h].astype(np.float64)
                    s = scale * (kk @ qq)
                    m = s.max()
                    p = np.exp(s - m)
                    out[row, h] = (p @ vv) / p.sum()
                    lse[row, h] = m + np.log(p.sum())
                    vmax[row, h] = np.abs(vv).max()
                    dlogit[row, h] = abs(scale) * np.abs(qq).max() * 2.0 ** -16 * np.abs(kk).sum(1).max()
        return out, lse, (vmax, dlogit)
