"""The training operators in 64 bits, from their formulas: attention of packed sequences with its gradients,
rotary positions with axes, layer norm with its gradients, the norm of gradients. Test infrastructure."""
from __future__ import annotations

import numpy as np


def visible(n, causal, window=0, sinks=0):
    """[n, n]: whether row i sees token j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    if not causal:
        return np.ones((n, n), bool)
    see = j <= i
    if window > 0:
        see &= (j > i - window) | (j < sinks)
    return see


def attention(lens, q, k, v, scale, causal=True, window=0, sinks=0, dout=None, unit=None, floor=False, few=False):
    """Packed sequences of ``lens`` tokens; q [T, hq, D], k and v [T, hk, D]. A dict of out, lse and, with ``dout``,
    dq, dk, dv; with ``unit`` (half a step of the 16-bit type) also of ``e_out`` and so on: how far a result may be
    off whose products take P and dS rounded to the type, with fp32 logits and sums (``floor``: the type is fp16,
    which holds them to a floor as well; ``few``: delta is summed from P and dP, not from the rounded
    o, and P and dS enter the gradients' products to twice the type's bits)."""
    T, hq, D = q.shape
    hk, G = k.shape[1], hq // k.shape[1]
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    r = {"out": np.zeros((T, hq, D)), "lse": np.full((T, hq), -np.inf)}
    if dout is not None:
        dout = dout.astype(np.float64)
        r.update(dq=np.zeros((T, hq, D)), dk=np.zeros((T, hk, D)), dv=np.zeros((T, hk, D)))
    if unit is not None:
        r.update({"e_" + n: np.zeros_like(x) for n, x in r.items()})
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        see = visible(n, causal, window, sinks)
        for h in range(hq):
            g = h // G
            qi, ki, vi = q[rows, h], k[rows, g], v[rows, g]
            s = np.where(see, scale * (qi @ ki.T), -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            p /= total
            o = p @ vi
            r["out"][rows, h] = o
            r["lse"][rows, h] = (m + np.log(total))[:, 0]
            if dout is not None:
                do = dout[rows, h]
                dp = do @ vi.T
                delta = (do * o).sum(1, keepdims=True)
                ds = p * (dp - delta)
                r["dq"][rows, h] = scale * ds @ ki
                r["dk"][rows, g] += scale * ds.T @ qi
                r["dv"][rows, g] += p.T @ do
            if unit is None:
                continue
            f32 = 2.0 ** -24
            # a logit in fp32: its sum of D products, and what is done to it after
            d = np.where(see, abs(scale) * (np.abs(qi) @ np.abs(ki.T)) * (D + 8) * f32 + 8 * np.abs(np.where(see, s, 0)) * f32, 0)
            d_row = d.max(1, keepdims=True)
            sums = n * f32 + 2.0 ** -18  # of weights; the hardware's exponentials and reciprocals
            e_p = p * (unit + d + d_row + sums)
            if floor:
                e_p = e_p + see * 2.0 ** -32
            e_o = e_p @ np.abs(vi) + n * f32 * (p @ np.abs(vi)) + unit * np.abs(o)
            r["e_out"][rows, h] = e_o
            r["e_lse"][rows, h] = d_row[:, 0] + sums + 2.0 ** -20 * np.abs(r["lse"][rows, h])
            if dout is None:
                continue
            e_delta = (np.abs(do) * (e_o + D * f32 * np.abs(o))).sum(1, keepdims=True)
            e_dp = (D + 2) * f32 * (np.abs(do) @ np.abs(vi.T))
            e_w = d + d_row + sums + 8 * np.abs(r["lse"][rows, h])[:, None] * f32  # of a weight before it is rounded
            if few:
                e_delta = (p * (np.abs(dp) * (e_w + (n + 2) * f32) + e_dp)).sum(1, keepdims=True)
            u = unit * unit if few else unit
            e_ds = np.abs(ds) * (u + e_w) + p * (1 + e_w) * (e_dp + e_delta)
            e_q = e_k = e_ds
            if floor:
                e_q = e_ds + 2.0 ** -32 * np.abs(ds).max(1, keepdims=True)
                e_k = e_ds + 2.0 ** -32 * np.abs(ds).max(0, keepdims=True)
            e_pv = p * (u + e_w) + (2.0 ** -39 if floor else 0.0)
            acc = (n + 8) * f32
            r["e_dq"][rows, h] = abs(scale) * (e_q @ np.abs(ki) + acc * np.abs(ds) @ np.abs(ki))
            r["e_dk"][rows, g] += abs(scale) * (e_k.T @ np.abs(qi) + G * acc * np.abs(ds).T @ np.abs(qi))
            r["e_dv"][rows, g] += e_pv.T @ np.abs(do) + G * acc * p.T @ np.abs(do)
    if unit is not None and dout is not None:
        for name in ("dq", "dk", "dv"):
            r["e_" + name] += unit * np.abs(r[name])
    return r


def rope(x, table, pos, axis, interleaved=False, inverse=False):
    """x fp32 [T, H, D], table fp32 [positions, rot], pos [T, axes]: fp32, each product and sum rounded."""
    rot = table.shape[1]
    half = rot // 2
    y = x.astype(np.float32).copy()
    p = np.clip(pos[:, axis], 0, len(table) - 1)                                # [T, half]
    c = table[p, np.arange(half)][:, None].astype(np.float32)
    s = table[p, half + np.arange(half)][:, None].astype(np.float32)
    s = -s if inverse else s
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    x1, x2 = y[..., a].copy(), y[..., b].copy()
    y[..., a] = x1 * c - x2 * s
    y[..., b] = x2 * c + x1 * s
    return y


def layer_norm(x, w, b, eps, dy=None):
    """A dict of y, mean, rstd and, with ``dy``, dx, dw, db in 64 bits."""
    x = x.astype(np.float64)
    K = x.shape[1]
    w = np.ones(K) if w is None else w.astype(np.float64)
    b = np.zeros(K) if b is None else b.astype(np.float64)
    mean = x.mean(1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    xh = (x - mean) * rstd
    r = {"y": xh * w + b, "mean": mean[:, 0], "rstd": rstd[:, 0], "xh": xh}
    if dy is not None:
        dy = dy.astype(np.float64)
        g = dy * w
        r["dx"] = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
        r["dw"], r["db"] = (dy * xh).sum(0), dy.sum(0)
    return r


def grad_norm(grads, scale=1.0):
    return scale * np.sqrt(sum(np.square(g.astype(np.float64)).sum() for g in grads))


def grad_factor(norm, max_norm, scale=1.0):
    """The factor in fp32, from the fp32 norm."""
    return np.float32(scale * min(1.0, max_norm / (float(norm) + 1e-6)))
