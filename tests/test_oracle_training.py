"""The training operators' oracle against other derivations: gradients against differences and against the graph of
the forward formula in 64 bits, rotations against complex numbers, hand values."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import training_oracle as ref

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("lens,hq,hk,how", [
    ([5, 1, 0, 7], 4, 2, {}), ([6, 9], 3, 1, {"causal": False}), ([12], 2, 2, {"window": 3, "sinks": 2}),
    ([4, 8], 2, 1, {"window": 1}), ([7], 6, 3, {"window": 20, "sinks": 1}),
])
def test_attention_against_differences_and_the_graph(lens, hq, hk, how):
    rng = np.random.default_rng(len(lens) + hq)
    T, D, scale = sum(lens), 5, 0.7
    q, k, v = (rng.standard_normal((T, h, D)) for h in (hq, hk, hk))
    do = rng.standard_normal((T, hq, D))
    r = ref.attention(lens, q, k, v, scale, dout=do, **how)

    def loss(q, k, v):
        return (ref.attention(lens, q, k, v, scale, **how)["out"] * do).sum()

    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in x.shape)
            h = 1e-5
            up, down = x.copy(), x.copy()
            up[at] += h
            down[at] -= h
            args = {"dq": (q, k, v), "dk": (q, k, v), "dv": (q, k, v)}[name]
            pick = {"dq": 0, "dk": 1, "dv": 2}[name]
            hi, lo = list(args), list(args)
            hi[pick], lo[pick] = up, down
            d = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(d - r[name][at]) <= 1e-7 * max(1, abs(d)), (name, at)
    # the graph of the formula
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    outs, at = [], 0
    for n in lens:
        kk = tk[at:at + n].repeat_interleave(hq // hk, 1)
        vv = tv[at:at + n].repeat_interleave(hq // hk, 1)
        s = torch.einsum("ihc,jhc->hij", tq[at:at + n], kk) * scale
        see = torch.tensor([[(not how.get("causal", True)) or (j <= i and (
            not how.get("window") or j > i - how["window"] or j < how.get("sinks", 0))) for j in range(n)] for i in range(n)],
            dtype=torch.bool).reshape(n, n)
        s = s.masked_fill(~see, -np.inf)
        outs.append(torch.einsum("hij,jhc->ihc", torch.softmax(s, -1), vv))
        at += n
    out = torch.cat(outs)
    assert np.allclose(out.detach().numpy(), r["out"], atol=1e-13)
    out.backward(torch.tensor(do))
    for t, name in ((tq, "dq"), (tk, "dk"), (tv, "dv")):
        assert np.allclose(t.grad.numpy(), r[name], atol=1e-12)


def test_attention_by_hand():
    """Two tokens, one channel: the second row weighs 1 : e."""
    q, k, v = np.array([[[0.0]], [[1.0]]]), np.array([[[0.0]], [[1.0]]]), np.array([[[10.0]], [[20.0]]])
    r = ref.attention([2], q, k, v, 1.0)
    w = np.e / (1 + np.e)
    assert np.allclose(r["out"][:, 0, 0], [10, 10 + 10 * w]) and np.allclose(r["lse"][:, 0], [0, np.log(1 + np.e)])
    assert ref.visible(5, True, 2, 1).astype(int).tolist() == [
        [1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations_are_complex_products(interleaved):
    rng = np.random.default_rng(1)
    T, H, D, rot, axis = 6, 3, 10, 8, np.array([0, 1, 1, 0])
    table = rng.standard_normal((20, rot)).astype(np.float32)
    angle = rng.uniform(0, 6, (20, rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = rng.integers(0, 20, (T, 2))
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    y = ref.rope(x, table, pos, axis, interleaved)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle[pos[:, axis], np.arange(4)])[:, None]
    assert np.allclose(y[..., a], z.real, atol=1e-6) and np.allclose(y[..., b], z.imag, atol=1e-6)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    back = ref.rope(y, table, pos, axis, interleaved, inverse=True)
    assert np.allclose(back, x, atol=1e-6)


@pytest.mark.parametrize("affine", [False, True])
def test_layer_norm_against_differences(affine):
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((4, 7)) * 3 + 1, rng.standard_normal((4, 7))
    w, b = (1 + rng.standard_normal(7), rng.standard_normal(7)) if affine else (None, None)
    r = ref.layer_norm(x, w, b, 1e-3, dy)

    def loss(x, w, b):
        return (ref.layer_norm(x, w, b, 1e-3)["y"] * dy).sum()

    for name, pick in (("dx", 0), ("dw", 1), ("db", 2)) if affine else (("dx", 0),):
        args = [x, w, b]
        for at in np.ndindex(args[pick].shape):
            hi, lo = list(args), list(args)
            hi[pick], lo[pick] = args[pick].copy(), args[pick].copy()
            hi[pick][at] += 1e-5
            lo[pick][at] -= 1e-5
            d = (loss(*hi) - loss(*lo)) / 2e-5
            assert abs(d - r[name][at]) <= 1e-7 * max(1, abs(d)), (name, at)


def test_norm_and_factor_by_hand():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    assert ref.grad_norm(g) == 5.0 and ref.grad_norm(g, 0.5) == 2.5
    assert ref.grad_factor(5.0, 10.0) == 1.0 and abs(ref.grad_factor(5.0, 1.0) - 0.2) < 1e-6
    assert ref.grad_factor(5.0, np.inf, 0.25) == 0.25
