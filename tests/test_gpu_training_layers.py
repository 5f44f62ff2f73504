"""The training operators as they are used: differentiable functions, the attention layer's training form against
its parts and its serving form, clipping of parameters' gradients, all of them in one step."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import training_oracle as ref

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


def randn(seed, *shape, dtype=torch.float16, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale
    return torch.from_numpy(x).cuda().to(dtype)


def leaf(t):
    return t.detach().clone().requires_grad_()


def test_functions_have_the_library_s_gradients():
    print("[case] functions", flush=True)
    b = m8.PackedRows.of([50, 70], rows=130)
    q, k, v, g = (randn(i, 130, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    for how in ({}, {"causal": False}, {"window": 20, "sinks": 2, "scale": 0.2}):
        tq, tk, tv = map(leaf, (q, k, v))
        out = m8.packed_attention(tq, tk, tv, b, **how)
        out.backward(g)
        want, lse = m8.llmint8_attention(b, q, k, v, **how)
        grads = m8.llmint8_attention_backward(b, q, k, v, want, lse, g, **how)
        assert torch.equal(out[:120], want[:120]) and (out[120:] == 0).all()
        for t, d in zip((tq, tk, tv), grads):
            assert torch.equal(t.grad[:120], d[:120]) and (t.grad[120:] == 0).all()
    table = m8.llmint8_rope_table(m8.rope_frequencies(64)[0], 200)
    pos = torch.from_numpy(np.random.default_rng(9).integers(0, 200, (130, 2)).astype(np.int32)).cuda()
    axis = m8.rope_axes([20, 12], turns=True)
    tq, tk = leaf(q), leaf(k)
    rq, rk = m8.rotary(tq, tk, table, pos, axis)
    (rq * g).sum().backward(retain_graph=True)
    assert torch.equal(tq.grad, m8.llmint8_rope(table, pos, axis, g, inverse=True)[0]) and (tk.grad == 0).all()
    only, none = m8.rotary(leaf(q), None, table, pos, axis)
    assert none is None and torch.equal(only, rq)
    x, w, bias, dy = randn(20, 4, 33, 100), randn(21, 100), randn(22, 100), randn(23, 4, 33, 100)
    for lw, lb in ((leaf(w), leaf(bias)), (leaf(w), None), (None, leaf(bias)), (None, None), (w, leaf(bias))):
        lx = leaf(x)
        y = m8.layer_norm(lx, lw, lb)
        y.backward(dy)
        flat, stats = m8.llmint8_layer_norm(x.view(-1, 100), None if lw is None else lw.detach(),
                                            None if lb is None else lb.detach())
        dx, dw, db = m8.llmint8_layer_norm_backward(dy.view(-1, 100), x.view(-1, 100), stats,
                                                    None if lw is None else lw.detach(), sums=True)
        assert torch.equal(y.view(-1, 100), flat) and torch.equal(lx.grad.view(-1, 100), dx)
        if lw is not None and lw.requires_grad:
            assert torch.equal(lw.grad, dw)
        if lb is not None:
            assert torch.equal(lb.grad, db)


def test_strided_expanded_and_shared_inputs():
    print("[case] strided", flush=True)
    b = m8.PackedRows.of([40])
    x = randn(1, 40, 4, 64)
    one = leaf(x[:, :1])
    # every head is the same tensor, expanded: the gradient is the sum over the heads
    out = m8.packed_attention(one.expand(40, 4, 64), one, one, b)
    out.sum().backward()  # an expanded gradient of ones
    q, k, v = leaf(x[:, :1].expand(40, 4, 64).contiguous()), leaf(x[:, :1]), leaf(x[:, :1])
    m8.packed_attention(q, k, v, b).backward(torch.ones_like(q))
    want = q.grad.sum(1, keepdim=True).float() + k.grad.float() + v.grad.float()
    assert torch.allclose(one.grad.float(), want, rtol=2 ** -8, atol=2 ** -8 * float(want.abs().max()))
    y = leaf(randn(2, 30, 1).expand(30, 64).contiguous().t().contiguous().t())  # columns first in memory
    z = m8.layer_norm(y * 1.0)
    z.backward(torch.ones_like(z))
    assert y.grad.shape == y.shape and torch.isfinite(y.grad).all()
    two = leaf(x.view(40, -1))
    first, = torch.autograd.grad(m8.layer_norm(two).float().pow(2).sum(), two, create_graph=True)
    with pytest.raises(RuntimeError):  # there are no second derivatives
        first.float().sum().backward()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("how", [{}, {"causal": False}, {"window": 7, "sinks": 1}])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_gradients_of_short_sequences_are_rounded_once(dtype, dim, how):
    """Where sums go over 256 tokens at most, the result's rounding is the only one to count: P and dS take part to
    twice the type's bits, and o, rounded, would bring do times half a step of it into every dS of a row."""
    print(f"[case] short {dtype} {dim} {how}", flush=True)
    lens = [1, 2, 3, 60, 17, 256, 5, 130]
    T = sum(lens)
    q, k, v, do = (randn(200 + i, T, h, dim, dtype=dtype) for i, h in enumerate((4, 2, 2, 4)))
    v = v + 8  # o is far from zero, its rounding as well
    b = m8.PackedRows.of(lens)
    out, lse = m8.llmint8_attention(b, q, k, v, **how)
    grads = m8.llmint8_attention_backward(b, q, k, v, out, lse, do, **how)
    unit = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    host = [t.float().cpu().numpy() for t in (q, k, v)]
    want = ref.attention(lens, *host, np.float32(1 / np.sqrt(dim)), dout=do.float().cpu().numpy(), unit=unit, floor=dtype == torch.float16,
                         few=True, **how)
    for name, t in zip(("dq", "dk", "dv"), grads):
        off = np.abs(t.float().cpu().numpy() - want[name]) / (want["e_" + name] + (2.0 ** -25 if unit == 2.0 ** -11 else 2.0 ** -134))
        print(f"  {name} {off.max():.2f} of its bound", flush=True)
        assert off.max() <= 1


def layer(cache=None, seed=5, hidden=256, nq=4, heads=2, dim=64, dtype=torch.float16, **kw):
    rope = m8.llmint8_rope_table(m8.rope_frequencies(dim)[0], 400)
    if cache is None:
        kw.update(heads=heads, dim=dim)
    return m8.Int8SelfAttention(randn(seed, (nq + 2 * heads) * dim, hidden, dtype=dtype, scale=0.05),
                                randn(seed + 1, hidden, nq * dim, dtype=dtype, scale=0.05), nq, cache, rope, **kw)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("axes", [False, True])
def test_the_layer_is_its_parts(dtype, axes):
    """Bit for bit: norm, int8 linear, rotation, attention, int8 linear, each with its gradient."""
    print(f"[case] layer {dtype} {axes}", flush=True)
    lens, T, hidden, nq, heads, dim = [70, 1, 90], 170, 256, 4, 2, 64
    rows = m8.PackedRows.of(lens, rows=T)
    w, bias = leaf(1 + randn(7, hidden, dtype=torch.float32, scale=0.1)), leaf(randn(8, hidden, dtype=torch.float32, scale=0.1))
    axis = m8.rope_axes([16, 8, 8]) if axes else None
    pos = torch.from_numpy(np.random.default_rng(3).integers(0, 400, (T, 3)).astype(np.int32)).cuda() if axes else None
    net = layer(dtype=dtype, norm=m8.LayerNorm(w, bias), axis=axis, window=50, sinks=3)
    X, g = leaf(randn(10, T, hidden, dtype=dtype)), randn(11, T, hidden, dtype=dtype)
    Y = net.packed(X, rows, pos)
    Y.backward(g)
    X2, w2, b2 = leaf(X), leaf(w), leaf(bias)
    qkv = net.qkv(m8.layer_norm(X2, w2, b2)).view(T, nq + 2 * heads, dim)
    q, k = m8.rotary(qkv[:, :nq], qkv[:, nq:nq + heads], net.rope, rows.positions() if pos is None else pos,
                     axis or [0] * 32)
    o = m8.packed_attention(q, k, qkv[:, nq + heads:], rows, window=50, sinks=3)
    Y2 = net.out(o.view(T, -1))
    Y2.backward(g)
    assert torch.equal(Y, Y2)
    for a, b in ((X, X2), (w, w2), (bias, b2)):
        assert torch.isfinite(a.grad).all() and torch.equal(a.grad, b.grad)
    assert float(X.grad[:161].abs().max()) > 0 and float(w.grad.abs().max()) > 0


def test_training_and_serving_forms_agree():
    """The same layer over a cache: equal but for the int8 of the cached keys and values (2^-8 of a page's largest,
    twice, through a softmax; the layer's outlier columns are decided over the same rows)."""
    print("[case] both forms", flush=True)
    cache = m8.KVCache.empty(20, 2, 64, 16)
    axis = m8.rope_axes([16, 16])
    net = layer(cache, norm=m8.LayerNorm(), axis=axis)
    lens = [60, 33]
    X = randn(30, 93, 256)
    pos = torch.stack([torch.cat([torch.arange(n) for n in lens]), torch.arange(93) % 7], 1).int().cuda()
    with torch.no_grad():
        want = net.packed(X, m8.PackedRows.of(lens), pos)
        seqs = m8.PagedSequences(cache)
        got = net(X, seqs.extend([seqs.add(), seqs.add()], lens), pos)
    off = float((got.float() - want.float()).norm() / want.float().norm())
    assert off < 2.0 ** -5, off  # each of k and v is off by 1/254 of a page's largest, about four of its root mean square
    with pytest.raises(ValueError, match="pos"):
        net.packed(X, m8.PackedRows.of(lens))
    with pytest.raises(ValueError, match="cache"):
        layer()(X, None)


def test_a_training_step_of_all_of_them():
    """An adapter beside the frozen layer and its norm: gradients against the formula's in 64 bits where the layer is
    linear enough to have one (a threshold that sends every column through the 16-bit product), then clipped."""
    print("[case] step", flush=True)
    T, hidden, r = 100, 256, 8
    rows = m8.PackedRows.of([64, 36])
    w, bias = leaf(torch.ones(hidden, device="cuda")), leaf(torch.zeros(hidden, device="cuda"))
    net = layer(norm=m8.LayerNorm(w, bias), threshold=2.0 ** -14)
    A, B = leaf(randn(40, r, hidden, dtype=torch.float32, scale=0.05)), leaf(randn(41, hidden, r, dtype=torch.float32, scale=0.05))
    X, g = randn(42, T, hidden), randn(43, T, hidden, scale=8.0)
    Y = net.packed(X + ((X.float() @ A.t()) @ B.t()).half(), rows)
    Y.backward(g)
    grads = [p.grad.clone() for p in (A, B, w, bias)]
    norm = m8.clip_grad_norm([A, B, w, bias, torch.zeros(1)], 0.5)
    assert abs(float(norm) / ref.grad_norm([x.cpu().numpy() for x in grads]) - 1) < 2.0 ** -22
    for p, x in zip((A, B, w, bias), grads):
        assert torch.equal(p.grad.cpu(), x.cpu() * float(ref.grad_factor(norm.item(), 0.5)))
    # 64 bits, by torch's graph
    D = torch.float64
    WQ, WO = ((lin.Wq.double() * lin.sW.double()[:, None] / 127).cpu() for lin in (net.qkv, net.out))
    a, bb, ww, bi = (x.detach().cpu().to(D).requires_grad_() for x in (A, B, w, bias))
    x = X.cpu().to(D)
    h = torch.nn.functional.layer_norm(x + (x @ a.t()) @ bb.t(), (hidden,), ww, bi, 1e-5)
    qkv = (h @ WQ.t()).view(T, 8, 64)
    ang = torch.cat([torch.arange(64), torch.arange(36)]).to(D)[:, None] * torch.tensor(m8.rope_frequencies(64)[0], dtype=D)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    turned = torch.cat([qkv[:, :6, :32] * c - qkv[:, :6, 32:] * s, qkv[:, :6, 32:] * c + qkv[:, :6, :32] * s], -1)
    outs, at = [], 0
    for n in (64, 36):
        q, k, v = turned[at:at + n, :4], turned[at:at + n, 4:], qkv[at:at + n, 6:]
        k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
        sc = torch.einsum("ihc,jhc->hij", q, k) / 8
        sc = sc.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -np.inf)
        outs.append(torch.einsum("hij,jhc->ihc", sc.softmax(-1), v))
        at += n
    y = torch.cat(outs).reshape(T, -1) @ WO.t()
    y.backward(g.cpu().to(D))
    # about a dozen roundings to fp16 (2^-11 of a value, in the worst case all of one sign) lie between
    for got, want in zip(grads, (a, bb, ww, bi)):
        off = float((got.cpu().double() - want.grad).norm() / want.grad.norm())
        print(f"  gradient off by {off:.2e}", flush=True)
        assert off < 16 * 2.0 ** -11
    assert float((Y.detach().cpu().double() - y.detach()).norm() / y.detach().norm()) < 12 * 2.0 ** -11


def test_many_batches_give_every_row_once():
    """Work is dealt by the sequences' lengths: batches of 1 to 150 sequences, each row the same as alone."""
    print("[case] batches", flush=True)
    rng = np.random.default_rng(50)
    for seqs, top in ((1, 700), (2, 400), (63, 60), (64, 70), (65, 70), (150, 30), (30, 300)):
        lens = [int(n) for n in rng.integers(0, top, seqs)]
        T = sum(lens)
        q, k, v, do = (randn(seqs + i, T, h, 32, dtype=torch.bfloat16) for i, h in enumerate((6, 2, 2, 6)))
        b = m8.PackedRows.of(lens)
        out, lse = m8.llmint8_attention(b, q, k, v, window=100)
        grads = m8.llmint8_attention_backward(b, q, k, v, out, lse, do, window=100)
        at = np.concatenate([[0], np.cumsum(lens)])
        for i in rng.choice(seqs, min(seqs, 5), replace=False):
            r = slice(int(at[i]), int(at[i + 1]))
            if lens[i] == 0:
                continue
            one = m8.PackedRows.of([lens[i]])
            o1, l1 = m8.llmint8_attention(one, q[r], k[r], v[r], window=100)
            g1 = m8.llmint8_attention_backward(one, q[r], k[r], v[r], o1, l1, do[r], window=100)
            for x, y in zip((out, lse, *grads), (o1, l1, *g1)):
                assert torch.equal(x[r], y), (seqs, i)


def test_everything_in_a_captured_step():
    """Forward, backward, norm and clipping replay from one graph, on new values."""
    print("[case] captured step", flush=True)
    T = 96
    rows = m8.PackedRows(torch.tensor([0, 40, 96], dtype=torch.int32, device="cuda"), T, used=T)
    q, k, v, do = (randn(60 + i, T, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    x, w = randn(70, T, 256), torch.ones(256, device="cuda")
    table = m8.llmint8_rope_table(m8.rope_frequencies(64)[0], 100)
    axis = bytes(32)
    gs = [torch.zeros_like(t) for t in (q, k, v)]
    gset = m8.GradientSet(gs)

    def step():
        y, stats = m8.llmint8_layer_norm(x, w)
        dx, dw, db = m8.llmint8_layer_norm_backward(y, x, stats, w)
        pos = rows.positions()
        rq, rk = m8.llmint8_rope(table, pos, axis, q, k)
        out, lse = m8.llmint8_attention(rows, rq, rk, v)
        m8.llmint8_attention_backward(rows, rq, rk, v, out, lse, do, dq=gs[0], dk=gs[1], dv=gs[2])
        norm = m8.llmint8_grad_norm(gset)
        m8.llmint8_grad_clip(gset, norm, 0.1)
        return y, dx, dw, db, out, norm

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = step()
    for i in range(3):
        q.copy_(randn(80 + i, *q.shape))
        x.copy_(randn(90 + i, *x.shape))
        rows.cu.copy_(torch.tensor([0, 10 + 30 * i, 96], dtype=torch.int32))
        want = [t.clone() for t in (*step(), *gs)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*held, *gs), want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("count", [1, 119, 120, 121, 480, 481, 1000])
def test_batches_of_gradients(count):
    """Tensors go to a launch in batches; each is counted and scaled once, eagerly and in a replayed graph."""
    print(f"[case] {count} gradients", flush=True)
    grads = [randn(i, 1 + i * 37 % 300) if i % 5 else torch.zeros(0, dtype=torch.float16, device="cuda") for i in range(1, count + 1)]
    wide = [torch.zeros_like(g, dtype=torch.float32) for g in grads]
    gset = m8.GradientSet(grads, out=wide)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        m8.llmint8_grad_clip(gset, m8.llmint8_grad_norm(gset), 0.5)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            norm = m8.llmint8_grad_norm(gset)
            m8.llmint8_grad_clip(gset, norm, 0.5)
    for k in range(3):
        for g in grads:
            g.mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.grad_norm([g.cpu().numpy() for g in grads])
        assert abs(float(norm) - want) <= 2.0 ** -23 * want, k
        f = np.float32(ref.grad_factor(norm.item(), 0.5))
        assert np.array_equal(torch.cat(wide).cpu().numpy(), torch.cat(grads).cpu().numpy().astype(np.float32) * f), k


def test_the_example_runs_and_every_parameter_has_a_gradient():
    print("[case] example", flush=True)
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_training.py")
    spec = importlib.util.spec_from_file_location("adapter_training", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    blocks, losses, norms = example.main(["--layers", "2", "--steps", "3", "--tokens", "300"])
    assert all(torch.isfinite(x).all() for x in (*losses, *norms)) and all(float(x) > 0 for x in norms)
    for name, p in blocks.named_parameters():  # B of an adapter was zero in the first step, so A's is of later ones
        assert p.grad is not None and torch.isfinite(p.grad).all() and float(p.grad.abs().max()) > 0, name
    total = ref.grad_norm([p.grad.cpu().numpy() for p in blocks.parameters()])
    assert total <= 0.1 * (1 + 2.0 ** -20)  # clipped
