"""Calls of the training operators whose memory or metadata changes between them, inputs at odd places, and what is not
finite where the formula gives it no weight."""
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


def at_odd_place(t, first):
    flat = torch.empty(first + t.numel(), dtype=t.dtype, device=t.device)
    flat[first:] = t.flatten()
    return flat[first:].view(t.shape)


@pytest.mark.parametrize("first", [1, 3, 4])
def test_attention_takes_tensors_that_begin_at_an_odd_place(first):
    print(f"[case] odd place {first}", flush=True)
    b = m8.PackedRows.of([50, 70])
    q, k, v, g = (randn(i, 120, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    want = [leaf(t) for t in (q, k, v)]
    m8.packed_attention(*want, b).backward(g)
    odd = [at_odd_place(t, first).requires_grad_() for t in (q, k, v)]
    aux = torch.zeros(first, dtype=torch.float16, device="cuda")
    # the concatenation's gradient for the output is contiguous and begins at an odd place
    z = torch.cat([aux, m8.packed_attention(*odd, b).flatten()])
    z.backward(torch.cat([aux, g.flatten()]))
    for a, t in zip(odd, want):
        assert torch.equal(a.grad, t.grad)
    qkv = torch.cat([q, k, v], 1)
    x, y = leaf(qkv), at_odd_place(qkv, first).requires_grad_()
    m8.qkv_attention(x, 2, b).backward(g)
    torch.cat([aux, m8.qkv_attention(y, 2, b).flatten()]).backward(torch.cat([aux, g.flatten()]))
    assert torch.equal(x.grad, y.grad)


def layer(hidden=256, nq=4, heads=2, dim=64, **kw):
    rope = m8.llmint8_rope_table(m8.rope_frequencies(dim)[0], 400)
    return m8.Int8SelfAttention(randn(5, (nq + 2 * heads) * dim, hidden, scale=0.05),
                                randn(6, hidden, nq * dim, scale=0.05), nq, None, rope, heads=heads, dim=dim, **kw)


def poison():
    """Leaves NaN in the memory that the next tensors get."""
    held = [torch.full((n,), float("nan"), dtype=torch.float16, device="cuda") for n in (1 << k for k in range(10, 20))]
    del held


def test_rows_of_no_sequence_after_a_change_of_cu():
    """Rows that a shorter cu leaves to no sequence are zeros, in outputs and gradients; the layer's other rows do not
    see them."""
    print("[case] cu shrinks", flush=True)
    b = m8.PackedRows.of([70, 50])
    b.cu.copy_(torch.tensor([0, 40, 60], dtype=torch.int32))
    q, k, v, g = (randn(i, 120, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    now = m8.PackedRows.of([40, 20], rows=120)
    got, want = [leaf(t) for t in (q, k, v)], [leaf(t) for t in (q, k, v)]
    for ts, batch in ((got, b), (want, now)):
        poison()
        out = m8.packed_attention(*ts, batch)
        assert (out[60:] == 0).all()
        poison()
        out.backward(g)
        for t in ts:
            assert (t.grad[60:] == 0).all()
    for a, t in zip(got, want):
        assert torch.equal(a.grad, t.grad)
    w = leaf(torch.ones(256, device="cuda"))
    net = layer(norm=m8.LayerNorm(w))
    X, dy = randn(10, 120, 256), randn(11, 120, 256)
    res = []
    for batch in (b, now):
        x = leaf(X)
        w.grad = None
        poison()
        y = net.packed(x, batch)
        poison()
        y.backward(dy)
        res.append((y.detach(), x.grad, w.grad.clone()))
    for a, t in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, t)


def test_rows_of_no_sequence_in_a_replayed_call():
    """A call captured with all rows in use, replayed on shorter sequences."""
    print("[case] replay on a shorter cu", flush=True)
    b = m8.PackedRows.of([70, 50])
    q, k, v, g = (randn(i, 120, h, 64) for i, h in enumerate((4, 2, 2, 4)))

    def step():
        ts = [t.detach().requires_grad_() for t in (q, k, v)]
        out = m8.packed_attention(*ts, b)
        return (out.detach(), *torch.autograd.grad(out, ts, g))

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = step()
    for cu in ([0, 70, 120], [0, 10, 25], [0, 0, 0], [0, 70, 120]):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        for t in held:
            t.fill_(float("nan"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, t in zip(held, want):
            assert torch.equal(a, t) and (a[cu[-1]:] == 0).all(), cu


def test_a_set_follows_gradients_that_move():
    """Module.half() and the like give gradients other memory and types: the set's calls clip what is there now, and
    leave alone what was."""
    print("[case] moved gradients", flush=True)
    model = torch.nn.Sequential(*(torch.nn.Linear(33, 33) for _ in range(3))).cuda()
    params = list(model.parameters())
    for i, p in enumerate(params):
        p.grad = randn(i, *p.shape, dtype=torch.float32)
    gset = m8.GradientSet([p.grad for p in params])
    for change in (None, model.half, model.float, model.bfloat16):
        before = [p.grad.detach() for p in params]
        kept = [t.clone() for t in before]
        if change is not None:
            change()
        now = [p.grad.clone() for p in params]
        norm = m8.llmint8_grad_norm(gset)
        m8.llmint8_grad_clip(gset, norm, 0.5)
        want = ref.grad_norm([t.float().cpu().numpy() for t in now])
        assert abs(float(norm) / want - 1) <= 2.0 ** -22
        f = float(ref.grad_factor(norm.item(), 0.5))
        for p, t in zip(params, now):
            assert torch.equal(p.grad, (t.float() * f).to(t.dtype)), change
        if change is not None:
            assert all(torch.equal(a, b) for a, b in zip(before, kept)), change


def step(b, q, k, v, do, how):
    out, lse = m8.llmint8_attention(b, q, k, v, **how)
    return (out, lse, *m8.llmint8_attention_backward(b, q, k, v, out, lse, do, **how))


HOW = [{}, {"causal": False}, {"window": 40, "sinks": 3}, {"window": 200}]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("how", HOW)
def test_rows_whose_logits_are_all_minus_infinity(dtype, dim, how):
    """The softmax of such a row is not a number, nor are its output and what it gives to gradients; the others'
    are what they are without it."""
    print(f"[case] no logit {dtype} {dim} {how}", flush=True)
    lens, hq, hk = [70, 1, 330, 2], 4, 2
    T = sum(lens)
    q, k, v, do = (randn(i, T, h, dim, dtype=dtype) for i, h in enumerate((hq, hk, hk, hq)))
    b = m8.PackedRows.of(lens)
    want = step(b, q, k, v, do, how)
    q[70], k[70, 0, 3] = q[70].abs() + 0.5, float("-inf")              # a sequence of one token
    q[401:, :2], k[401:, 0, 7] = q[401:, :2].abs() + 0.5, float("-inf")  # both tokens of one
    out, lse, dq, dk, dv = step(b, q, k, v, do, how)
    rows = [70, 401, 402]
    for x, y, heads in ((out, want[0], 2), (dq, want[2], 2), (dk, want[3], 1), (dv, want[4], 1)):
        assert torch.isnan(x[rows, :heads]).all()
        assert torch.equal(x[:70], y[:70]) and torch.equal(x[71:401], y[71:401])
    assert (lse[rows, :2] == float("-inf")).all() and torch.equal(lse[71:401], want[1][71:401])


def minus_infinity(dtype, dim, how, lens):
    """A step where a key's logits are all -infinity, the same with logits far below all others, the rows that see the
    key, and a call of the step with another value in the infinity's place."""
    hq, hk, T = 4, 2, sum(lens)
    first, n = (0, lens[0]) if len(lens) == 1 else (lens[0], lens[1])
    at = first + 70
    q, k, v, do = (randn(i, T, h, dim, dtype=dtype) for i, h in enumerate((hq, hk, hk, hq)))
    q[:, :, CHANNEL] = q[:, :, CHANNEL].abs() + 2.0
    b = m8.PackedRows.of(lens)
    k[at, 0] = 0
    k[at, 0, CHANNEL] = -60000.0  # times 2 / 16 at least, scaled: under -3000
    want = step(b, q, k, v, do, how)
    k[at, 0] = randn(9, dim, dtype=dtype)

    def run(value):
        k[at, 0, CHANNEL] = value
        got = step(b, q, k, v, do, how)
        torch.cuda.synchronize()
        return got

    see = ref.visible(n, how.get("causal", True), how.get("window", 0), how.get("sinks", 0))
    rows = torch.tensor([first + int(i) for i in np.flatnonzero(see[:, at - first])], device="cuda")
    assert len(rows) > 30
    return run(float("-inf")), want, rows, run


CHANNEL = 5
KEYS = [pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16]), pytest.mark.parametrize("dim", [64, 80, 128, 256]),
        pytest.mark.parametrize("how", HOW), pytest.mark.parametrize("lens", [[100, 150, 30], [700]])]


def keys(test):
    for mark in KEYS:
        test = mark(test)
    return test


@keys
def test_a_key_of_minus_infinity_has_no_weight(dtype, dim, how, lens):
    """A token whose logits are -infinity has the weight 0, as one whose logits are far below all others: the same bits."""
    print(f"[case] -inf key {dtype} {dim} {how} {lens}", flush=True)
    got, want, _, _ = minus_infinity(dtype, dim, how, lens)
    for name, x, y in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        if name != "dq":
            assert torch.equal(x, y), name


@keys
def test_what_a_key_of_minus_infinity_gives_to_dq(dtype, dim, how, lens):
    """The same bits too, but in the channel of the infinity, which is 0 times it; whether a mask crosses the token's tile
    makes no difference. Of rows whose logit is infinite or NaN all is NaN, and of no others."""
    print(f"[case] -inf key, dq {dtype} {dim} {how} {lens}", flush=True)
    got, want, rows, run = minus_infinity(dtype, dim, how, lens)
    x, y = got[2].clone(), want[2].clone()
    assert torch.isnan(x[rows, :2, CHANNEL]).all()
    x[rows, :2, CHANNEL] = y[rows, :2, CHANNEL] = 0
    assert torch.equal(x, y)
    same = torch.ones(len(x), dtype=torch.bool, device="cuda")
    same[rows] = False
    for value in (float("inf"), float("nan")):
        got = run(value)
        for x, y in zip(got[:3], want[:3]):
            assert torch.isnan(x[rows, :2]).all()
            assert torch.equal(x[same], y[same]) and torch.equal(x[:, 2:], y[:, 2:])


def test_layer_norm_of_more_rows_than_a_launch_has_work_items_for():
    """64 work items to a row: 2^26 rows and a few more."""
    print("[case] many rows", flush=True)
    n = (1 << 26) + 5
    x = (torch.arange(n, device="cuda") % 2039).to(torch.float16).view(n, 1)
    bias = torch.full((1,), 3.0, dtype=torch.float16, device="cuda")
    y, stats = m8.llmint8_layer_norm(x, None, bias)
    assert (y == 3.0).all() and torch.equal(stats[:, :1], x.float())
    y, _ = m8.llmint8_layer_norm(x, None, bias, y=x, stats=False)  # in place
    assert (x == 3.0).all()
