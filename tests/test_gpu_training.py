"""Packed attention, rotary positions with axes, layer norm and gradient clipping on the GPU against the oracle.

Attention's bound is the oracle's, element by element: from the rounding of P and dS to the 16-bit type and of
each output, and from fp32 logits and sums (oracle/training_oracle.py). Rotations are bit for bit. Layer norm: see
``norm_bounds``. The norm of gradients is within 2^-23 of itself (one rounding to fp32; 64-bit sums), clipped
values are bit for bit those of the factor from that norm.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import training_oracle as ref

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


def _say(msg):
    print(f"[case] {msg}", flush=True)


def host(t):
    return t.detach().float().cpu().numpy()


def values(rng, shape, dtype, scale=1.0, wide=False):
    """A device tensor [rows, heads, dim]; ``wide``: a slice of a larger one that holds NaN around it."""
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    x[..., rng.integers(0, shape[-1])] *= 4.0
    t = torch.from_numpy(x).cuda().to(TD[dtype])
    if wide:
        big = torch.full((shape[0], shape[1] + 3, shape[2]), float("nan"), dtype=TD[dtype], device="cuda")
        big[:, 1:1 + shape[1]] = t
        t = big[:, 1:1 + shape[1]]
    return t


def below(name, got, want, bound):
    off = np.abs(host(got).astype(np.float64) - want)
    assert np.isfinite(off).all(), name
    worst = float((off / np.maximum(bound, 1e-300)).max(initial=0.0))
    print(f"  {name}: {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, (name, worst)


def tiny(dtype):
    """Half a step of the type's smallest values."""
    return 2.0 ** -25 if dtype == "f16" else 0.0


def check_attention(lens, tensors, dtype, how, outs):
    q, k, v, do = tensors
    scale = how.get("scale")
    scale = 1 / np.sqrt(q.shape[2]) if scale is None else scale
    T = sum(lens)
    want = ref.attention(lens, *(host(t[:T]) for t in (q, k, v)), np.float32(scale), how.get("causal", True),
                         how.get("window", 0), how.get("sinks", 0), host(do[:T]), U[dtype], dtype == "f16")
    for name, t in outs.items():
        below(name, t[:T], want[name], want["e_" + name] + (tiny(dtype) if name != "lse" else 0))


ATTENTION = [
    # lens, q_heads, heads, dim, dtype, options
    ([1], 1, 1, 8, "f16", {}),
    ([5, 0, 1, 64, 65, 0], 2, 1, 16, "bf16", {}),
    ([130, 63, 200], 8, 2, 64, "f16", {}),
    ([257, 1, 300], 3, 3, 80, "bf16", {}),
    ([129, 128, 127], 5, 1, 128, "f16", {}),
    ([700], 4, 2, 128, "bf16", {"window": 100, "sinks": 4}),
    ([400, 33], 2, 2, 256, "f16", {}),
    ([150, 90], 4, 2, 200, "bf16", {"causal": False}),
    ([300, 64], 6, 2, 72, "f16", {"causal": False}),
    ([90, 333], 7, 1, 96, "bf16", {"window": 1}),
    ([1000, 200], 4, 1, 40, "f16", {"window": 64, "sinks": 70}),
    ([190, 320], 2, 1, 128, "f16", {"window": 130, "sinks": 129}),
    ([500], 33, 1, 24, "bf16", {"window": 400}),
    ([100, 257], 4, 4, 64, "bf16", {"scale": -0.3}),
    ([70, 140], 2, 1, 64, "f16", {"scale": 0.0}),
    ([2, 3, 0, 1] * 130, 2, 1, 64, "bf16", {}),
]


@pytest.mark.parametrize("case", range(len(ATTENTION)))
@pytest.mark.parametrize("wide", [False, True])
def test_attention_and_its_gradients(case, wide):
    lens, hq, hk, dim, dtype, how = ATTENTION[case]
    _say(f"attention {ATTENTION[case]} wide={wide}")
    rng = np.random.default_rng(case)
    T = sum(lens)
    q, do = values(rng, (T, hq, dim), dtype, wide=wide), values(rng, (T, hq, dim), dtype, 0.5, wide=wide)
    k, v = values(rng, (T, hk, dim), dtype, wide=wide), values(rng, (T, hk, dim), dtype, wide=wide)
    b = m8.PackedRows.of(lens)
    out, lse = m8.llmint8_attention(b, q, k, v, **how)
    dq, dk, dv = m8.llmint8_attention_backward(b, q, k, v, out, lse, do, **how)
    torch.cuda.synchronize()
    check_attention(lens, (q, k, v, do), dtype, how, {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv})


@pytest.mark.parametrize("dtype,grad", [("f16", 2.0 ** -16), ("f16", 400.0), ("bf16", 2.0 ** -60), ("bf16", 2.0 ** 40)])
def test_gradients_of_any_size(dtype, grad):
    """Loss-scaled gradients, and ones far below the type's usual range: dS keeps its bits, and rows differ."""
    _say(f"gradients of {grad} in {dtype}")
    rng = np.random.default_rng(5)
    lens, hq, hk, dim = [300, 77], 4, 2, 64
    T = sum(lens)
    q, k, v = (values(rng, (T, h, dim), dtype) for h in (hq, hk, hk))
    do = values(rng, (T, hq, dim), dtype, grad)
    do[::7] *= 2.0 ** -6
    do[150:153] = 0
    b = m8.PackedRows.of(lens)
    out, lse = m8.llmint8_attention(b, q, k, v)
    dq, dk, dv = m8.llmint8_attention_backward(b, q, k, v, out, lse, do)
    check_attention(lens, (q, k, v, do), dtype, {}, {"dq": dq, "dk": dk, "dv": dv})


def test_sharp_and_flat_softmax():
    """Logits of hundreds: one token takes everything, the others' weights vanish; and a running maximum that keeps
    rising from tile to tile."""
    _say("sharp softmax")
    rng = np.random.default_rng(6)
    for dtype in ("f16", "bf16"):
        lens, dim = [400], 64
        q, k, v, do = (values(rng, (400, 2, dim), dtype) for _ in range(4))
        k *= torch.linspace(0.1, 20.0, 400, device="cuda").to(k.dtype)[:, None, None]
        b = m8.PackedRows.of(lens)
        out, lse = m8.llmint8_attention(b, q, k, v)
        grads = m8.llmint8_attention_backward(b, q, k, v, out, lse, do)
        check_attention(lens, (q, k, v, do), dtype, {}, dict(zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads))))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("how", [{}, {"window": 40, "sinks": 3}])
def test_what_is_not_finite_reaches_only_what_sees_it(value, dtype, how):
    _say(f"{value} in {dtype} {how}")
    rng = np.random.default_rng(7)
    lens, hq, hk, dim = [100, 150, 30], 2, 1, 64
    T = sum(lens)
    clean = [values(rng, (T, h, dim), dtype) for h in (hq, hk, hk, hq)]
    b = m8.PackedRows.of(lens)

    def run(q, k, v, do):
        out, lse = m8.llmint8_attention(b, q, k, v, **how)
        return (out, lse, *m8.llmint8_attention_backward(b, q, k, v, out, lse, do, **how))

    want = run(*clean)
    at = 100 + 70  # a token in the middle of the second sequence
    see = ref.visible(150, True, how.get("window", 0), how.get("sinks", 0))
    rows = {100 + int(i) for i in np.flatnonzero(see[:, 70])}        # the rows that see it
    seen_by = {100 + int(j) for i in rows for j in np.flatnonzero(see[i - 100])}
    own = {100 + int(j) for j in np.flatnonzero(see[70])}            # the tokens that its row sees
    for which, name in enumerate(("q", "k", "v", "do")):
        t = [x.clone() for x in clean]
        t[which][at, 0, 5] = value
        got = run(*t)
        row_set = {"q": {at}, "do": set()}.get(name, rows)
        # outputs of rows: those that see the token; gradients of tokens: those that an affected row sees
        for i, (x, y) in enumerate(zip(got, want)):
            part = ("out", "lse", "dq", "dk", "dv")[i]
            if part in ("out", "lse"):
                may = row_set if not (part == "lse" and name in ("v", "do")) else set()
            elif part == "dq":
                may = {"q": {at}, "do": {at}}.get(name, rows)
            else:
                may = own if name in ("q", "do") else seen_by
            same = torch.tensor([r not in may for r in range(T)], device="cuda")
            assert torch.equal(x[same], y[same]), (name, part)
        if name in ("k", "v"):
            odd = torch.tensor(sorted(rows), device="cuda")
            assert not torch.isfinite(got[0][odd, 0].float()).all(-1).any() or name == "k" and value != value * 0 + value
        if name == "v":  # the infinity itself, where its weight is not zero
            x = got[0][odd, 0, 5].float()
            assert (torch.isnan(x) if value != value else (x == value) | torch.isnan(x)).all()


def test_other_sequences_and_unused_rows():
    """Rows of no sequence hold NaN and are left alone; so are outputs there."""
    _say("unused rows")
    rng = np.random.default_rng(8)
    lens, hq, hk, dim, T = [70, 3, 129], 4, 2, 64, 260
    used = sum(lens)
    t = [values(rng, (T, h, dim), "bf16") for h in (hq, hk, hk, hq)]
    for x in t:
        x[used:] = float("nan")
    b = m8.PackedRows.of(lens, rows=T)
    outs = [torch.full((T, h, dim), 7.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hq, hk, hk)]
    lse = torch.full((T, hq), 7.0, device="cuda")
    m8.llmint8_attention(b, *t[:3], out=outs[0], lse=lse)
    m8.llmint8_attention_backward(b, *t[:3], outs[0], lse, t[3], dq=outs[1], dk=outs[2], dv=outs[3])
    torch.cuda.synchronize()
    for x in (*outs, lse):
        assert (x[used:] == 7.0).all()
    check_attention(lens, t, "bf16", {}, dict(zip(("out", "dq", "dk", "dv", "lse"), (*outs, lse))))


@pytest.mark.parametrize("cu", [[0, 500, 100, 400], [-5, 90, 2 ** 30, -2 ** 31], [100, 100, 50, 300], [0, 0, 0, 0],
                                [300, 300, 300, 2 ** 31 - 1]])
def test_hostile_starts_stay_inside(cu):
    """Whatever cu holds, nothing outside the tensors is written (guard rows on both sides)."""
    _say(f"cu {cu}")
    rng = np.random.default_rng(9)
    T, hq, hk, dim = 300, 4, 2, 64
    t = [values(rng, (T, h, dim), "f16") for h in (hq, hk, hk, hq)]
    big = [torch.full((T + 200, h, dim), 5.0, dtype=torch.float16, device="cuda") for h in (hq, hq, hk, hk)]
    outs = [x[100:100 + T] for x in big]
    lse = torch.full((T + 200, hq), 5.0, device="cuda")
    b = m8.PackedRows(torch.tensor(cu, dtype=torch.int32, device="cuda"), T)
    m8.llmint8_attention(b, *t[:3], out=outs[0], lse=lse[100:100 + T])
    m8.llmint8_attention_backward(b, *t[:3], outs[0], lse[100:100 + T], t[3], dq=outs[1], dk=outs[2], dv=outs[3])
    torch.cuda.synchronize()
    for x in (*big, lse):
        assert (x[:100] == 5.0).all() and (x[100 + T:] == 5.0).all()


def test_attention_repeats_itself_and_replays():
    """The same bits every time; a captured graph follows cu and the inputs."""
    _say("graph")
    rng = np.random.default_rng(10)
    T, hq, hk, dim = 500, 8, 2, 128
    t = [values(rng, (T, h, dim), "bf16") for h in (hq, hk, hk, hq)]
    b = m8.PackedRows(torch.tensor([0, 200, 500], dtype=torch.int32, device="cuda"), T)

    def run():
        out, lse = m8.llmint8_attention(b, *t[:3])
        return (out, lse, *m8.llmint8_attention_backward(b, *t[:3], out, lse, t[3]))

    first = run()
    for x, y in zip(first, run()):
        assert torch.equal(x, y)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            held = run()
    for cu in ([0, 200, 500], [0, 499, 500], [0, 0, 500], [0, 200, 500]):
        b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y), cu


def test_attention_on_another_stream():
    _say("stream")
    rng = np.random.default_rng(11)
    t = [values(rng, (300, h, 64), "f16") for h in (4, 4, 4, 4)]
    b = m8.PackedRows.of([300])
    want, lse = m8.llmint8_attention(b, *t[:3])
    grads = m8.llmint8_attention_backward(b, *t[:3], want, lse, t[3])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, l2 = m8.llmint8_attention(b, *t[:3], stream=s)
    again = m8.llmint8_attention_backward(b, *t[:3], out, l2, t[3], stream=s)
    s.synchronize()
    for x, y in zip((want, lse, *grads), (out, l2, *again)):
        assert torch.equal(x, y)


def test_attention_with_rows_far_apart():
    """Offsets past 2^32 bytes: few tokens at large strides."""
    _say("far rows")
    rng = np.random.default_rng(12)
    T, dim, stride = 300, 64, 1 << 23
    big = torch.empty((T * stride,), dtype=torch.float16, device="cuda")
    t = []
    for i, h in enumerate((2, 1, 1, 2)):
        x = torch.as_strided(big, (T, h, dim), (stride, dim, 1), i * 4096)
        x.copy_(values(rng, (T, h, dim), "f16"))
        t.append(x)
    outs = [torch.as_strided(big, (T, h, dim), (stride, dim, 1), 65536 + i * 4096) for i, h in enumerate((2, 2, 1, 1))]
    b = m8.PackedRows.of([300])
    _, lse = m8.llmint8_attention(b, *t[:3], out=outs[0])
    m8.llmint8_attention_backward(b, *t[:3], outs[0], lse, t[3], dq=outs[1], dk=outs[2], dv=outs[3])
    check_attention([300], t, "f16", {}, dict(zip(("out", "dq", "dk", "dv"), outs)))


# ---- rotary positions


ROPE = [
    # rows, heads, k_heads, dim, rot, sections, turns, interleaved, dtype
    (1, 1, 0, 2, 2, (1,), False, False, "f16"),
    (7, 3, 1, 72, 72, (12, 12, 12), False, False, "bf16"),
    (33, 8, 2, 128, 128, (16, 24, 24), False, False, "bf16"),
    (33, 8, 2, 128, 128, (24, 20, 20), True, True, "f16"),
    (50, 5, 5, 80, 40, (7, 13), True, False, "f16"),
    (41, 2, 1, 64, 24, (5, 0, 7), False, True, "bf16"),
    (2500, 40, 8, 64, 64, (8, 8, 8, 8), False, False, "bf16"),
    (9, 2, 2, 46, 22, (11,), False, False, "f16"),
    (9, 2, 2, 46, 22, (4, 7), True, True, "f16"),
    (5, 2, 0, 500, 256, (64, 64), False, False, "bf16"),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_bit_for_bit(case, inverse):
    rows, heads, k_heads, dim, rot, sections, turns, interleaved, dtype = ROPE[case]
    _say(f"rope {ROPE[case]} inverse={inverse}")
    rng = np.random.default_rng(case)
    axis = m8.rope_axes(sections, turns)
    if 2 * len(axis) != rot:
        axis = (axis * rot)[:rot // 2]
    freq, _ = m8.rope_frequencies(rot)
    table = m8.llmint8_rope_table(freq, 300)
    pos = rng.integers(-3, 310, (rows, len(sections))).astype(np.int32)  # some outside the table
    posd = torch.from_numpy(pos).cuda()
    q = values(rng, (rows, heads, dim), dtype, wide=case % 2 == 1)
    k = values(rng, (rows, k_heads, dim), dtype) if k_heads else None
    out = m8.llmint8_rope(table, posd, axis, q, k, interleaved, inverse)
    for x, y in zip((q, k), out):
        if x is None:
            assert y is None
            continue
        want = torch.from_numpy(ref.rope(host(x), host(table), pos, axis, interleaved, inverse)).to(TD[dtype])
        assert torch.equal(y.cpu(), want)
    if k is not None:  # in place
        again = m8.llmint8_rope(table, posd, axis, q, k, interleaved, inverse, q_out=q, k_out=k)
        assert again[0] is q and torch.equal(q, out[0]) and torch.equal(k, out[1])


def test_rope_of_one_axis_is_the_cache_s():
    """The keys' and queries' rotation of llmint8_kv_append, on the same table."""
    _say("rope as the cache's")
    rng = np.random.default_rng(3)
    n, hq, hk, dim = 70, 4, 2, 64
    cache = m8.KVCache.empty(4, hk, dim, 64)
    seqs = m8.PagedSequences(cache)
    batch = seqs.extend([seqs.add()], [n])
    table = m8.llmint8_rope_table(m8.rope_frequencies(dim)[0], 100)
    k, v, q = (values(rng, (n, h, dim), "bf16") for h in (hk, hk, hq))
    want = m8.llmint8_kv_append(cache, batch, k, v, q, rope=table)
    got, _ = m8.llmint8_rope(table, torch.arange(n, dtype=torch.int32, device="cuda"), [0] * 32, q)
    assert torch.equal(want, got)


# ---- layer norm


NORM = [
    # rows, K, dtype, weight type, row pitch beyond K
    (1, 1, "f16", None, 0), (3, 7, "bf16", "bf16", 0), (5, 8, "f32", "f32", 3), (70, 100, "f16", "f32", 1),
    (33, 1001, "f16", "f16", 0), (600, 1024, "bf16", "f32", 8), (700, 1030, "bf16", "bf16", 0), (9, 2049, "f32", "f32", 0),
    (300, 4096, "f16", "f32", 0), (1100, 4096, "bf16", "f32", 0), (5, 8191, "bf16", "f32", 0), (40, 8200, "f16", "f16", 2),
    (7, 16384, "bf16", "f32", 0), (3, 16385, "f32", "f32", 0), (300, 20000, "bf16", "bf16", 0), (2, 65536, "f16", "f32", 0),
    (260, 64, "f32", None, 0),
]


def norm_bounds(r, x, w, b, dy, eps, u, uw):
    """How far results may be off. Statistics: sums of K values in fp32, in a tree of at most 32 values to a lane and
    11 levels, so (K's share aside) about 48 roundings: c = 64 of 2^-24. With them
      xh: c (1 + |xh| + |mean| rstd), as x - mean is rounded against values of the mean's size
      y = xh w + b: that times |w|, and three roundings;  dx: the same through its three terms."""
    f, c = 2.0 ** -24, 64 * 2.0 ** -24
    K = x.shape[1]
    w = np.ones(K) if w is None else np.abs(w)
    b = np.zeros(K) if b is None else np.abs(b)
    xh, rstd = np.abs(r["xh"]), r["rstd"][:, None]
    size = np.abs(x).mean(1, keepdims=True) * rstd  # of what the mean sums
    e_x = c * (1 + xh + 2 * size) + c * xh * (1 + size)
    e = {"y": u * np.abs(r["y"]) + e_x * w + 3 * f * (xh * w + b)}
    if dy is not None:
        g, n = np.abs(dy) * w, x.shape[0]
        m1, m2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
        e_m2 = c * m2 + (g * e_x).mean(1, keepdims=True)
        e["dx"] = u * np.abs(r["dx"]) + rstd * (c * (g + m1 + xh * m2) * (1 + size) + e_x * m2 + xh * e_m2)
        a = (n + 64) * f  # a column's sum: at most as many additions as rows
        e["dw"] = uw * np.abs(r["dw"]) + (np.abs(dy) * (e_x + a * xh)).sum(0)
        e["db"] = uw * np.abs(r["db"]) + a * np.abs(dy).sum(0)
    return e


@pytest.mark.parametrize("case", range(len(NORM)))
def test_layer_norm_and_its_gradients(case):
    rows, K, dtype, wt, pitch = NORM[case]
    _say(f"norm {NORM[case]}")
    rng = np.random.default_rng(case)
    eps = 1e-5

    def rows_of(scale, shift):
        x = rng.standard_normal((rows, K)) * scale * np.exp(rng.standard_normal((rows, 1))) + shift
        t = torch.full((rows, K + pitch), float("nan"), dtype=TD[dtype], device="cuda")
        t[:, :K] = torch.from_numpy(x.astype(np.float32)).cuda().to(TD[dtype])
        return t[:, :K]

    x, dy = rows_of(1.0, 0.5), rows_of(0.1, 0.0)
    w = b = None
    if wt:
        w = torch.from_numpy((1 + 0.3 * rng.standard_normal(K)).astype(np.float32)).cuda().to(TD[wt])
        b = torch.from_numpy((0.2 * rng.standard_normal(K)).astype(np.float32)).cuda().to(TD[wt])
    wh, bh = (None if t is None else host(t).astype(np.float64) for t in (w, b))
    r = ref.layer_norm(host(x), wh, bh, eps, host(dy))
    e = norm_bounds(r, host(x).astype(np.float64), wh, bh, host(dy).astype(np.float64), eps, U[dtype], U[wt or dtype])
    y, stats = m8.llmint8_layer_norm(x, w, b, eps)
    dx, dw, db = m8.llmint8_layer_norm_backward(dy, x, stats, w)
    torch.cuda.synchronize()
    below("y", y, r["y"], e["y"] + tiny(dtype))
    below("dx", dx, r["dx"], e["dx"] + tiny(dtype))
    if wt:
        below("dw", dw, r["dw"], e["dw"] + tiny(wt))
        below("db", db, r["db"], e["db"] + tiny(wt))
        # the same without the sums, and bit for bit again
        alone = m8.llmint8_layer_norm_backward(dy, x, stats, w, sums=False)
        assert alone[1] is None and torch.equal(alone[0], dx)
        again = m8.llmint8_layer_norm_backward(dy, x, stats, w)
        assert all(torch.equal(s, t) for s, t in zip(again, (dx, dw, db)))
    else:
        assert dw is None and db is None
    alone, none = m8.llmint8_layer_norm(x, w, b, eps, stats=False)
    assert none is None and torch.equal(alone, y)


def test_layer_norm_of_rows_that_do_not_vary_and_of_none():
    _say("flat rows")
    x = torch.full((4, 300), 3.0, dtype=torch.float16, device="cuda")
    w = torch.ones(300, dtype=torch.float16, device="cuda")
    y, stats = m8.llmint8_layer_norm(x, w, eps=1e-5)
    assert (y == 0).all() and (stats[:, 0] == 3.0).all()
    x[1, 7] = float("nan")
    y, stats = m8.llmint8_layer_norm(x, w)
    assert torch.isnan(y[1]).all() and (y[[0, 2, 3]] == 0).all()
    none = torch.empty((0, 300), dtype=torch.float16, device="cuda")
    y, stats = m8.llmint8_layer_norm(none, w)
    dx, dw, db = m8.llmint8_layer_norm_backward(none, none, stats, w)
    assert y.shape == dx.shape == (0, 300) and (dw == 0).all() and (db == 0).all()


# ---- the gradients' norm


def grads_of(rng, sizes, dtypes):
    out = []
    for i, n in enumerate(sizes):
        big = torch.from_numpy((rng.standard_normal(n + 1) * 10.0 ** rng.integers(-3, 2)).astype(np.float32)).cuda()
        out.append(big.to(TD[dtypes[i % len(dtypes)]])[i % 2:][:n])  # every other one starts at an odd value
    return out


@pytest.mark.parametrize("sizes,dtypes", [
    ([1], ["f16"]), ([0, 5, 0], ["f32"]), ([16384, 16385, 8191, 3], ["bf16", "f32", "f16"]),
    (list(range(1, 300)), ["f16", "bf16", "f32"]), ([3_000_001, 7], ["bf16"]), ([], ["f32"]),
])
@pytest.mark.parametrize("scale,max_norm", [(1.0, 1.0), (1 / 64, 1e9), (0.37, float("inf"))])
def test_gradients_are_clipped(sizes, dtypes, scale, max_norm):
    _say(f"clip {len(sizes)} {dtypes} {scale} {max_norm}")
    rng = np.random.default_rng(len(sizes))
    grads = grads_of(rng, sizes, dtypes)
    want = ref.grad_norm([host(g) for g in grads], scale)
    norm = m8.llmint8_grad_norm(grads, scale, device="cuda")
    got = float(norm)
    assert abs(got - want) <= 2.0 ** -23 * want, (got, want)
    f = ref.grad_factor(norm.item(), max_norm, scale)
    wide = [torch.zeros_like(g, dtype=torch.float32) for g in grads]
    m8.llmint8_grad_clip(m8.GradientSet(grads, out=wide), norm, max_norm, scale)
    for g, o in zip(grads, wide):
        assert np.array_equal(o.cpu().numpy(), host(g) * f)
    expect = [torch.from_numpy(host(g) * f).to(g.dtype) for g in grads]
    done = m8.llmint8_grad_clip(grads, norm, max_norm, scale)
    for g, e in zip(done, expect):
        assert torch.equal(g.cpu(), e)


def test_large_and_odd_gradients():
    _say("odd gradients")
    big = torch.full((20000,), 3e30, device="cuda")  # squares leave fp32
    assert abs(float(m8.llmint8_grad_norm([big])) / (3e30 * 20000 ** 0.5) - 1) < 2.0 ** -22
    small = torch.full((1000,), 1e-30, device="cuda")
    assert abs(float(m8.llmint8_grad_norm([small])) / (1e-30 * 1000 ** 0.5) - 1) < 2.0 ** -22
    bad = [torch.ones(10, device="cuda"), torch.tensor([1.0, float("nan")], device="cuda")]
    norm = m8.llmint8_grad_norm(bad)
    assert torch.isnan(norm)
    m8.llmint8_grad_clip(bad, norm, 1.0)
    assert all(torch.isnan(g).all() for g in bad)
    t = torch.arange(24.0, device="cuda").view(4, 6).t()  # dense in another order
    norm = m8.llmint8_grad_norm([t, None])
    m8.llmint8_grad_clip([t], norm, 1.0)
    assert torch.allclose(t, torch.arange(24.0, device="cuda").view(4, 6).t() / norm)
