"""Batches of the int8 key/value cache as a server forms them: calls with more rows than the sequences use,
rows that are turned where they stand, mixed calls, other streams. Setup and bounds: test_gpu_kvcache."""
from __future__ import annotations

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402
from test_gpu_kvcache import TD, Setup, _say, check_attention  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


PADDED = [
    # lens, counts, rows of the call, heads, q_heads, dim, page, rot, interleaved, dtype
    ([100], [50], 128, 2, 4, 128, 64, 128, False, "f16"),             # tokens 50..99 reach two pages
    ([77, 31, 500], [1, 1, 1], 64, 2, 8, 64, 16, 64, False, "bf16"),   # a step
    ([77, 130, 500], [17, 17, 17], 300, 4, 4, 64, 16, 16, True, "f16"),  # drafts
    ([300, 141, 90], [170, 0, 90], 512, 2, 6, 128, 32, 128, False, "bf16"),  # prompts
    ([50, 40], [20, 3], 256, 2, 2, 48, 16, 22, True, "f16"),           # partners read one by one
    ([70, 141], [30, 100], 131, 1, 2, 256, 128, 24, False, "bf16"),
]


@pytest.mark.parametrize("case", PADDED)
def test_append_turns_q_once_where_it_stands_in_a_call_with_unused_rows(case):
    lens, counts, rows, heads, q_heads, dim, page, rot, inter, dtype = case
    _say(f"padded append {case}")
    s = Setup(81, lens, counts, heads, dim, page)
    used, s.rows = s.rows, rows
    rope_np = oracle.rope_table(m8.rope_frequencies(rot)[0], max(lens) + 1)
    rope = torch.from_numpy(rope_np).cuda()
    k, kx = s.values(heads, dtype)
    v, vx = s.values(heads, dtype)
    q, qx = s.values(q_heads, dtype, wide=True)
    want = torch.from_numpy(s.ref.append(s.cu, s.lens, s.table, kx, vx, qx, rope_np, inter)).to(TD[dtype])
    want[used:] = q[used:].cpu()
    m8.llmint8_kv_append(s.cache, s.batch(), k, v, q=q, rope=rope, interleaved=inter, q_out=q)
    s.same_cache()
    assert torch.equal(q.cpu(), want)
    gk, gv = m8.llmint8_kv_gather(s.cache, s.batch(), TD[dtype], k=torch.full_like(k, 5.0), v=torch.full_like(v, 5.0))
    for b, n in enumerate(lens):
        kx, vx, _ = s.ref.tokens(s.table, b, n - counts[b], n)
        at = slice(s.cu[b], s.cu[b + 1])
        assert torch.equal(gk[at].cpu(), torch.from_numpy(kx).to(TD[dtype])), b
        assert torch.equal(gv[at].cpu(), torch.from_numpy(vx).to(TD[dtype])), b
    assert (gk[used:] == 5).all() and (gv[used:] == 5).all()


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_layer_gives_the_batch_s_rows_the_same_whatever_memory_holds(rows):
    """Unused rows of a call to Int8SelfAttention: the output projection decides its outlier columns over all
    rows, so those of the attention must not be what memory held before."""
    g = torch.Generator(device="cuda").manual_seed(7)
    hidden, q_heads, heads, dim, used = 256, 8, 2, 32, 3
    W = (torch.randn(((q_heads + 2 * heads) * dim, hidden), device="cuda", generator=g) / 16).half()
    Wo = (torch.randn((hidden, q_heads * dim), device="cuda", generator=g) / 16).half()
    X = torch.zeros((rows, hidden), device="cuda").half()
    X[:used] = torch.randn((used, hidden), device="cuda", generator=g).half()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = []
    for poison in (0.0, 100.0, -3.0):
        cache = m8.KVCache.empty(4, heads, dim, 16)
        layer = m8.Int8SelfAttention(W, Wo, q_heads, cache)
        held = [torch.full((rows, q_heads, dim), poison, device="cuda").half() for _ in range(40)]
        del held
        out.append(layer(X, m8.KVBatch(ints([0, 1, used]), ints([1, 2]), ints([[2], [0]]), rows)))
    for y in out:
        same = bool((y == out[0]).all())
        assert same and bool((y[used:] == 0).all()) and bool((y[:used] != 0).any())


def test_calls_on_another_stream_while_the_current_one_takes_memory():
    """No workspace and no outputs given: what the calls take is not the current stream's to reuse."""
    s = Setup(83, [9000, 700], [1, 3], 2, 128, 64)
    q, _ = s.values(8, "f16")
    k, _ = s.values(2, "f16")
    b = s.batch(9000)
    size = m8.llmint8_kv_attention_workspace_bytes(s.cache, b, 8)
    assert size > 0
    m8.llmint8_kv_append(s.cache, b, k, k)
    want = m8.llmint8_kv_attention(s.cache, b, q)
    W = torch.randn((256, 128), device="cuda").half()
    Wq, sW = m8.llmint8_quantize_weight(W)
    X = torch.randn((300, 128), device="cuda").half()
    Y = m8.llmint8_linear(X, Wq, sW)
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the calls below wait for this; what is taken here runs before them
        got = m8.llmint8_kv_attention(s.cache, b, q, stream=side)
        y = m8.llmint8_linear(X, Wq, sW, stream=side)
        other = [torch.full((n,), 77, dtype=torch.uint8, device="cuda")
                 for n in (size, size, size // 2, y.numel() * 2, got.numel() * 2, 1 << 20)]
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(y, Y)
        assert all(bool((t == 77).all()) for t in other)


def test_layer_refuses_input_that_requires_a_gradient():
    hidden, q_heads, heads, dim = 64, 2, 1, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    W, Wo, X = (torch.randn(n, device="cuda", generator=g).half() for n in
                (((q_heads + 2 * heads) * dim, hidden), (hidden, q_heads * dim), (5, hidden)))
    cache = m8.KVCache.empty(2, heads, dim, 16)
    layer = m8.Int8SelfAttention(W, Wo, q_heads, cache)
    seqs = m8.PagedSequences(cache)
    batch = seqs.extend([seqs.add()], [5])
    want = layer(X, batch)
    with pytest.raises(ValueError, match="gradient"):
        layer(X.requires_grad_(), batch)
    with torch.no_grad():
        assert torch.equal(layer(X, batch), want)


@pytest.mark.parametrize("lens,counts,q_heads,cu", [
    ([6000, 5000, 4000], [236, 2, 2], 4, [0, 236, 4, 240]),    # kv_prompt in parts: tokens 128..131 are nobody's
    ([6000, 5000, 4000], [4, 4, 4], 4, [0, 12, 0, 12]),        # kv_step in parts
])
def test_the_join_takes_no_row_of_a_run_that_there_is_not(lens, counts, q_heads, cu):
    """cu that falls leaves rows that no run holds, whose notes are what the workspace held: here places past
    the end of a run, or parts past the last one. Such rows are left alone, and so is what lies around."""
    s = Setup(85, lens, counts, 2, 64, 16)
    q, _ = s.values(q_heads, "bf16")
    b = s.batch(max(lens), cu)
    size = m8.llmint8_kv_attention_workspace_bytes(s.cache, b, q_heads)
    assert size > 0
    notes = s.rows * q_heads
    for place, parts in ((255, 1), (0x7fffff00, 1), (0, 2 ** 31 - 1), (-1, 5), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
        print(f"[case] {cu} note {place} {parts}", flush=True)
        space = torch.full((size // 4 + 2048,), 7, dtype=torch.int32, device="cuda")
        ws = space[1024:1024 + size // 4]
        ws[-2 * notes:] = torch.tensor([place, parts] * notes, dtype=torch.int32, device="cuda")
        out = torch.full((s.rows, q_heads, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        m8.llmint8_kv_attention(s.cache, b, q, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert (space[:1024] == 7).all() and (space[1024 + size // 4:] == 7).all()
        assert out.isfinite().all()
        if counts[0] == 236:
            assert (out[128:132] == 3.0).all()


PAST = [
    # table entries, lens, counts, heads, q_heads, dim, page, dtype
    (2, [33, 20], [1, 3], 2, 4, 64, 16, "f16"),          # one token past 32
    (3, [60, 48, 400], [30, 4, 2], 2, 2, 128, 16, "bf16"),
    (1, [100, 70], [80, 70], 1, 4, 64, 64, "f16"),
    (40, [700, 640], [90, 200], 1, 2, 64, 16, "bf16"),   # kv_prompt
    (300, [5000, 4790, 6000], [4, 4, 4], 1, 2, 64, 16, "f16"),  # in parts
]


@pytest.mark.parametrize("case", PAST)
def test_tokens_past_the_table(case):
    """Lengths that the table has no entries for: tokens there are written nowhere, read as zeros and are not
    seen; all others keep their places."""
    width, lens, counts, heads, q_heads, dim, page, dtype = case
    _say(f"past the table {case}")
    s = Setup(87, [min(n, width * page) for n in lens], counts, heads, dim, page, width=width)
    s.lens = list(lens)
    rope_np = oracle.rope_table(m8.rope_frequencies(dim)[0], max(lens))
    rope = torch.from_numpy(rope_np).cuda()
    k, kx = s.values(heads, dtype)
    v, vx = s.values(heads, dtype)
    q, qx = s.values(q_heads, dtype)
    qr = m8.llmint8_kv_append(s.cache, s.batch(), k, v, q=q, rope=rope)
    want = torch.from_numpy(s.ref.append(s.cu, s.lens, s.table, kx, vx, qx, rope_np)).to(TD[dtype])
    s.same_cache()
    assert torch.equal(qr.cpu(), want)
    gk, gv = m8.llmint8_kv_gather(s.cache, s.batch(), TD[dtype])
    for b, n in enumerate(lens):
        kx, vx, there = s.ref.tokens(s.table, b, n - counts[b], n)
        at = slice(s.cu[b], s.cu[b + 1])
        assert torch.equal(gk[at].cpu(), torch.from_numpy(kx).to(TD[dtype])), b
        assert torch.equal(gv[at].cpu(), torch.from_numpy(vx).to(TD[dtype])), b
        assert there.tolist() == [j < width * page for j in range(n - counts[b], n)]
    q = (qr, want.float().numpy())
    check_attention(s, q_heads, dtype, q=q, hints=(0, max(lens)))
    check_attention(s, q_heads, dtype, q=q, hints=(0, max(lens)), window=40, sinks=2)


def test_layer_in_a_captured_graph_with_a_fixed_number_of_rows():
    """As a server replays it: eight rows to a call, of which each step uses some, over growing sequences. Every
    replay against eager calls on a cache of their own."""
    g = torch.Generator(device="cuda").manual_seed(11)
    hidden, q_heads, heads, dim, rows, page = 256, 8, 2, 32, 8, 16
    W = (torch.randn(((q_heads + 2 * heads) * dim, hidden), device="cuda", generator=g) / 16).half()
    Wo = (torch.randn((hidden, q_heads * dim), device="cuda", generator=g) / 16).half()
    f, mag = m8.rope_frequencies(dim)
    rope = m8.llmint8_rope_table(f, 100, mag)
    X = torch.zeros((rows, hidden), device="cuda").half()
    table = torch.tensor([[5, 1, 7], [0, 4, 2], [3, 6, 8]], dtype=torch.int32, device="cuda")
    cu = torch.zeros((4,), dtype=torch.int32, device="cuda")
    lens = torch.zeros((3,), dtype=torch.int32, device="cuda")
    batch = m8.KVBatch(cu, lens, table, rows)
    mine, theirs = ([m8.Int8SelfAttention(W, Wo, q_heads, m8.KVCache.empty(9, heads, dim, page), rope=rope)][0] for _ in range(2))
    mine(X, batch)  # what a first call sets up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = mine(X, batch)
    held = [0, 0, 0]
    for counts in ([5, 2, 1], [1, 1, 1], [1, 0, 1], [3, 4, 0], [1, 1, 1], [0, 0, 0], [2, 1, 5], [1, 1, 1]):
        held = [h + n for h, n in zip(held, counts)]
        cu.copy_(torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32))
        lens.copy_(torch.tensor(held, dtype=torch.int32))
        X.copy_(torch.randn((rows, hidden), device="cuda", generator=g))
        graph.replay()
        got = Y.clone()
        want = theirs(X, batch)
        torch.cuda.synchronize()
        used = sum(counts)
        assert torch.equal(got, want), counts
        assert (got[used:] == 0).all() and (used == 0 or bool((got[:used] != 0).any()))
    for a, b in zip(mine.cache._t[:2], theirs.cache._t[:2]):
        for s, n in enumerate(held):
            for e in range(0, n, page):
                p = int(table[s, e // page])
                part = (lambda t: t[p, :, :n - e]) if a.shape[2] == page else (lambda t: t[p, :, :, :n - e])
                assert torch.equal(part(a), part(b))
