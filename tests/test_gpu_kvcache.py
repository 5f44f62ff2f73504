"""The int8 key/value cache on the GPU against the CPU oracle: writing (codes, magnitudes bit for bit),
reading back (bit for bit), attention over it.

Attention's bound, per row, derived from the arithmetic (u: unit roundoff of the output type):
  |o - o_ref| <= u |o_ref| + vmax (2^-10 + 2 d + 2^-13)
vmax: the largest |v| the row sees. 2^-10: the weights are held in 16 bits, either as fixed point of half a
step 2^-16 of the tile's largest over the 64 tokens of a tile, or in fp16 (2^-11 of each). d: what a q held to
2^-16 of its largest channel changes a logit by, which changes a weight by the factor 1 + d and the sum as
well. 2^-13: fp32 logits, exponentials and sums. lse: d + 2^-13 + 2^-20 |lse|.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TD = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


def _say(msg):
    print(f"[case] {msg}", flush=True)


class Setup:
    """A cache with random pages, tables of shuffled pages, and the oracle of the same content."""

    def __init__(self, seed, lens, counts, heads, dim, page, spare=2, width=None):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.counts = list(lens), list(counts)
        need = [-(-n // page) for n in lens]
        self.width = width or max(need + [1])
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lens), self.width), 2 ** 30, np.int32)  # unused entries name no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        K = rng.integers(-127, 128, (pages, heads, page, dim), dtype=np.int8)
        V = rng.integers(-127, 128, (pages, heads, dim, page), dtype=np.int8)
        # scales of pages differ by orders of magnitude; some pages hold zeros
        aK = (0.5 + 3 * rng.random((pages, heads))).astype(np.float32)
        aV = (2.0 ** rng.uniform(-6, 3, (pages, heads))).astype(np.float32)
        zero = rng.random((pages, heads)) < 0.1
        V[zero] = 0
        aV[zero] = 0
        for p in order[at:]:  # pages of nobody hold the worst
            aK[p] = np.nan
            aV[p] = np.inf
            K[p] = V[p] = -128
        self.heads, self.dim, self.page, self.pages = heads, dim, page, pages
        self.ref = oracle.KVOracle(K, V, aK, aV)
        self.cache = m8.KVCache(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (K, V, aK, aV)))

    def batch(self, max_len=0, cu=None, lens=None):
        dev = [torch.from_numpy(np.asarray(x, np.int32)).cuda()
               for x in (self.cu if cu is None else cu, self.lens if lens is None else lens, self.table)]
        return m8.KVBatch(dev[0], dev[1], dev[2], self.rows, max_len=max_len)

    def values(self, heads, dtype, scale=1.0, wide=False):
        """(device tensor [rows, heads, dim], its exact values)."""
        x = (self.rng.standard_normal((self.rows, heads, self.dim)) * scale).astype(np.float32)
        x[..., self.rng.integers(0, self.dim)] *= 8.0  # an outlier channel
        t = torch.from_numpy(x).cuda().to(TD[dtype])
        if wide:  # a slice of a wider tensor, other tokens' data between
            big = torch.full((self.rows, heads + 3, self.dim), 99.0, dtype=TD[dtype], device="cuda")
            big[:, 1:1 + heads] = t
            t = big[:, 1:1 + heads]
        return t, t.float().cpu().numpy()

    def same_cache(self):
        """Codes of every token that a sequence holds, and its pages' magnitudes, bit for bit."""
        torch.cuda.synchronize()
        K, V, aK, aV = (t.cpu().numpy() for t in (self.cache.K, self.cache.V, self.cache.aK, self.cache.aV))
        for b, n in enumerate(self.lens):
            for j in range(0, n, self.page):
                p, m = self.ref.page_of(self.table, b, j), min(self.page, n - j)
                if p < 0:
                    continue
                assert np.array_equal(aK[p], self.ref.aK[p]) and np.array_equal(aV[p], self.ref.aV[p]), (b, j)
                assert np.array_equal(K[p, :, :m], self.ref.K[p, :, :m]), (b, j)
                assert np.array_equal(V[p, :, :, :m], self.ref.V[p, :, :, :m]), (b, j)


APPEND = [
    # lens, counts, heads, q_heads, dim, page, rot, interleaved, dtype
    ([1], [1], 1, 1, 16, 16, 0, False, "f16"),
    ([64, 65, 63, 1, 200], [1, 1, 1, 1, 1], 2, 8, 128, 64, 128, False, "bf16"),
    ([130, 0, 17, 300], [130, 0, 5, 170], 3, 6, 80, 16, 80, False, "f16"),      # half of 40: not vectors of 8
    ([100, 257, 33], [37, 128, 33], 2, 4, 96, 32, 24, False, "bf16"),           # pairs inside a vector
    ([90, 128], [90, 64], 1, 5, 256, 128, 256, True, "f16"),
    ([77, 31, 500], [17, 17, 17], 4, 4, 64, 16, 16, True, "bf16"),
    ([50, 20], [50, 3], 2, 2, 48, 64, 22, True, "f16"),                         # rot ends inside a vector
    ([70, 141], [30, 100], 2, 2, 128, 64, 32, False, "f16"),
    ([300, 299], [300, 170], 16, 32, 64, 32, 64, False, "bf16"),
]


@pytest.mark.parametrize("case", APPEND)
def test_append_is_bit_exact(case):
    lens, counts, heads, q_heads, dim, page, rot, inter, dtype = case
    _say(f"append {case}")
    s = Setup(5, lens, counts, heads, dim, page)
    rope_np = oracle.rope_table(m8.rope_frequencies(rot)[0], max(lens) + 1) if rot else None
    rope = torch.from_numpy(rope_np).cuda() if rot else None
    for step in range(2):  # the second call writes larger values over the same slots
        k, kx = s.values(heads, dtype, 1.0 + 5 * step, wide=True)
        v, vx = s.values(heads, dtype, 1.0 + 5 * step)
        q, qx = s.values(q_heads, dtype, wide=True)
        out = m8.llmint8_kv_append(s.cache, s.batch(), k, v, q=q, rope=rope, interleaved=inter)
        want = s.ref.append(s.cu, s.lens, s.table, kx, vx, qx, rope_np, inter)
        s.same_cache()
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(TD[dtype]))
    # q where it stands
    back = m8.llmint8_kv_append(s.cache, s.batch(), k, v, q=q, rope=rope, interleaved=inter, q_out=q)
    assert back is q and torch.equal(q.cpu(), torch.from_numpy(want).to(TD[dtype]))


@pytest.mark.parametrize("page,dtype", [(16, "f16"), (64, "bf16"), (128, "f16")])
def test_append_token_by_token_moves_old_codes_to_the_grown_scale(page, dtype):
    heads, dim, n = 2, 64, 2 * page + 5
    s = Setup(9, [n, n], [1, 1], heads, dim, page)
    grow = 2.0 ** s.rng.uniform(-4, 4, n)
    for t in range(n):
        s.lens = [t + 1, t + 1]
        k, kx = s.values(heads, dtype, grow[t])
        v, vx = s.values(heads, dtype, grow[(t * 7) % n])
        m8.llmint8_kv_append(s.cache, s.batch(), k, v)
        s.ref.append(s.cu, s.lens, s.table, kx, vx)
    s.same_cache()


def test_append_zeros_tiny_values_and_rows_without_a_place():
    s = Setup(11, [40, 3, 90], [20, 7, 5], 2, 32, 16)  # seven rows for three tokens: four have no position
    s.table[2, 90 // 16] = -1                          # and the last page of the third does not exist
    k, kx = s.values(2, "bf16")
    v, vx = s.values(2, "bf16")
    k[:10] = 0
    kx[:10] = 0
    v[:20] = 1e-35
    vx[:20] = v[:20].float().cpu().numpy()
    q, qx = s.values(4, "bf16")
    sentinel = torch.full_like(q, 7.0)
    rope = oracle.rope_table([1.0, 0.25], 100)
    m8.llmint8_kv_append(s.cache, s.batch(), k, v, q=q, rope=torch.from_numpy(rope).cuda(), q_out=sentinel)
    s.ref.append(s.cu, s.lens, s.table, kx, vx, qx, rope)
    s.same_cache()
    assert (sentinel[20:24] == 7.0).all() and not (sentinel[24:27] == 7.0).all()


GATHER = [([1], 1, 16, 16, "f16"), ([100, 0, 64, 65], 2, 128, 64, "bf16"), ([33, 500], 3, 80, 32, "f16"),
          ([129], 8, 256, 128, "bf16"), ([31, 16, 17], 1, 112, 16, "f16"), ([700, 90], 4, 64, 64, "f16")]


@pytest.mark.parametrize("case", GATHER)
@pytest.mark.parametrize("whole", [True, False])
def test_gather_is_bit_exact(case, whole):
    lens, heads, dim, page, dtype = case
    counts = lens if whole else [min(n, 1 + n // 3) for n in lens]
    s = Setup(21, lens, counts, heads, dim, page)
    if len(lens) > 1:
        s.table[-1, 0] = -5  # a page that does not exist reads as zeros
    big = torch.full((s.rows, heads, dim + 24), 5.0, dtype=TD[dtype], device="cuda")
    k, v = m8.llmint8_kv_gather(s.cache, s.batch(), TD[dtype], k=big[:, :, :dim])
    for b, n in enumerate(lens):
        kx, vx, _ = s.ref.tokens(s.table, b, n - counts[b], n)
        rows = slice(s.cu[b], s.cu[b + 1])
        assert torch.equal(k[rows].cpu(), torch.from_numpy(kx).to(TD[dtype])), b
        assert torch.equal(v[rows].cpu(), torch.from_numpy(vx).to(TD[dtype])), b
    assert (big[:, :, dim:] == 5.0).all()


def check_attention(s, q_heads, dtype, q=None, hints=(0,), lse=True, **kw):
    if q is None:
        q = s.values(q_heads, dtype)
    want, want_lse, (vmax, d) = s.ref.attention(s.cu, s.lens, s.table, q[1], **kw)
    for hint in hints:
        got_lse = torch.full((s.rows, q_heads), 3.0, device="cuda")
        out = torch.full((s.rows, q_heads, s.dim), 3.0, dtype=TD[dtype], device="cuda")
        m8.llmint8_kv_attention(s.cache, s.batch(hint), q[0], out=out, lse=got_lse if lse else None, **kw)
        o = out.double().cpu().numpy()
        tol = U[dtype] * np.abs(want) + (vmax * (2.0 ** -10 + 2 * d + 2.0 ** -13))[..., None] + 2.0 ** -24
        err = np.abs(o - want)
        assert np.isfinite(o).all()
        worst = float((err / tol).max()) if o.size else 0.0
        print(f"[case] max_len {hint}: {worst:.3f} of the bound", flush=True)
        assert worst <= 1.0, worst
        seen = np.isfinite(want_lse)
        assert (o[~seen] == 0).all()
        if lse:
            L = got_lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(L), ~seen)
            assert (np.abs(L[seen] - want_lse[seen]) <= (d[seen] + 2.0 ** -13 + 2.0 ** -20 * np.abs(want_lse[seen]))).all()


ATTEND = [
    # lens, counts, heads, q_heads, dim, page, dtype, options
    ([1], [1], 1, 1, 16, 16, "f16", {}),
    ([1, 2, 63, 64, 65, 200], [1, 1, 1, 1, 1, 1], 2, 8, 128, 64, "bf16", {}),
    ([700, 0, 33], [1, 0, 1], 2, 2, 64, 16, "f16", {}),
    ([300, 129], [1, 1], 1, 16, 128, 32, "f16", {}),
    ([300, 129], [1, 1], 1, 20, 80, 32, "bf16", {}),                            # a group over two runs of rows
    ([260, 100, 3], [5, 7, 6], 2, 10, 96, 64, "f16", {}),                       # six rows of three tokens
    ([260, 77], [9, 77], 2, 6, 256, 128, "bf16", {}),
    ([500, 320, 1], [130, 320, 1], 2, 4, 128, 64, "f16", {}),                   # prompts
    ([600, 90], [400, 90], 1, 7, 64, 16, "bf16", {}),
    ([333, 401], [333, 150], 2, 2, 112, 32, "f16", {"window": 50, "sinks": 3}),
    ([900, 70, 400], [1, 1, 1], 2, 8, 128, 64, "bf16", {"window": 100, "sinks": 70}),
    ([900, 70, 400], [3, 3, 3], 2, 4, 64, 16, "f16", {"window": 1, "sinks": 0}),
    ([900, 70, 400], [2, 2, 2], 2, 4, 64, 128, "f16", {"window": 64, "sinks": 1}),
    ([200, 90], [60, 30], 2, 4, 128, 64, "f16", {"causal": False}),
    ([200, 90], [150, 1], 2, 4, 64, 32, "bf16", {"causal": False, "scale": 0.3}),
    ([450, 450], [200, 200], 1, 12, 256, 64, "f16", {"window": 130, "sinks": 5}),
    ([80, 40], [40, 40], 2, 2, 128, 16, "bf16", {"scale": -0.05}),
    ([80, 40], [40, 40], 2, 2, 128, 16, "f16", {"scale": 0.0}),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention(case):
    lens, counts, heads, q_heads, dim, page, dtype, kw = case
    _say(f"attention {case}")
    s = Setup(31, lens, counts, heads, dim, page)
    check_attention(s, q_heads, dtype, hints=(0, max(lens), 1, 10 ** 6), **kw)


def test_attention_of_strided_rows_into_strided_rows():
    s = Setup(33, [150, 70], [20, 4], 2, 64, 16)
    q = s.values(6, "f16", wide=True)
    want = m8.llmint8_kv_attention(s.cache, s.batch(), q[0].contiguous())
    big = torch.full((s.rows, 9, 64), 5.0, dtype=torch.float16, device="cuda")
    got = m8.llmint8_kv_attention(s.cache, s.batch(), q[0], out=big[:, 2:8])
    assert torch.equal(got, want) and (big[:, :2] == 5).all() and (big[:, 8:] == 5).all()
    # heads outermost
    qh = q[0].permute(1, 0, 2).contiguous().permute(1, 0, 2)
    oh = torch.empty((6, s.rows, 64), dtype=torch.float16, device="cuda").permute(1, 0, 2)
    assert torch.equal(m8.llmint8_kv_attention(s.cache, s.batch(), qh, out=oh), want)


@pytest.mark.parametrize("counts", [[1, 1, 1], [90, 1, 40]])
def test_attention_does_not_see_pages_that_do_not_exist(counts):
    s = Setup(35, [300, 64, 200], counts, 2, 128, 32)
    s.table[0, 2], s.table[0, 5], s.table[1, :] = -1, 2 ** 30, s.pages  # the second sequence has none at all
    check_attention(s, 4, "f16")
    check_attention(s, 4, "bf16", window=70, sinks=100)


@pytest.mark.parametrize("counts", [[1, 1], [200, 30]])
def test_attention_of_extreme_values(counts):
    """Logits in the hundreds, rows of zeros, a page's values 2^40 times another's."""
    s = Setup(37, [400, 90], counts, 2, 64, 64)
    s.ref.aV[s.table[0, 1]] = 2.0 ** 20
    s.ref.aV[s.table[0, 3]] = 2.0 ** -20
    s.cache.aV.copy_(torch.from_numpy(s.ref.aV))
    q, qx = s.values(4, "bf16", 10.0)
    q[0, 1] = 0
    qx[0, 1] = 0
    check_attention(s, 4, "bf16", q=(q, qx))


def test_attention_parts_join_whatever_the_hint():
    """One long sequence: the same rows from one part, a few and many."""
    s = Setup(39, [9000], [1], 1, 64, 64)
    check_attention(s, 2, "f16", hints=(1, 300, 2000, 9000, 0, 10 ** 8))
    s = Setup(40, [9000, 20], [4, 2], 1, 64, 16, width=700)
    check_attention(s, 2, "bf16", hints=(1, 9000, 0))


def test_rows_past_the_batch_are_left_alone():
    s = Setup(41, [100, 30], [3, 2], 2, 64, 16)
    s.rows = 9
    q, _ = s.values(4, "f16")
    for hint in (0, 100):
        out = torch.full((9, 4, 64), 3.0, dtype=torch.float16, device="cuda")
        m8.llmint8_kv_attention(s.cache, s.batch(hint), q, out=out)
        assert (out[5:] == 3.0).all() and not (out[:5] == 3.0).any(dim=2).all()


def test_hostile_batches_stay_inside_the_buffers():
    """cu that falls, leaves the rows or starts late, lengths past the table or below zero: no fault, and
    what is outside is untouched."""
    s = Setup(43, [100, 60, 40], [4, 4, 4], 2, 64, 16)
    q, _ = s.values(4, "f16")
    k, _ = s.values(2, "f16")
    guard = torch.full((3 * s.rows, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    for cu in ([0, 8, 4, 12], [0, 4, 900, 12], [-5, 4, 8, 12], [3, 3, 3, 3], [12, 8, 4, 0], [0, 4, 8, 2 ** 31 - 1]):
        for lens in ([100, 60, 40], [2 ** 31 - 1, -7, 0]):
            print(f"[case] {cu} {lens}", flush=True)
            b = s.batch(cu=cu, lens=lens)
            m8.llmint8_kv_append(s.cache, b, k, k, q=q, q_out=guard[s.rows:2 * s.rows])
            m8.llmint8_kv_attention(s.cache, b, q, out=guard[s.rows:2 * s.rows], window=20, sinks=3)
            m8.llmint8_kv_attention(s.cache, b, q, out=guard[s.rows:2 * s.rows])
            m8.llmint8_kv_gather(s.cache, b, k=guard[s.rows:2 * s.rows, :2], v=guard[s.rows:2 * s.rows, 2:])
            torch.cuda.synchronize()
            assert (guard[:s.rows] == 9).all() and (guard[2 * s.rows:] == 9).all()


def test_empty_calls():
    s = Setup(45, [5], [0], 2, 64, 16)
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    m8.llmint8_kv_append(s.cache, s.batch(), e, e)
    assert m8.llmint8_kv_attention(s.cache, s.batch(), e).shape == (0, 2, 64)
    assert m8.llmint8_kv_gather(s.cache, s.batch())[0].shape == (0, 2, 64)


def test_rope_table_and_frequencies():
    for f, mag in (m8.rope_frequencies(128), m8.rope_frequencies(64, 5e5, "yarn", 8.0, 8192),
                   m8.rope_frequencies(2), m8.rope_frequencies(96, 1e4, "linear", 4.0)):
        got = m8.llmint8_rope_table(f, 70000, mag).cpu().numpy()
        want = oracle.rope_table(f, 70000, mag)
        assert np.abs(got - want).max() <= 2.0 ** -23 * mag  # both from 64 bits: a step of rounding at most
    long = m8.llmint8_rope_table([1.0], 3_000_000).cpu().numpy()[-1]
    assert abs(long[0] - math.cos(2_999_999.0)) < 1e-6


def test_offsets_past_32_bits():
    """Pages whose codes begin past 2^32 bytes."""
    heads, dim, page = 8, 128, 64
    per = heads * dim * page
    pages = (2 ** 32) // per + 40
    c = m8.KVCache.empty(pages, heads, dim, page)
    ids = [pages - 1, 3, pages - 17, pages - 30]
    rng = np.random.default_rng(3)
    n = 230
    x = torch.from_numpy(rng.standard_normal((n, heads, dim)).astype(np.float32)).cuda().half()
    mk = lambda p, cache: m8.KVBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),  # noqa: E731
                                     torch.tensor([n], dtype=torch.int32, device="cuda"),
                                     torch.tensor([p], dtype=torch.int32, device="cuda"), n)
    small = m8.KVCache.empty(4, heads, dim, page)
    res = []
    for cache, p in ((c, ids), (small, [2, 0, 3, 1])):
        b = mk(p, cache)
        m8.llmint8_kv_append(cache, b, x, x)
        k, v = m8.llmint8_kv_gather(cache, b)
        res.append((k, v, m8.llmint8_kv_attention(cache, b, x),
                    m8.llmint8_kv_attention(cache, b, x, window=50, sinks=2)))
    for y, z in zip(*res):
        assert torch.equal(y, z)


def test_other_streams_and_graph_replay():
    s = Setup(47, [500, 200, 64], [1, 1, 1], 2, 128, 64)
    q, qx = s.values(8, "bf16")
    k, kx = s.values(2, "bf16")
    b = s.batch(500)
    rope_np = oracle.rope_table(m8.rope_frequencies(128)[0], 600)
    rope = torch.from_numpy(rope_np).cuda()
    ws = torch.empty((m8.llmint8_kv_attention_workspace_bytes(s.cache, b, 8),), dtype=torch.uint8, device="cuda")
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    qr = torch.empty_like(q)

    def step(stream=None):
        m8.llmint8_kv_append(s.cache, b, k, k, q=q, rope=rope, q_out=qr, stream=stream)
        m8.llmint8_kv_attention(s.cache, b, qr, out=out, workspace=ws, stream=stream)

    step()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        q2, _ = s.values(8, "bf16")
        q.copy_(q2)
        b.length.add_(1 if i == 2 else 0)  # the sequences grow between replays
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got), i


def test_same_result_every_time():
    s = Setup(49, [5000, 700], [3, 1], 2, 128, 64)
    q, _ = s.values(8, "f16")
    first = m8.llmint8_kv_attention(s.cache, s.batch(5000), q)
    for _ in range(5):
        assert torch.equal(m8.llmint8_kv_attention(s.cache, s.batch(5000), q), first)


def test_python_checks_of_arguments():
    s = Setup(51, [40], [4], 2, 64, 16)
    k, _ = s.values(2, "f16")
    q, _ = s.values(4, "f16")
    b = s.batch()
    with pytest.raises(ValueError):
        m8.llmint8_kv_append(s.cache, b, k, k.bfloat16())
    with pytest.raises(ValueError):
        m8.llmint8_kv_append(s.cache, b, k[:3], k[:3])
    with pytest.raises(ValueError):
        m8.llmint8_kv_append(s.cache, b, k.float(), k.float())
    with pytest.raises(ValueError):
        m8.llmint8_kv_append(s.cache, b, k, k, q_out=q)
    with pytest.raises(m8.Llmint8Error):
        m8.llmint8_kv_append(s.cache, b, k, k, rope=torch.zeros((9, 66), device="cuda"))
    with pytest.raises(ValueError):
        m8.llmint8_kv_attention(s.cache, b, q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(m8.Llmint8Error):
        m8.llmint8_kv_attention(s.cache, b, s.values(5, "f16")[0])
    with pytest.raises(m8.Llmint8Error):
        m8.llmint8_kv_attention(s.cache, b, q, causal=False, window=8)
    with pytest.raises(m8.Llmint8Error):
        m8.llmint8_kv_attention(s.cache, b, torch.zeros((4, 4, 68), dtype=torch.float16, device="cuda")[:, :, 4:])
    with pytest.raises(ValueError):
        m8.KVBatch(b.cu.long(), b.length, b.table, 4)
    with pytest.raises(ValueError):
        m8.KVCache(s.cache.K, s.cache.K, s.cache.aK, s.cache.aV)


def test_paged_sequences_keep_pages_apart():
    c = m8.KVCache.empty(10, 1, 16, 16)
    p = m8.PagedSequences(c)
    a, b = p.add(), p.add()
    t = p.extend([a, b], [40, 16])
    assert t.cu.tolist() == [0, 40, 56] and t.length.tolist() == [40, 16] and p.free_pages() == 6
    used = t.table[0, :3].tolist() + t.table[1, :1].tolist()
    assert len(set(used)) == 4
    t = p.extend([b], [1])
    assert t.length.tolist() == [17] and p.free_pages() == 5
    with pytest.raises(RuntimeError):
        p.extend([a], [200])
    assert p.length(a) == 40 and p.free_pages() == 5
    with pytest.raises(ValueError):
        p.extend([a, a], [1, 1])
    p.release(a)
    assert p.free_pages() == 8
    assert p.whole([b]).cu.tolist() == [0, 17]


def test_attention_layer_over_steps():
    """A prompt, then single tokens, through Int8SelfAttention: every call against the oracle fed with the
    layer's own projections."""
    torch.manual_seed(3)
    hidden, q_heads, heads, dim = 256, 8, 2, 32
    c = m8.KVCache.empty(12, heads, dim, 16)
    ref = oracle.KVOracle(*(np.zeros(tuple(t.shape), t.cpu().numpy().dtype) for t in (c.K, c.V, c.aK, c.aV)))
    f, mag = m8.rope_frequencies(dim)
    rope_np = oracle.rope_table(f, 100, mag)
    W = (torch.randn(((q_heads + 2 * heads) * dim, hidden), device="cuda") / 16).half()
    Wo = (torch.randn((hidden, q_heads * dim), device="cuda") / 16).half()
    layer = m8.Int8SelfAttention(W, Wo, q_heads, c, rope=torch.from_numpy(rope_np).cuda(), window=30, sinks=2)
    seqs = m8.PagedSequences(c)
    ids = [seqs.add(), seqs.add()]
    for counts in ([37, 20], [1, 1], [1, 1], [0, 3], [1, 1]):
        batch = seqs.extend(ids, counts)
        X = torch.randn((sum(counts), hidden), device="cuda").half()
        got = layer(X, batch)
        qkv = layer.qkv(X).view(-1, q_heads + 2 * heads, dim).float().cpu().numpy()
        cu, lens, table = (t.cpu().numpy() for t in (batch.cu, batch.length, batch.table))
        q = ref.append(cu, lens, table, qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:],
                       qkv[:, :q_heads], rope_np)
        q = q.astype(np.float16).astype(np.float32)
        o, _, (vmax, d) = ref.attention(cu, lens, table, q, window=30, sinks=2)
        tol = 2.0 ** -11 * np.abs(o) + (vmax * (2.0 ** -10 + 2 * d + 2.0 ** -13))[..., None] + 2.0 ** -24
        mine = m8.llmint8_kv_attention(c, batch, torch.from_numpy(q).cuda().half(), window=30, sinks=2)
        assert (np.abs(mine.double().cpu().numpy() - o) <= tol).all()
        assert torch.equal(layer.out(mine.view(-1, q_heads * dim)), got)


MORE = [
    # lens, counts, heads, q_heads, dim, page, dtype, options
    ([3 + 7 * b % 90 for b in range(300)], [b % 3 for b in range(300)], 2, 4, 32, 16, "f16", {}),     # many sequences
    ([40] * 520 + [5000], [1] * 521, 1, 2, 64, 16, "bf16", {}),                 # and one of them is cut
    ([5000] + [30] * 99, [1] * 100, 1, 32, 32, 64, "f16", {}),                  # more than 2048 rows to join
    ([2600, 3, 4100], [20, 3, 17], 2, 4, 128, 16, "bf16", {"window": 2500, "sinks": 40}),
    ([5000], [200], 1, 1, 128, 64, "f16", {}),                                  # a prompt's tokens in parts
    ([5000], [200], 1, 1, 80, 16, "bf16", {}),
    ([3000, 2500], [90, 300], 1, 2, 256, 32, "f16", {"window": 1500, "sinks": 7}),
    ([3000], [130], 2, 2, 64, 128, "bf16", {"causal": False}),
    ([4000], [140], 1, 1, 48, 16, "f16", {}),
    ([200, 90], [130, 90], 1, 3, 256, 16, "bf16", {}),                          # every width of page and head
    ([200, 90], [130, 90], 1, 3, 176, 128, "f16", {}),
    ([200, 90], [130, 90], 1, 3, 96, 32, "bf16", {}),
    ([200, 90], [130, 90], 1, 3, 16, 32, "f16", {}),
    ([70, 20], [2, 1], 1, 130, 16, 16, "f16", {}),                              # a group longer than a run
    ([70, 20], [40, 20], 1, 257, 16, 64, "bf16", {}),
    ([129, 1], [129, 1], 1, 128, 32, 16, "bf16", {}),
]


@pytest.mark.parametrize("case", MORE)
def test_attention_of_many_sequences_long_contexts_and_other_heads(case):
    lens, counts, heads, q_heads, dim, page, dtype, kw = case
    _say(f"attention {len(lens)} sequences to {max(lens)} {case[2:]}")
    s = Setup(61, lens, counts, heads, dim, page)
    check_attention(s, q_heads, dtype, hints=(0, max(lens)), **kw)


def test_append_and_gather_of_many_sequences():
    n = 530
    s = Setup(63, [1 + 13 * b % 70 for b in range(n)], [1 + b % 2 if b % 70 else 0 for b in range(n)], 2, 48, 32)
    k, kx = s.values(2, "bf16")
    v, vx = s.values(2, "bf16")
    m8.llmint8_kv_append(s.cache, s.batch(), k, v)
    s.ref.append(s.cu, s.lens, s.table, kx, vx)
    s.same_cache()
    gk, gv = m8.llmint8_kv_gather(s.cache, s.batch(), torch.bfloat16)
    for b in range(n):
        kx, vx, _ = s.ref.tokens(s.table, b, max(s.lens[b] - s.counts[b], 0), s.lens[b])
        rows = slice(s.cu[b + 1] - len(kx), s.cu[b + 1])
        assert torch.equal(gk[rows].cpu(), torch.from_numpy(kx).bfloat16()), b
        assert torch.equal(gv[rows].cpu(), torch.from_numpy(vx).bfloat16()), b


@pytest.mark.parametrize("lens,counts", [([6000, 5000, 40], [4, 4, 4]), ([600, 500, 40], [80, 80, 80])])
def test_hostile_batches_on_cut_and_prompt_calls(lens, counts):
    s = Setup(65, lens, counts, 2, 64, 16)
    q, _ = s.values(4, "bf16")
    n = s.rows
    guard = torch.full((3 * n, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3 * n, 4), 9.0, device="cuda")
    for cu in ([0, n - 4, 4, n], [0, 4, 90000, n], [-5, 4, 8, n], [3, 3, 3, 3], [n, 8, 4, 0], [0, 4, 8, 2 ** 31 - 1]):
        for length in (lens, [2 ** 31 - 1, -7, 0]):
            print(f"[case] {cu} {length}", flush=True)
            m8.llmint8_kv_attention(s.cache, s.batch(max(lens), cu, length), q, out=guard[n:2 * n], lse=lse[n:2 * n])
            torch.cuda.synchronize()
            for x in (guard, lse):
                assert (x[:n] == 9).all() and (x[2 * n:] == 9).all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("counts", [[1, 1], [4, 20], [300, 40]])
def test_values_that_are_not_finite(counts, page):
    """A NaN among a head's keys, an infinity among another's values: all of their pages reads as NaN and what
    sees one of their tokens gets NaN; every other row gets what it does without them."""
    lens, heads, q_heads, dim, dtype = [300, 40], 3, 6, 64, "bf16"
    s = Setup(67, lens, lens, heads, dim, page)
    k, kx = s.values(heads, dtype)
    v, vx = s.values(heads, dtype)
    s.ref.append(s.cu, s.lens, s.table, kx, vx)
    nan_at, inf_at = 150, 260  # of the first sequence
    k[nan_at, 0, 5] = math.nan
    v[inf_at, 1, 63] = -math.inf
    m8.llmint8_kv_append(s.cache, s.batch(), k, v)
    gk, gv = m8.llmint8_kv_gather(s.cache, s.batch(), torch.bfloat16)
    kx, vx, _ = s.ref.tokens(s.table, 0, 0, 300)
    want_k, want_v = (torch.from_numpy(x).bfloat16() for x in (kx, vx))
    pages = [slice(x // page * page, min(x // page * page + page, 300)) for x in (nan_at, inf_at)]
    want_k[pages[0], 0] = math.nan
    want_v[pages[1], 1] = math.nan
    for got, want in ((gk[:300].cpu(), want_k), (gv[:300].cpu(), want_v)):
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
    s.counts = counts
    s.cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    s.rows = int(s.cu[-1])
    for kw in ({}, {"window": 60, "sinks": 2}):
        q, qx = s.values(q_heads, dtype)
        bad = counts[0] - 1  # a row with a NaN of its own, on the head of neither
        q[bad, 5, 9] = math.nan
        want, want_lse, (vmax, d) = s.ref.attention(s.cu, s.lens, s.table, qx, **kw)
        lse = torch.empty((s.rows, q_heads), device="cuda")
        for hint in (0, 300):
            o = m8.llmint8_kv_attention(s.cache, s.batch(hint), q, lse=lse, **kw).double().cpu().numpy()
            L = lse.double().cpu().numpy()
            pos = 300 - counts[0] + np.arange(counts[0])
            no = np.zeros((s.rows, q_heads), bool)
            for h, sl in ((0, pages[0]), (1, pages[1])):
                sees = (pos >= sl.start) & ((pos - kw["window"] < sl.stop - 1) if kw else True)
                no[:counts[0], 2 * h:2 * h + 2] = sees[:, None]
            no[bad, 5] = True
            assert np.array_equal(np.isnan(o).any(2), no) and np.array_equal(np.isnan(o).all(2), no)
            assert np.array_equal(np.isnan(L), no)
            tol = U[dtype] * np.abs(want) + (vmax * (2.0 ** -10 + 2 * d + 2.0 ** -13))[..., None] + 2.0 ** -24
            assert (np.abs(o - want)[~no] <= tol[~no]).all()
            assert (np.abs(L - want_lse)[~no] <= (d + 2.0 ** -13 + 2.0 ** -20 * np.abs(want_lse))[~no]).all()


@pytest.mark.parametrize("dim,page,dtype,longest", [(64, 64, "bf16", 200), (64, 16, "f16", 4400), (80, 32, "bf16", 4400),
                                                    (96, 64, "f16", 4400), (96, 16, "f16", 150), (112, 16, "bf16", 150),
                                                    (112, 128, "bf16", 4400), (128, 64, "f16", 150), (48, 16, "f16", 150),
                                                    (128, 32, "bf16", 4400), (256, 64, "f16", 4400), (192, 16, "f16", 99)])
def test_attention_of_drafted_tokens_of_a_large_batch(dim, page, dtype, longest):
    """Runs of two sixteens, enough of them to fill half the chip: some of one sixteen only, some of no rows."""
    heads, G = 16, 5
    counts = [(0, 3, 4, 5, 6, 9)[b % 6] for b in range(26)]
    lens = [max(n, 5 + 37 * b % 150) for b, n in enumerate(counts)]
    lens[4] = longest
    s = Setup(71, lens, counts, heads, dim, page)
    _say(f"drafts {dim} {page} {dtype} {longest}")
    check_attention(s, heads * G, dtype, hints=(0, 1))
    check_attention(s, heads * G, dtype, window=64, sinks=2)


def test_example_of_a_server():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main("--layers 1 --users 3 --steps 4 --q-heads 8 --heads 2 --dim 64 --context 300".split())
