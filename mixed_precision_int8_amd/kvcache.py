"""The int8 key/value cache: binding of llmint8_kv_* and llmint8_rope_table, the page
bookkeeping of a server (``PagedSequences``) and an attention block on int8 linears
(``Int8SelfAttention``). As elsewhere, every computation runs in the library's HIP
kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


class _Cache(ctypes.Structure):
    _fields_ = [("K", _vp), ("V", _vp), ("aK", _vp), ("aV", _vp), ("pages", _i64), ("heads", _i64),
                ("page", _i64), ("dim", _i64)]


class _Batch(ctypes.Structure):
    _fields_ = [("cu", _vp), ("len", _vp), ("table", _vp), ("seqs", _i64), ("rows", _i64),
                ("width", _i64), ("max_len", _i64)]


def _m8():
    import mixed_precision_int8_amd as m8
    return m8


def _stream(stream, device):
    """The stream's handle. The current one's is asked for without a Stream object around it where torch
    has such a call (0.1 us, 2 us otherwise: a sixth of a short call's time on the host)."""
    import torch
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return raw(device.index)


class KVCache:
    """A pool of cache pages: K int8 [pages, heads, page, dim], V int8 [pages, heads, dim, page] and the
    magnitudes aK, aV fp32 [pages, heads], held by the caller (see ``KVCache.empty``)."""

    __slots__ = ("_t", "_c", "_ref", "pages", "heads", "page", "dim", "device")

    def __init__(self, K, V, aK, aV):
        import torch
        m8 = _m8()
        if K.dim() != 4:
            raise ValueError(f"K: expected [pages, heads, page, dim], got {tuple(K.shape)}")
        self.pages, self.heads, self.page, self.dim = K.shape
        m8._need(K, torch.int8, (self.pages, self.heads, self.page, self.dim), "K")
        m8._need(V, torch.int8, (self.pages, self.heads, self.dim, self.page), "V")
        m8._need(aK, torch.float32, (self.pages, self.heads), "aK")
        m8._need(aV, torch.float32, (self.pages, self.heads), "aV")
        if not K.device == V.device == aK.device == aV.device:
            raise ValueError("K, V, aK and aV: expected on one device")
        self.device = K.device
        self._t = (K, V, aK, aV)
        self._c = _Cache(K.data_ptr(), V.data_ptr(), aK.data_ptr(), aV.data_ptr(), *K.shape)
        self._ref = ctypes.c_void_p(ctypes.addressof(self._c))

    @classmethod
    def empty(cls, pages, heads, dim, page=64, device="cuda"):
        import torch
        return cls(torch.empty((pages, heads, page, dim), dtype=torch.int8, device=device),
                   torch.empty((pages, heads, dim, page), dtype=torch.int8, device=device),
                   torch.empty((pages, heads), dtype=torch.float32, device=device),
                   torch.empty((pages, heads), dtype=torch.float32, device=device))

    K = property(lambda self: self._t[0])
    V = property(lambda self: self._t[1])
    aK = property(lambda self: self._t[2])
    aV = property(lambda self: self._t[3])

    def memory_bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._t)


class KVBatch:
    """The sequences of a call: ``cu`` int32 [seqs + 1] (rows cu[b]..cu[b+1]-1 are the last tokens of
    sequence b), ``length`` int32 [seqs] (tokens in the cache, these rows included), ``table`` int32
    [seqs, width] (pages). The contents may change between calls; ``rows`` is the number of rows of the
    call's tensors, ``max_len`` about the largest length (it sizes the work; any value is correct).
    ``positions``, where the host knows it: the rows' positions are below it (``PagedSequences`` sets it)."""

    __slots__ = ("_t", "_c", "_ref", "seqs", "rows", "device", "positions")

    def __init__(self, cu, length, table, rows, max_len=0, positions=None):
        import torch
        m8 = _m8()
        self.seqs = length.shape[0] if length.dim() == 1 else -1
        m8._need(length, torch.int32, (self.seqs,), "length")
        m8._need(cu, torch.int32, (self.seqs + 1,), "cu")
        if table.dim() != 2:
            raise ValueError(f"table: expected [seqs, width], got {tuple(table.shape)}")
        m8._need(table, torch.int32, (self.seqs, table.shape[1]), "table")
        if not cu.device == length.device == table.device:
            raise ValueError("cu, length and table: expected on one device")
        self.rows = int(rows)
        if self.rows < 0 or max_len < 0:
            raise ValueError("rows and max_len: expected >= 0")
        self.device = cu.device
        self.positions = positions
        self._t = (cu, length, table)
        self._c = _Batch(cu.data_ptr(), length.data_ptr(), table.data_ptr(), self.seqs, self.rows,
                         table.shape[1], int(max_len))
        self._ref = ctypes.c_void_p(ctypes.addressof(self._c))

    cu = property(lambda self: self._t[0])
    length = property(lambda self: self._t[1])
    table = property(lambda self: self._t[2])


def _grad_enabled():
    import torch
    return torch.is_grad_enabled()


def _rows(t, dtype, rows, heads, dim, device, name):
    """(pointer, token stride, head stride) of 16-bit rows [rows, heads, dim] with dense channels. The calls
    have no backward: a tensor that takes part in a graph would leave it without a word, so it is refused."""
    if t.requires_grad and _grad_enabled():
        raise ValueError(f"{name}: requires a gradient, and the key/value cache has none to give (detach it, or "
                         "call under torch.no_grad())")
    if t.dtype != dtype or t.shape != (rows, heads, dim) or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {(rows, heads, dim)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    st, sh, sc = t.stride()
    if sc != 1 and dim > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the channels must be dense, got strides {t.stride()}")
    return t.data_ptr(), st, sh


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0, beta_fast=32.0,
                     beta_slow=1.0):
    """(frequencies [rot / 2], magnitude) of rotary positions over ``rot`` channels: base^(-2i/rot), for
    long contexts scaled by ``factor``. ``scaling``: None; "linear" (all divided by the factor); "ntk"
    (the base raised so that the slowest is divided by it); "yarn" (Peng et al., "YaRN: Efficient Context
    Window Extension of Large Language Models", 2023: frequencies that turn more than ``beta_fast`` times
    within the ``original`` context stay, those under ``beta_slow`` turns are divided, a ramp between, and
    the magnitude 0.1 ln(factor) + 1)."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot: expected even and >= 2, got {rot}")
    if factor < 1:
        raise ValueError(f"factor: expected >= 1, got {factor}")
    half = rot // 2
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(half)]
    if scaling is None or scaling == "ntk":
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "yarn":
        raise ValueError(f"scaling: None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if original <= 0:
        raise ValueError("yarn: the original context length is needed")

    def index(turns):  # where a frequency turns that often within the original context
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rot - 1)
    out = []
    for i, x in enumerate(f):
        ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        out.append(x * (1 - ramp) + x / factor * ramp)
    return out, (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


def llmint8_rope_table(freq, rows, magnitude=1.0, table=None, device="cuda", stream=None):
    """fp32 [rows, 2 * len(freq)]: magnitude * cos(p f_i), then magnitude * sin(p f_i)."""
    import torch
    m8 = _m8()
    lib = m8.load_library()
    n = len(freq)
    if table is None:
        table = m8._empty((rows, 2 * n), torch.float32, device, stream)
    m8._need(table, torch.float32, (rows, 2 * n), "table")
    arr = (ctypes.c_double * max(n, 1))(*[float(x) for x in freq])
    m8._check(lib.llmint8_rope_table(arr, n, rows, float(magnitude), table.data_ptr(),
                                     _stream(stream, table.device)),
              "llmint8_rope_table")
    return table


def _same_device(cache, batch):
    if cache.device != batch.device:
        raise ValueError(f"batch: expected on {cache.device}, got {batch.device}")


def llmint8_kv_append(cache, batch, k, v, q=None, rope=None, interleaved=False, q_out=None, stream=None):
    """Write k, v [rows, heads, dim] (fp16 or bf16) to the cache, k rotated by ``rope`` (fp32 [positions,
    rot], from ``llmint8_rope_table``) on the way. ``q`` [rows, q_heads, dim], if given, is rotated into
    ``q_out`` (new by default; may be ``q``), which is returned. Positions that ``rope`` has no row for are
    refused where the batch knows its ``positions``; otherwise they take its last row."""
    import torch
    m8 = _m8()
    lib = m8.load_library()
    _same_device(cache, batch)
    code = m8._act_dtype(k.dtype)
    n, dev = batch.rows, cache.device
    kr = _rows(k, k.dtype, n, cache.heads, cache.dim, dev, "k")
    vr = _rows(v, k.dtype, n, cache.heads, cache.dim, dev, "v")
    qr = orr = (None, 0, 0)
    heads = 0
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else -1
        qr = _rows(q, k.dtype, n, heads, cache.dim, dev, "q")
        if q_out is None:
            q_out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
                     else m8._empty(q.shape, q.dtype, dev, stream))
        orr = _rows(q_out, k.dtype, n, heads, cache.dim, dev, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    table, table_rows, rot = None, 0, 0
    if rope is not None:
        if rope.dim() != 2 or rope.dtype != torch.float32 or not rope.is_contiguous() or rope.device != dev:
            raise ValueError(f"rope: expected contiguous fp32 [positions, rot] on {dev}, got {rope.dtype} "
                             f"{tuple(rope.shape)} on {rope.device}")
        table_rows, rot = rope.shape
        if batch.positions is not None and batch.positions > table_rows:
            raise ValueError(f"rope: {table_rows} positions, and the batch's rows reach {batch.positions}")
        table = rope.data_ptr()
    m8._check(lib.llmint8_kv_append(cache._ref, batch._ref, code, *kr, *vr, *qr, *orr, heads, table,
                                    table_rows, rot, 1 if interleaved else 0, _stream(stream, dev)),
              "llmint8_kv_append")
    return q_out


def llmint8_kv_gather(cache, batch, dtype=None, k=None, v=None, stream=None):
    """(k, v) [rows, heads, dim] in ``dtype`` (fp16 by default): the batch's tokens read back."""
    import torch
    m8 = _m8()
    lib = m8.load_library()
    _same_device(cache, batch)
    dtype = dtype or (k.dtype if k is not None else v.dtype if v is not None else torch.float16)
    code = m8._act_dtype(dtype)
    shape, dev = (batch.rows, cache.heads, cache.dim), cache.device
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=dev) if stream is None else m8._empty(shape, dtype, dev, stream)
    if v is None:
        v = (torch.empty_like(k, memory_format=torch.contiguous_format) if stream is None
             else m8._empty(shape, dtype, dev, stream))
    m8._check(lib.llmint8_kv_gather(cache._ref, batch._ref, code, *_rows(k, dtype, *shape, dev, "k"),
                                    *_rows(v, dtype, *shape, dev, "v"), _stream(stream, dev)),
              "llmint8_kv_gather")
    return k, v


def llmint8_kv_attention_workspace_bytes(cache, batch, q_heads, window=0, sinks=0) -> int:
    return int(_m8().load_library().llmint8_kv_attention_workspace_bytes(cache._ref, batch._ref, q_heads,
                                                                         window, sinks))


def llmint8_kv_attention(cache, batch, q, scale=None, causal=True, window=0, sinks=0, out=None, lse=None,
                         workspace=None, stream=None):
    """out [rows, q_heads, dim] = attention of q (fp16 or bf16, rotated) over the cache. ``scale`` is
    1 / sqrt(dim) by default; ``window`` > 0 keeps the last ``window`` tokens and the first ``sinks`` ones
    of what a row sees; ``lse`` fp32 [rows, q_heads] receives the log sums."""
    import torch
    m8 = _m8()
    lib = m8.load_library()
    _same_device(cache, batch)
    code = m8._act_dtype(q.dtype)
    n, dev = batch.rows, cache.device
    heads = q.shape[1] if q.dim() == 3 else -1
    qr = _rows(q, q.dtype, n, heads, cache.dim, dev, "q")
    if out is None:
        out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
               else m8._empty(q.shape, q.dtype, dev, stream))
    orr = _rows(out, q.dtype, n, heads, cache.dim, dev, "out")
    if lse is not None:
        m8._need(lse, torch.float32, (n, heads), "lse")
        if lse.device != dev:
            raise ValueError(f"lse: expected on {dev}, got {lse.device}")
    if workspace is None:
        need = lib.llmint8_kv_attention_workspace_bytes(cache._ref, batch._ref, heads, window, sinks)
        if need > 0:
            workspace = m8._empty((need,), torch.uint8, dev, stream)
    else:
        m8._need_workspace(workspace, dev)
    m8._check(lib.llmint8_kv_attention(cache._ref, batch._ref, code, *qr, heads,
                                       1.0 / math.sqrt(cache.dim) if scale is None else float(scale),
                                       1 if causal else 0, window, sinks, *orr,
                                       None if lse is None else lse.data_ptr(), m8._ptr(workspace),
                                       m8._ws_bytes(workspace), _stream(stream, dev)),
              "llmint8_kv_attention")
    return out


class PagedSequences:
    """Which pages of a cache belong to which sequence: the bookkeeping of a server, on the host.

    ``extend`` reserves room for new tokens and returns the ``KVBatch`` of the call that writes and
    attends to them; ``release`` gives a sequence's pages back."""

    def __init__(self, cache):
        self.cache = cache
        self._free = list(range(cache.pages - 1, -1, -1))
        self._pages, self._len, self._next = {}, {}, 0

    def add(self) -> int:
        """A new, empty sequence."""
        s = self._next
        self._next += 1
        self._pages[s], self._len[s] = [], 0
        return s

    def release(self, seq):
        self._free.extend(reversed(self._pages.pop(seq)))
        del self._len[seq]

    def length(self, seq) -> int:
        return self._len[seq]

    def free_pages(self) -> int:
        return len(self._free)

    def extend(self, seqs, counts) -> KVBatch:
        """The batch of a call that brings ``counts[i]`` new tokens to sequence ``seqs[i]``."""
        import torch
        seqs, counts = list(seqs), [int(n) for n in counts]
        if len(seqs) != len(counts) or len(set(seqs)) != len(seqs) or min(counts, default=0) < 0:
            raise ValueError("extend: one count >= 0 for each of a list of different sequences")
        P = self.cache.page
        need = sum(max(0, -(-(self._len[s] + n) // P) - len(self._pages[s])) for s, n in zip(seqs, counts))
        if need > len(self._free):
            raise RuntimeError(f"key/value cache full: {need} pages needed, {len(self._free)} free")
        for s, n in zip(seqs, counts):
            self._len[s] += n
            while len(self._pages[s]) * P < self._len[s]:
                self._pages[s].append(self._free.pop())
        return self._batch(seqs, counts)

    def whole(self, seqs) -> KVBatch:
        """The batch that names every token of the sequences (to read them back)."""
        seqs = list(seqs)
        return self._batch(seqs, [self._len[s] for s in seqs])

    def _batch(self, seqs, counts):
        import torch
        width = max([len(self._pages[s]) for s in seqs] + [1])
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        lens = [self._len[s] for s in seqs]
        table = [self._pages[s] + [0] * (width - len(self._pages[s])) for s in seqs]
        # one transfer for the three arrays
        flat = torch.tensor(cu + lens + [p for t in table for p in t], dtype=torch.int32).to(self.cache.device)
        b = len(seqs)
        parts = [flat[:b + 1].clone(), flat[b + 1:2 * b + 1].clone(), flat[2 * b + 1:].clone()]
        return KVBatch(parts[0], parts[1], parts[2].view(b, width), cu[-1], max_len=max(lens, default=0),
                       positions=max((n for n, m in zip(lens, counts) if m > 0), default=0))


class Int8SelfAttention:
    """Self-attention of a decoder layer on int8 weights and an int8 cache: q, k, v from one Int8Linear,
    rotated and written by ``llmint8_kv_append``, attended by ``llmint8_kv_attention``, and projected by a
    second Int8Linear. ``qkv_weight`` is [(q_heads + 2 heads) * dim, hidden], ``out_weight`` [hidden,
    q_heads * dim]. For serving: there is no backward through the cache, and X that requires a gradient is
    refused (but under ``torch.no_grad()``)."""

    def __init__(self, qkv_weight, out_weight, q_heads, cache, rope=None, interleaved=False, window=0,
                 sinks=0, threshold=6.0):
        m8 = _m8()
        if qkv_weight.shape[0] != (q_heads + 2 * cache.heads) * cache.dim:
            raise ValueError(f"qkv_weight: expected {(q_heads + 2 * cache.heads) * cache.dim} rows, got "
                             f"{qkv_weight.shape[0]}")
        self.qkv = m8.Int8Linear(qkv_weight, threshold)
        self.out = m8.Int8Linear(out_weight, threshold)
        self.cache, self.q_heads = cache, int(q_heads)
        self.rope, self.interleaved, self.window, self.sinks = rope, interleaved, window, sinks

    def forward(self, X, batch):
        """Y [rows, hidden] for the batch's new tokens X [rows, hidden], which join the cache. Rows of X past
        the batch's attend to nothing: their attention is zero."""
        import torch
        c, nq = self.cache, self.q_heads
        qkv = self.qkv(X).view(X.shape[0], nq + 2 * c.heads, c.dim)
        q = llmint8_kv_append(c, batch, qkv[:, nq:nq + c.heads], qkv[:, nq + c.heads:], qkv[:, :nq],
                              self.rope, self.interleaved, q_out=qkv[:, :nq])
        # the attention writes the batch's rows only, and the second projection decides its outlier columns over
        # all rows: what memory held in the others must not reach it
        o = torch.zeros((X.shape[0], nq, c.dim), dtype=qkv.dtype, device=qkv.device)
        llmint8_kv_attention(c, batch, q, window=self.window, sinks=self.sinks, out=o)
        return self.out(o.view(X.shape[0], nq * c.dim))

    __call__ = forward
