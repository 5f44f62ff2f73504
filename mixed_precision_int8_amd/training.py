"""Training through a layer on int8 weights: binding of llmint8_attention, llmint8_rope, llmint8_layer_norm,
llmint8_grad_* and their gradients, and the differentiable functions on top of them (``packed_attention``,
``rotary``, ``layer_norm``, ``LayerNorm``). As elsewhere, every computation runs in the library's HIP kernels;
there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct
import sys

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64

m8 = sys.modules[__package__]  # the package: its loader and helpers are looked up when a call needs them
torch = None                   # imported by the first call, as elsewhere in the package

# llmint8_rows and llmint8_attention_shape as the calls hand them over: packed, which costs a third of filling
# a ctypes structure (12 of them to an attention step with its gradient)
_ROWS = struct.Struct("=3q").pack
_SHAPE = struct.Struct("=6qfi2q").pack


class _Grad(ctypes.Structure):
    _fields_ = [("data", _vp), ("out", _vp), ("n", _i64), ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


def bind(lib):
    """Argument types of the library's entry points of this file."""
    i, p, d = ctypes.c_int, ctypes.POINTER, ctypes.c_double
    r = ctypes.c_char_p  # packed structures
    types = {
        "attention": [r, i, r, r, r, r, _vp, _vp],
        "attention_backward": [r, i, r, r, r, r, _vp, r, r, r, r, _vp, ctypes.c_size_t, _vp],
        "rope": [i, r, r, _i64, r, r, _i64, _i64, _i64, _vp, _i64, ctypes.c_char_p, _vp, _i64, _i64, i, i, _vp],
        "layer_norm": [_vp, _i64, i, _i64, _i64, _vp, _vp, i, ctypes.c_float, _vp, _i64, _vp, _vp],
        "layer_norm_backward": [_vp, _i64, _vp, _i64, i, _i64, _i64, _vp, i, _vp, _vp, _i64, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp],
        "grad_norm": [p(_Grad), _i64, d, _vp, _vp, ctypes.c_size_t, _vp],
        "grad_clip": [p(_Grad), _i64, _vp, d, d, _vp],
    }
    sizes = {
        "attention_backward_workspace_bytes": [r],
        "layer_norm_workspace_bytes": [_i64, _i64],
        "grad_norm_workspace_bytes": [p(_Grad), _i64],
    }
    for names, result in ((types, ctypes.c_int), (sizes, ctypes.c_size_t)):
        for name, args in names.items():
            fn = getattr(lib, "llmint8_" + name)
            fn.argtypes, fn.restype = args, result


def _library():
    global torch
    if torch is None:
        import torch as t
        torch = t
    return m8.load_library()


def _handle(stream, device):
    return m8.kvcache._stream(stream, device)


_NOTHING = contextlib.nullcontext()


def _on(device):
    """The call's device as the current one: a launch on a device's default stream goes to the current device."""
    if device.type != "cuda" or device.index in (None, torch._C._cuda_getDevice()):
        return _NOTHING
    return torch.cuda.device(device)


def _dtype(dtype, name):
    if dtype == torch.float16:
        return m8.LLMINT8_DTYPE_F16
    if dtype == torch.bfloat16:
        return m8.LLMINT8_DTYPE_BF16
    if dtype == torch.float32:
        return m8.LLMINT8_DTYPE_F32
    raise ValueError(f"{name}: fp16, bf16 or fp32 only, got {dtype}")


def _half(dtype):
    if dtype == torch.float16:
        return m8.LLMINT8_DTYPE_F16
    if dtype == torch.bfloat16:
        return m8.LLMINT8_DTYPE_BF16
    raise ValueError(f"fp16 or bf16 only, got {dtype}")


def _plain(tensors, names, instead):
    """The calls named as the library's leave the graph without a word, so what would need one is refused."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{names}: one requires a gradient, which this call does not record: use {instead} (or "
                             "detach it, or call under torch.no_grad())")


def _rows(t, dtype, shape, device, name):
    """16-bit rows [rows, heads, dim] with dense channels, as the library takes them."""
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    st, sh, sc = t.stride()
    if sc != 1 and shape[2] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the channels must be dense, got strides {t.stride()}")
    return _ROWS(t.data_ptr(), st, sh)


def _new(shape, dtype, device, stream):
    return torch.empty(shape, dtype=dtype, device=device) if stream is None else m8._empty(shape, dtype, device, stream)


def _like(t, stream):
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return m8._empty(t.shape, t.dtype, t.device, stream)


# ---- attention


class PackedRows:
    """Sequences one after the other: rows cu[b] .. cu[b+1]-1 (``cu`` int32 [seqs + 1], device memory) are sequence
    b of a call whose tensors have ``rows`` rows. The contents of ``cu`` may change between calls and between a
    captured graph's replays.

    ``used``, where the host knows it: cu[seqs] (rows past it belong to no sequence). It is of what cu holds now: after
    an operation on cu, and in a captured call, it counts as unknown, until it is assigned anew. ``max_len``, if known:
    no sequence is longer, whatever cu will hold (``of`` knows it of its lengths only; it may be assigned). Operations
    on cu are seen as autograd sees them, by its version; who writes its memory behind that (``cu.data``, a kernel of
    their own) gives neither."""

    __slots__ = ("cu", "seqs", "rows", "device", "_used", "_max_len", "_version", "_of")

    def __init__(self, cu, rows, max_len=0, used=None):
        _library()
        self.seqs = cu.shape[0] - 1 if cu.dim() == 1 else -1
        if self.seqs < 0:
            raise ValueError(f"cu: expected [seqs + 1], got {tuple(cu.shape)}")
        m8._need(cu, torch.int32, (self.seqs + 1,), "cu")
        self.rows = int(rows)
        if self.rows < 0:
            raise ValueError(f"rows: expected >= 0, got {rows}")
        self.cu, self.device = cu, cu.device
        self.max_len, self.used = max_len, used

    @property
    def used(self):
        return self._used

    @used.setter
    def used(self, used):
        if used is not None and used < 0:
            raise ValueError(f"used: expected >= 0, got {used}")
        self._used = None if used is None else min(int(used), self.rows)
        self._version = None if self.cu.is_inference() else self.cu._version  # None: changes of cu are not seen

    @property
    def max_len(self):
        return self._max_len

    @max_len.setter
    def max_len(self, max_len):
        if max_len < 0:
            raise ValueError(f"max_len: expected >= 0, got {max_len}")
        self._max_len, self._of = int(max_len), None

    @classmethod
    def of(cls, lengths, rows=None, device="cuda"):
        """Of sequences of these lengths (a list), in a call of ``rows`` rows (their sum by default)."""
        _library()
        at = [0]
        for n in lengths:
            if n < 0:
                raise ValueError(f"lengths: expected >= 0, got {n}")
            at.append(at[-1] + int(n))
        if rows is not None and rows < at[-1]:
            raise ValueError(f"rows: {rows}, and the sequences have {at[-1]}")
        with torch.inference_mode(False):  # inference tensors have no version
            cu = torch.tensor(at, dtype=torch.int32).to(device)
        batch = cls(cu, at[-1] if rows is None else rows, max_len=max(lengths, default=0), used=at[-1])
        batch._of = batch._version
        return batch

    def used_rows(self):
        """``used`` while it holds, else None."""
        if self.used is None or self._version is None or self.cu._version != self._version:
            return None
        with _on(self.device):  # torch asks about the current device's stream
            return None if torch.cuda.is_current_stream_capturing() else self.used

    def longest(self):
        """No sequence has more tokens, as far as the host knows."""
        if self._of is not None:
            return self.max_len if self.cu._version == self._of else self.rows
        return self.max_len or self.rows

    def positions(self):
        """int32 [rows]: every row's place in its sequence, from what cu holds now (rows of no sequence: any)."""
        row = torch.arange(self.rows, dtype=torch.int32, device=self.device)
        seq = torch.searchsorted(self.cu[1:], row, right=True, out_int32=True)
        return (row - self.cu[seq]).clamp_(min=0)


def _shape(batch, q, k, scale, causal, window, sinks):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q and k: expected [rows, heads, dim], got {tuple(q.shape)} and {tuple(k.shape)}")
    dim = q.shape[2]
    return _SHAPE(batch.cu.data_ptr(), batch.seqs, batch.rows, q.shape[1], k.shape[1], dim,
                  1.0 / math.sqrt(max(dim, 1)) if scale is None else float(scale), 1 if causal else 0, window, sinks)


def llmint8_attention(batch, q, k, v, scale=None, causal=True, window=0, sinks=0, out=None, lse=None, stream=None):
    """(out [rows, q_heads, dim], lse fp32 [rows, q_heads]): attention of each of the batch's sequences over its own
    tokens. q [rows, q_heads, dim], k and v [rows, heads, dim], fp16 or bf16; ``scale`` is 1 / sqrt(dim) by default;
    ``window`` > 0 (causal) keeps the last ``window`` tokens and the first ``sinks`` ones. Rows of no sequence are
    left as they were."""
    lib = _library()
    _plain((q, k, v), "q, k and v", "packed_attention")
    dev, dt = batch.device, q.dtype
    s = _shape(batch, q, k, scale, causal, window, sinks)
    code = _half(dt)
    heads, dim, n = q.shape[1], q.shape[2], batch.rows
    wide, narrow = (n, heads, dim), (n, k.shape[1], dim)
    rows = [_rows(q, dt, wide, dev, "q"), _rows(k, dt, narrow, dev, "k"), _rows(v, dt, narrow, dev, "v")]
    if out is None:
        out = _like(q, stream)
    rows.append(_rows(out, dt, wide, dev, "out"))
    if lse is None:
        lse = _new(wide[:2], torch.float32, dev, stream)
    else:
        m8._need(lse, torch.float32, wide[:2], "lse")
        if lse.device != dev:
            raise ValueError(f"lse: expected on {dev}, got {lse.device}")
    with _on(dev):
        m8._check(lib.llmint8_attention(s, code, *rows, lse.data_ptr(), _handle(stream, dev)), "llmint8_attention")
    return out, lse


def llmint8_attention_backward_workspace_bytes(batch, q_heads, heads, dim) -> int:
    s = _SHAPE(batch.cu.data_ptr(), batch.seqs, batch.rows, q_heads, heads, dim, 1.0, 1, 0, 0)
    return int(_library().llmint8_attention_backward_workspace_bytes(s))


def llmint8_attention_backward(batch, q, k, v, out, lse, dout, scale=None, causal=True, window=0, sinks=0, dq=None,
                               dk=None, dv=None, workspace=None, stream=None):
    """(dq, dk, dv) of ``llmint8_attention`` for the gradient ``dout`` of ``out``, from its inputs and results."""
    lib = _library()
    dev, dt = batch.device, q.dtype
    s = _shape(batch, q, k, scale, causal, window, sinks)
    code = _half(dt)
    heads, dim, n = q.shape[1], q.shape[2], batch.rows
    wide, narrow = (n, heads, dim), (n, k.shape[1], dim)
    dq = _like(q, stream) if dq is None else dq
    dk = _like(k, stream) if dk is None else dk
    dv = _like(v, stream) if dv is None else dv
    m8._need(lse, torch.float32, wide[:2], "lse")
    if lse.device != dev:
        raise ValueError(f"lse: expected on {dev}, got {lse.device}")
    rows = (_rows(q, dt, wide, dev, "q"), _rows(k, dt, narrow, dev, "k"), _rows(v, dt, narrow, dev, "v"),
            _rows(out, dt, wide, dev, "out"))
    more = (_rows(dout, dt, wide, dev, "dout"), _rows(dq, dt, wide, dev, "dq"), _rows(dk, dt, narrow, dev, "dk"),
            _rows(dv, dt, narrow, dev, "dv"))
    if workspace is None:
        workspace = _new((max(1, 8 * n * heads),), torch.uint8, dev, stream)
    else:
        m8._need_workspace(workspace, dev)
    with _on(dev):
        m8._check(lib.llmint8_attention_backward(s, code, *rows, lse.data_ptr(), *more, workspace.data_ptr(),
                                                 m8._ws_bytes(workspace), _handle(stream, dev)),
                  "llmint8_attention_backward")
    return dq, dk, dv


# ---- rotary positions with axes


def rope_axes(sections, turns=False):
    """The axis of every pair (a list for ``llmint8_rope``) where ``sections[a]`` pairs follow axis a: one section
    after the other, or in turns (pair 0 axis 0, pair 1 axis 1, ..., for as long as a section has pairs left)."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0 or sum(left) < 1 or len(left) > 8:
        raise ValueError(f"sections: expected 1 to 8 numbers of pairs, got {sections}")
    if not turns:
        return [a for a, n in enumerate(left) for _ in range(n)]
    axis = []
    while sum(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                axis.append(a)
    return axis


def llmint8_rope(table, pos, axis, q, k=None, interleaved=False, inverse=False, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): q [rows, heads, dim] and, if given, k [rows, k_heads, dim] (fp16 or bf16) with their first
    ``rot`` channels turned: pair i by row ``pos[row, axis[i]]`` of ``table`` (fp32 [positions, rot], from
    ``llmint8_rope_table``). ``pos`` int32 [rows, axes] or [rows]; ``axis``: the axis of every pair
    (``rope_axes``), a list or bytes. ``inverse`` turns back, which is the gradient. The outputs are new by default;
    they may be the inputs."""
    lib = _library()
    _plain((q, k), "q and k", "rotary")
    dev, dt = q.device, q.dtype
    code = _half(dt)
    if q.dim() != 3 or not q.is_cuda or (k is not None and k.dim() != 3):
        raise ValueError(f"q and k: expected CUDA [rows, heads, dim], got {tuple(q.shape)} on {q.device}")
    n, heads, dim = q.shape
    if (table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous() or table.device != dev):
        raise ValueError(f"table: expected contiguous fp32 [positions, rot] on {dev}, got {table.dtype} "
                         f"{tuple(table.shape)} on {table.device}")
    if pos.dim() not in (1, 2) or pos.shape[0] != n or pos.dtype != torch.int32 or not pos.is_contiguous() or pos.device != dev:
        raise ValueError(f"pos: expected contiguous int32 [{n}, axes] on {dev}, got {pos.dtype} {tuple(pos.shape)} on "
                         f"{pos.device}")
    rot, axes = table.shape[1], 1 if pos.dim() == 1 else pos.shape[1]
    axis = bytes(axis)
    if 2 * len(axis) != rot:
        raise ValueError(f"axis: expected one for each of {rot // 2} pairs, got {len(axis)}")
    q_out = _like(q, stream) if q_out is None else q_out
    xr, yr = _rows(q, dt, q.shape, dev, "q"), _rows(q_out, dt, q.shape, dev, "q_out")
    x2 = y2 = None
    heads2 = 0
    if k is not None:
        heads2 = k.shape[1]
        shape = (n, heads2, dim)
        k_out = _like(k, stream) if k_out is None else k_out
        x2, y2 = _rows(k, dt, shape, dev, "k"), _rows(k_out, dt, shape, dev, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    with _on(dev):
        m8._check(lib.llmint8_rope(code, xr, yr, heads, x2, y2, heads2, n, dim, pos.data_ptr(), axes, axis,
                                   table.data_ptr(), table.shape[0], rot, 1 if interleaved else 0,
                                   1 if inverse else 0, _handle(stream, dev)), "llmint8_rope")
    return q_out, k_out


# ---- layer norm


def _norm_rows(t, dtype, shape, device, name):
    if t.dtype != dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    if t.stride(1) != 1 and shape[1] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the channels must be dense, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0)


def _norm_weight(w, K, dtype, w_dtype, device, name):
    if w is None:
        return None
    if w.dtype != w_dtype or w_dtype not in (dtype, torch.float32) or w.shape != (K,) or not w.is_contiguous() \
            or w.device != device:
        raise ValueError(f"{name}: expected contiguous [{K}] of {dtype} or fp32 on {device} (weight and bias alike), "
                         f"got {w.dtype} {tuple(w.shape)} on {w.device}")
    return w.data_ptr()


def llmint8_layer_norm(x, weight=None, bias=None, eps=1e-5, y=None, stats=True, stream=None):
    """(y, stats): layer norm of x [rows, K] (fp16, bf16 or fp32). weight and bias [K] are of x's type or fp32, or
    None. stats fp32 [rows, 2] (what the backward call reads) is new, a tensor of the caller's, or None with
    ``stats=False``."""
    lib = _library()
    _plain((x, weight, bias), "x, weight and bias", "layer_norm")
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"x: expected CUDA [rows, K], got {tuple(x.shape)} on {x.device}")
    n, K = x.shape
    dev, dt = x.device, x.dtype
    code = _dtype(dt, "x")
    w_dtype = weight.dtype if weight is not None else bias.dtype if bias is not None else dt
    w = _norm_weight(weight, K, dt, w_dtype, dev, "weight")
    b = _norm_weight(bias, K, dt, w_dtype, dev, "bias")
    y = _like(x, stream) if y is None else y
    xr, yr = _norm_rows(x, dt, (n, K), dev, "x"), _norm_rows(y, dt, (n, K), dev, "y")
    if stats is True:
        stats = _new((n, 2), torch.float32, dev, stream)
    elif stats is False:
        stats = None
    else:
        m8._need(stats, torch.float32, (n, 2), "stats")
        if stats.device != dev:
            raise ValueError(f"stats: expected on {dev}, got {stats.device}")
    with _on(dev):
        m8._check(lib.llmint8_layer_norm(*xr, code, n, K, w, b, _dtype(w_dtype, "weight"), float(eps), *yr,
                                         None if stats is None else stats.data_ptr(), _handle(stream, dev)),
                  "llmint8_layer_norm")
    return y, stats


def llmint8_layer_norm_workspace_bytes(rows: int, K: int) -> int:
    return int(_library().llmint8_layer_norm_workspace_bytes(rows, K))


def llmint8_layer_norm_backward(dy, x, stats, weight=None, dx=None, dw=None, db=None, sums=None, workspace=None,
                                stream=None):
    """(dx, dw, db) of ``llmint8_layer_norm`` for the gradient ``dy`` of y, from x and its stats. dw and db take
    the weight's type; they are formed where there is a weight, or as ``sums`` says."""
    lib = _library()
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"x: expected CUDA [rows, K], got {tuple(x.shape)} on {x.device}")
    n, K = x.shape
    dev, dt = x.device, x.dtype
    code = _dtype(dt, "x")
    given = next((t for t in (weight, dw, db) if t is not None), None)
    w_dtype = dt if given is None else given.dtype
    if sums is None:
        sums = given is not None
    if sums:
        dw = _new((K,), w_dtype, dev, stream) if dw is None else dw
        db = _new((K,), w_dtype, dev, stream) if db is None else db
    w = _norm_weight(weight, K, dt, w_dtype, dev, "weight")
    wr, br = _norm_weight(dw, K, dt, w_dtype, dev, "dw"), _norm_weight(db, K, dt, w_dtype, dev, "db")
    dx = _like(x, stream) if dx is None else dx
    m8._need(stats, torch.float32, (n, 2), "stats")
    if stats.device != dev:
        raise ValueError(f"stats: expected on {dev}, got {stats.device}")
    gr, xr = _norm_rows(dy, dt, (n, K), dev, "dy"), _norm_rows(x, dt, (n, K), dev, "x")
    dr = _norm_rows(dx, dt, (n, K), dev, "dx")
    if workspace is not None:
        m8._need_workspace(workspace, dev)
    with _on(dev):
        if workspace is None and (wr or br):
            workspace = _new((lib.llmint8_layer_norm_workspace_bytes(n, K),), torch.uint8, dev, stream)
        m8._check(lib.llmint8_layer_norm_backward(*gr, *xr, code, n, K, w, _dtype(w_dtype, "weight"), stats.data_ptr(),
                                                  *dr, wr, br, m8._ptr(workspace), m8._ws_bytes(workspace),
                                                  _handle(stream, dev)), "llmint8_layer_norm_backward")
    return dx, dw, db


# ---- the gradients' norm


class GradientSet:
    """Gradients of a model as ``llmint8_grad_norm`` and ``llmint8_grad_clip`` take them: dense tensors (fp16, bf16
    or fp32) on one device, and where to write them clipped: themselves, or ``out``, of their types or fp32. The set
    holds the tensors; their values may change between calls, and their memory and types too (``Module.half()`` gives
    the gradients of a model others): every call looks at them again. A program whose gradients are the same tensors
    in every step makes it once."""

    __slots__ = ("_grads", "_out", "device", "_arr", "_need", "_both", "_seen")

    def __init__(self, grads, out=None):
        _library()
        self._grads = tuple(g for g in grads if g is not None)
        self._out = self._grads if out is None else tuple(out)
        self._read()

    grads = property(lambda self: self._grads, doc="The gradients, those that were None left out.")
    out = property(lambda self: self._out, doc="The tensors that are written.")

    def _read(self):
        """The tensors' memory, as the library takes it, and what it was read from."""
        if len(self.out) != len(self.grads):
            raise ValueError(f"out: {len(self.out)} tensors for {len(self.grads)} gradients")
        self._seen, self._both = None, ((), None)
        self.device = self.grads[0].device if self.grads else None
        self._arr = (_Grad * max(1, len(self.grads)))()
        for a, g, o in zip(self._arr, self.grads, self.out):
            for t in (g, o):
                if t.device != self.device or not t.is_cuda or not _dense(t):
                    raise ValueError(f"gradients: expected dense CUDA tensors on {self.device}, got {tuple(t.shape)} "
                                     f"with strides {t.stride()} on {t.device}")
            if g is not o and (o.shape != g.shape or o.stride() != g.stride() and not (
                    g.is_contiguous() and o.is_contiguous())):
                raise ValueError(f"out: expected {tuple(g.shape)} with strides {g.stride()}, got {tuple(o.shape)} "
                                 f"with {o.stride()}")
            code, to = _dtype(g.dtype, "gradients"), _dtype(o.dtype, "out")
            if to not in (code, m8.LLMINT8_DTYPE_F32):
                raise ValueError(f"out: {g.dtype} or fp32, got {o.dtype}")
            a.data, a.out, a.n, a.dtype, a.out_dtype = g.data_ptr(), o.data_ptr(), g.numel(), code, to
        self._need = None
        # what is written is nobody else's: a tensor that is there twice would be scaled twice, or not
        spans = []
        for g, o in zip(self.grads, self.out):
            spans.append((o.data_ptr(), o.data_ptr() + o.numel() * o.element_size(), True))
            if g.data_ptr() != o.data_ptr() or g.dtype != o.dtype:
                spans.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), False))
        end = [0, 0]  # of what was written so far, and of what was only read
        for first, last, written in sorted(spans):
            if first < last:
                if first < end[1] or (written and first < end[0]):
                    raise ValueError("gradients: two of them, or two outputs, share memory that is written")
                end[1 if written else 0] = max(end[1 if written else 0], last)
        both = self.grads if self.out is self.grads else self.grads + self.out
        self._both = both, None
        if _describe() is not None:
            held, seen = (ctypes.py_object * max(1, len(both)))(*both), ctypes.create_string_buffer(32 * max(1, len(both)))
            if _tensors(held, len(both), seen, 1) == 0:
                self._both, self._seen = (both, held), seen
                return
        self._seen = _looks(both)

    def _current(self):
        """The set, read again if a tensor is not as it was: an address of before may be another tensor's by now."""
        both, held = self._both
        if self._seen is None:
            same = False
        elif held is not None:
            same = _tensors(held, len(both), self._seen, 0) == 1
        else:
            same = _looks(both) == self._seen
        if not same:
            self._read()
        return self

    def __len__(self):
        return len(self.grads)

    def workspace_bytes(self) -> int:
        self._current()
        return self._bytes()

    def _bytes(self):
        if self._need is None:
            self._need = int(_library().llmint8_grad_norm_workspace_bytes(self._arr, len(self)))
        return self._need


def _looks(tensors):
    """Address, count and type of every tensor. One list after the other: 0.12 us a tensor, a loop over the tensors takes
    half as much again."""
    return (list(map(torch.Tensor.data_ptr, tensors)), list(map(torch.Tensor.numel, tensors)), [t.dtype for t in tensors])


_TABLE = False  # not asked for yet


def _describe():
    """(llmint8_py_tensors, the exchange table of torch's tensors), which looks at them in a tenth of the time; None
    where this torch has no such table."""
    global _TABLE
    if _TABLE is False:
        try:
            get = ctypes.pythonapi.PyCapsule_GetPointer
            get.argtypes, get.restype = [ctypes.py_object, ctypes.c_char_p], _vp
            fn = ctypes.PyDLL(m8.library_path()).llmint8_py_tensors
            fn.argtypes, fn.restype = [_vp, _vp, _i64, _vp, ctypes.c_int], ctypes.c_int
            _TABLE = fn, get(torch.Tensor.__dlpack_c_exchange_api__, b"dlpack_exchange_api")
        except (AttributeError, OSError, ValueError):
            _TABLE = None
    return _TABLE


def _tensors(held, n, seen, write):
    fn, table = _TABLE
    try:
        return fn(table, held, n, seen, write)
    except Exception:  # a tensor that the table does not describe
        return -1


def _dense(t):
    """All of a tensor's memory is its own values, in whatever order of the axes."""
    if t.is_contiguous():
        return True
    n = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda x: x[1]):
        if size != 1 and stride != n:
            return False
        n *= size
    return True


def _set(grads):
    return grads._current() if isinstance(grads, GradientSet) else GradientSet(grads)


def llmint8_grad_norm(grads, scale=1.0, norm=None, workspace=None, device=None, stream=None):
    """fp32 scalar on the device: ``scale`` times the root of the sum of all squares of ``grads`` (a GradientSet, or
    a list of tensors, None among them left out). ``device`` is needed where there are none."""
    return _grad_norm(_set(grads), scale, norm, workspace, device, stream)


def _grad_norm(grads, scale, norm=None, workspace=None, device=None, stream=None):
    lib = _library()
    dev = grads.device or torch.device(device or "cuda")
    if norm is None:
        norm = _new((), torch.float32, dev, stream)
    else:
        m8._need(norm, torch.float32, (), "norm")
    dev = norm.device
    if grads.device not in (None, dev):
        raise ValueError(f"norm: expected on {grads.device}, got {dev}")
    if workspace is None:
        workspace = _new((grads._bytes(),), torch.uint8, dev, stream)
    else:
        m8._need_workspace(workspace, dev)
    with _on(dev):
        m8._check(lib.llmint8_grad_norm(grads._arr, len(grads), float(scale), norm.data_ptr(), workspace.data_ptr(),
                                        m8._ws_bytes(workspace), _handle(stream, dev)), "llmint8_grad_norm")
    return norm


def llmint8_grad_clip(grads, norm, max_norm, scale=1.0, stream=None):
    """The gradients times scale min(1, max_norm / (norm + 1e-6)), written where the set says (in place for a list
    of tensors); ``norm`` is an fp32 scalar on the device (from ``llmint8_grad_norm``). Returns the tensors
    written."""
    return _grad_clip(_set(grads), norm, max_norm, scale, stream)


def _grad_clip(grads, norm, max_norm, scale, stream=None):
    lib = _library()
    m8._need(norm, torch.float32, (), "norm")
    if grads.device not in (None, norm.device):
        raise ValueError(f"norm: expected on {grads.device}, got {norm.device}")
    with _on(norm.device):
        m8._check(lib.llmint8_grad_clip(grads._arr, len(grads), norm.data_ptr(), float(max_norm), float(scale),
                                        _handle(stream, norm.device)), "llmint8_grad_clip")
    return list(grads.out)


def clip_grad_norm(parameters, max_norm, scale=1.0):
    """Clips the gradients of ``parameters`` (tensors, or one; those without one are left out) in place, so that their norm
    is at most ``max_norm``; ``scale`` (1 / loss scale) is applied first. Returns the norm before clipping, an fp32
    scalar on the device."""
    _library()
    # a tensor is its own only parameter: as a list it would be its rows, which have no gradient
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = GradientSet([p.grad for p in parameters])
    if not len(grads):
        return torch.zeros((), dtype=torch.float32, device=parameters[0].device if parameters else "cuda")
    norm = _grad_norm(grads, scale)
    _grad_clip(grads, norm, max_norm, scale)
    return norm


# ---- differentiable functions


def _unused(t, batch):
    """A new output of a packed call: rows of no sequence are zeros, as the kernels leave them alone."""
    used = batch.used_rows()
    if used is None:
        t.zero_()
    elif used < batch.rows:
        t[used:].zero_()
    return t


def _empty_rows(shape, like, batch):
    return _unused(torch.empty(shape, dtype=like.dtype, device=like.device), batch)


def _functions():
    _library()

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, batch, how):
            q, k, v = _fit(q), _fit(k), _fit(v)
            out, lse = llmint8_attention(batch, q, k, v, out=_empty_rows(q.shape, q, batch), **how)
            # cu among them, so that a backward pass after a change of cu is an error
            ctx.save_for_backward(q, k, v, out, lse, batch.cu)
            ctx.batch, ctx.how = batch, how
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            q, k, v, out, lse, _ = ctx.saved_tensors
            b = ctx.batch
            grads = [_empty_rows(t.shape, t, b) for t in (q, k, v)]
            return (*llmint8_attention_backward(b, q, k, v, out, lse, _fit(dout), dq=grads[0], dk=grads[1], dv=grads[2],
                                                **ctx.how), None, None)

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, table, pos, axis, interleaved):
            ctx.save_for_backward(table, pos)
            ctx.how = axis, interleaved
            return llmint8_rope(table, pos, axis, _dense_channels(q), None if k is None else _dense_channels(k),
                                interleaved)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq, dk):
            table, pos = ctx.saved_tensors
            axis, interleaved = ctx.how
            return (*llmint8_rope(table, pos, axis, _dense_channels(dq), None if dk is None else _dense_channels(dk),
                                  interleaved, inverse=True), None, None, None, None)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, eps):
            y, stats = llmint8_layer_norm(x, weight, bias, eps)
            ctx.save_for_backward(x, stats, weight)
            ctx.w_dtype = weight.dtype if weight is not None else bias.dtype if bias is not None else x.dtype
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, stats, weight = ctx.saved_tensors
            K = x.shape[1]
            dw, db = (torch.empty((K,), dtype=ctx.w_dtype, device=x.device) if need else None
                      for need in ctx.needs_input_grad[1:3])
            dx, dw, db = llmint8_layer_norm_backward(_dense_channels(dy), x, stats, weight, dw=dw, db=db, sums=False)
            return dx, dw, db, None

    class QKV(torch.autograd.Function):
        """Attention from the output of a fused q, k, v projection [rows, q_heads + 2 heads, dim], turned in it;
        one gradient for all of it."""

        @staticmethod
        def forward(ctx, qkv, heads, rope, batch, how):
            nq, qkv = qkv.shape[1] - 2 * heads, _fit(qkv)
            if rope is not None:
                table, pos, axis, interleaved = rope
                turned, _ = llmint8_rope(table, pos, axis, qkv[:, :nq + heads], None, interleaved)
                q, k = turned[:, :nq], turned[:, nq:]
            else:
                q, k = qkv[:, :nq], qkv[:, nq:nq + heads]
            v = qkv[:, nq + heads:]
            out, lse = llmint8_attention(batch, q, k, v, out=_empty_rows(q.shape, q, batch), **how)
            ctx.save_for_backward(q, k, v, out, lse, batch.cu, *(rope[:2] if rope is not None else ()))
            ctx.batch, ctx.how, ctx.rope = batch, how, None if rope is None else rope[2:]
            return out

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dout):
            q, k, v, out, lse, _ = ctx.saved_tensors[:6]
            nq, n, b = q.shape[1], k.shape[1], ctx.batch
            d = _empty_rows((q.shape[0], nq + 2 * n, q.shape[2]), q, b)
            llmint8_attention_backward(b, q, k, v, out, lse, _fit(dout), dq=d[:, :nq], dk=d[:, nq:nq + n],
                                       dv=d[:, nq + n:], **ctx.how)
            if ctx.rope is not None:
                table, pos = ctx.saved_tensors[6:]
                part = d[:, :nq + n]
                llmint8_rope(table, pos, ctx.rope[0], part, None, ctx.rope[1], inverse=True, q_out=part)
            return d, None, None, None, None

    return {"attention": Attention, "rotary": Rotary, "norm": Norm, "qkv": QKV}


def _dense_channels(t):
    """A tensor as the kernels take it: inputs may be, and autograd hands on, expanded and strided ones."""
    strides = t.stride()
    return t if strides[-1] == 1 and 0 not in strides[:-1] and all(
        s >= t.shape[-1] for s in strides[:-1]) else t.contiguous()


def _fit(t):
    """_dense_channels, in 16-byte pieces as attention reads them."""
    t = _dense_channels(t)
    fine = t.data_ptr() % 16 == 0 and all(s % 8 == 0 for s in t.stride()[:-1])
    # a copy even of a contiguous tensor that only begins at an odd place, as slices of a flat one do: contiguous()
    # would hand back the tensor itself
    return t if fine else t.clone(memory_format=torch.contiguous_format)


_FN = None


def _fn(name):
    global _FN
    if _FN is None:
        _FN = _functions()
    return _FN[name].apply


def packed_attention(q, k, v, batch, scale=None, causal=True, window=0, sinks=0):
    """``llmint8_attention`` with gradients for q, k and v. Rows of no sequence are zeros, in the output and in the
    gradients."""
    how = {"scale": scale, "causal": causal, "window": window, "sinks": sinks}
    return _fn("attention")(q, k, v, batch, how)


def qkv_attention(qkv, heads, batch, rope=None, scale=None, causal=True, window=0, sinks=0):
    """``packed_attention`` of a fused projection's output [rows, q_heads + 2 heads, dim] (q, k, v side by side), its q
    and k turned by ``rope`` = (table, pos, axis, interleaved) first, with one gradient for all of qkv: the slices'
    gradients are written side by side, where separate functions would each give one of qkv's size, to be added."""
    how = {"scale": scale, "causal": causal, "window": window, "sinks": sinks}
    return _fn("qkv")(qkv, heads, rope, batch, how)


def rotary(q, k, table, pos, axis, interleaved=False):
    """(q, k) turned by ``llmint8_rope``, with gradients; k may be None."""
    return _fn("rotary")(q, k, table, pos, bytes(axis), interleaved)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """``llmint8_layer_norm`` over the last axis of x, with gradients for x, weight and bias."""
    shape = x.shape
    x2 = x.reshape(-1, shape[-1])
    return _fn("norm")(_dense_channels(x2), weight, bias, float(eps)).reshape(shape)


class LayerNorm:
    """Layer norm with a weight and bias that may be trained (tensors of the inputs' type or fp32; the bias, or
    both, may be None)."""

    def __init__(self, weight=None, bias=None, eps: float = 1e-5):
        self.weight, self.bias, self.eps = weight, bias, float(eps)

    def parameters(self):
        return [t for t in (self.weight, self.bias) if t is not None]

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)

    __call__ = forward
