"""The training operators' Python calls without a GPU (the library is a stand-in): refusals, where memory comes from,
and what the bookkeeping says."""
from __future__ import annotations

import contextlib
import ctypes

import pytest

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402
from mixed_precision_int8_amd import training  # noqa: E402

H, F = torch.float16, torch.float32


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Library:
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("bytes") else 0


@pytest.fixture
def setup(monkeypatch):
    """(the call's stream, [(stream of an allocation, tensor)], {id of a tensor: streams recorded})"""
    training._library()
    current, side = _Stream(11), _Stream(22)
    stack, made, used = [current], [], {}

    @contextlib.contextmanager
    def on(stream):
        stack.append(stream)
        yield
        stack.pop()

    def make(fn):
        def call(*a, **kw):
            t = fn(*a, **kw)
            made.append((stack[-1], t))
            return t
        return call

    monkeypatch.setattr(m8, "load_library", _Library)
    monkeypatch.setattr(m8, "_need", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stack[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: used.setdefault(id(t), []).append(s))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    args = dict(b=m8.PackedRows(torch.zeros(3, dtype=torch.int32), 6), q=torch.zeros((6, 4, 16), dtype=H),
                k=torch.zeros((6, 2, 16), dtype=H), lse=torch.zeros((6, 4)), table=torch.zeros((9, 16)),
                pos=torch.zeros((6, 2), dtype=torch.int32), x=torch.zeros((6, 24), dtype=H), w=torch.zeros(24, dtype=H),
                stats=torch.zeros((6, 2)), norm=torch.zeros(()))
    for name in ("empty", "zeros", "full", "empty_like"):
        monkeypatch.setattr(torch, name, make(getattr(torch, name)))
    return current, side, made, used, args


AXIS = [0, 1] * 4
CALLS = {
    "attention": lambda a, **kw: m8.llmint8_attention(a["b"], a["q"], a["k"], a["k"], **kw),
    "attention_backward": lambda a, **kw: m8.llmint8_attention_backward(
        a["b"], a["q"], a["k"], a["k"], a["q"], a["lse"], a["q"], **kw),
    "rope": lambda a, **kw: m8.llmint8_rope(a["table"], a["pos"], AXIS, a["q"], a["k"], **kw),
    "layer_norm": lambda a, **kw: m8.llmint8_layer_norm(a["x"], a["w"], a["w"], **kw),
    "layer_norm_backward": lambda a, **kw: m8.llmint8_layer_norm_backward(a["x"], a["x"], a["stats"], a["w"], **kw),
    "grad_norm": lambda a, **kw: m8.llmint8_grad_norm([a["x"]], **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_is_its_stream_s(setup, name):
    current, side, made, used, args = setup
    CALLS[name](args, stream=side)
    assert made
    for stream, t in made:
        assert stream is side and used.get(id(t)) == [current]


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_the_current_stream(setup, name):
    current, _, made, used, args = setup
    for stream in (None, current):
        CALLS[name](args, stream=stream)
    assert made and not used and all(stream is current for stream, _ in made)


@pytest.mark.parametrize("name", ["attention_backward", "layer_norm_backward", "grad_norm"])
def test_workspaces_that_are_not_the_call_s_memory_are_refused(setup, name):
    args = setup[-1]
    CALLS[name](args, workspace=torch.zeros(4096, dtype=torch.uint8))
    for bad in (torch.zeros(4096, dtype=torch.uint8, device="meta"), torch.zeros(8192, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            CALLS[name](args, workspace=bad)


def test_tensors_that_require_a_gradient_are_refused(setup):
    a = setup[-1]
    q = torch.zeros((6, 4, 16), dtype=H).requires_grad_()
    w = torch.zeros(24, dtype=H).requires_grad_()
    for call in (lambda: m8.llmint8_attention(a["b"], q, a["k"], a["k"]),
                 lambda: m8.llmint8_rope(a["table"], a["pos"], AXIS, a["q"], q * 2),
                 lambda: m8.llmint8_layer_norm(a["x"], w), lambda: m8.llmint8_layer_norm(a["x"], a["w"], w)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()


def test_arguments_that_do_not_fit_are_refused(setup):
    a = setup[-1]
    b, q, k, x = a["b"], a["q"], a["k"], a["x"]
    bad = [
        lambda: m8.llmint8_attention(b, q[:5], k, k), lambda: m8.llmint8_attention(b, q, k.float(), k),
        lambda: m8.llmint8_attention(b, q.float(), k.float(), k.float()), lambda: m8.llmint8_attention(b, q, k, k[:, :1]),
        lambda: m8.llmint8_attention(b, q[0], k, k), lambda: m8.llmint8_attention(b, q, k, k, out=k),
        lambda: m8.llmint8_attention(b, q.transpose(1, 2).contiguous().transpose(1, 2), k, k),
        lambda: m8.llmint8_attention(b, q.to("meta"), k, k),
        lambda: m8.llmint8_attention(b, q, k, k, lse=torch.zeros((6, 4), device="meta")),
        lambda: m8.llmint8_attention_backward(b, q, k, k, q, a["lse"], k),
        lambda: m8.llmint8_attention_backward(b, q, k, k, q, a["lse"], q, dk=q),
        lambda: m8.llmint8_rope(a["table"], a["pos"], AXIS[:7], q), lambda: m8.llmint8_rope(a["table"], a["pos"][:5], AXIS, q),
        lambda: m8.llmint8_rope(a["table"], a["pos"].long(), AXIS, q), lambda: m8.llmint8_rope(a["table"].half(), a["pos"], AXIS, q),
        lambda: m8.llmint8_rope(a["table"], a["pos"], AXIS, q, k_out=q), lambda: m8.llmint8_rope(a["table"], a["pos"], AXIS, q[0]),
        lambda: m8.llmint8_rope(a["table"], a["pos"], AXIS, q.float()),
        lambda: m8.llmint8_layer_norm(x[0]), lambda: m8.llmint8_layer_norm(x.t()), lambda: m8.llmint8_layer_norm(x.double()),
        lambda: m8.llmint8_layer_norm(x, a["w"][:5]), lambda: m8.llmint8_layer_norm(x, a["w"].bfloat16()),
        lambda: m8.llmint8_layer_norm(x, a["w"], a["w"].float()), lambda: m8.llmint8_layer_norm(x, y=x.float()),
        lambda: m8.llmint8_layer_norm_backward(x.float(), x, a["stats"]),
        lambda: m8.llmint8_layer_norm_backward(x, x, a["stats"], a["w"], dw=a["w"].float()),
        lambda: m8.GradientSet([x.double()]), lambda: m8.GradientSet([x[:, ::2]]), lambda: m8.GradientSet([x], out=[]),
        lambda: m8.GradientSet([x], out=[x.bfloat16()]), lambda: m8.GradientSet([x, x.to("meta")]),
        lambda: m8.GradientSet([x], out=[x.t()]),
        lambda: m8.PackedRows(torch.zeros((2, 2), dtype=torch.int32), 3), lambda: m8.PackedRows(b.cu, -1),
        lambda: m8.PackedRows.of([3, -1], device="cpu"), lambda: m8.PackedRows.of([3, 4], rows=6, device="cpu"),
        lambda: m8.rope_axes([]), lambda: m8.rope_axes([0, 0]), lambda: m8.rope_axes([3, -1]), lambda: m8.rope_axes([1] * 9),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)


def test_gradients_that_share_memory_are_refused(setup):
    x = setup[-1]["x"]
    flat = torch.zeros(100)
    ok = m8.GradientSet([flat[:50], flat[50:], None, x, torch.zeros(0)])
    assert len(ok) == 4
    m8.GradientSet([x, x], out=[torch.zeros((6, 24)), torch.zeros((6, 24))])  # read twice, written apart
    out = torch.zeros((6, 24))
    for grads, outs in (([x, x], None), ([flat[:51], flat[50:]], None), ([x, x.clone()], [out, out]),
                        ([flat[:50], flat[50:]], [flat[50:], torch.zeros(50)]),
                        ([flat[:60]], [flat[40:]]), ([flat, flat[3:4]], None)):
        with pytest.raises(ValueError, match="share"):
            m8.GradientSet(grads, out=outs)


def test_structures_are_packed_as_the_header_declares_them():
    class Shape(ctypes.Structure):
        _fields_ = [("cu", ctypes.c_void_p), ("seqs", ctypes.c_int64), ("rows", ctypes.c_int64),
                    ("q_heads", ctypes.c_int64), ("heads", ctypes.c_int64), ("dim", ctypes.c_int64),
                    ("scale", ctypes.c_float), ("causal", ctypes.c_int), ("window", ctypes.c_int64),
                    ("sinks", ctypes.c_int64)]

    values = (1 << 46, 2, 3, 4, 5, 6, 0.5, 1, 8, 9)
    assert bytes(Shape(*values)) == training._SHAPE(*values)

    class Rows(ctypes.Structure):
        _fields_ = [("data", ctypes.c_void_p), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]

    assert bytes(Rows(1 << 46, 7, 8)) == training._ROWS(1 << 46, 7, 8)


def test_axes_of_pairs():
    assert m8.rope_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert m8.rope_axes([2, 1, 3], turns=True) == [0, 1, 2, 0, 2, 2]
    assert m8.rope_axes([4]) == [0] * 4 and m8.rope_axes([0, 2]) == [1, 1]


def test_positions_of_packed_rows():
    training._library()
    cu = torch.tensor([0, 3, 3, 7], dtype=torch.int32)
    b = m8.PackedRows.__new__(m8.PackedRows)
    b.cu, b.rows, b.device = cu, 9, cu.device
    assert b.positions().tolist()[:7] == [0, 1, 2, 0, 1, 2, 3] and b.positions().dtype == torch.int32


def test_tensors_are_made_to_fit():
    x = torch.zeros((6, 4, 16))
    for t in (x, x[:, 1:3], x[::2], x[..., :8]):
        assert training._dense_channels(t) is t
    for t in (x.transpose(1, 2), x[:1].expand(6, 4, 16), x[..., :1].expand(6, 4, 16), x[:, :1].expand(6, 4, 16)):
        assert training._dense_channels(t).is_contiguous()
    assert training._fit(x[..., 4:]).data_ptr() == x.data_ptr() + 16 and training._fit(x[:, :2]).data_ptr() == x.data_ptr()
    h = x.half()
    assert training._fit(h[..., 4:]).is_contiguous() and training._fit(h[..., 8:]).data_ptr() == h.data_ptr() + 16


def test_sequences_longer_than_the_table_are_refused():
    layer = object.__new__(m8.Int8SelfAttention)
    layer.rope, layer.axis, layer.norm = torch.zeros((100, 32)), None, None
    rows = object.__new__(m8.PackedRows)
    rows.max_len = 101
    with pytest.raises(ValueError, match="100 positions"):
        layer.packed(torch.zeros((101, 8)), rows)
    with pytest.raises(ValueError, match="pos"):
        layer.packed(torch.zeros((101, 8)), rows, torch.zeros((101, 1)))
