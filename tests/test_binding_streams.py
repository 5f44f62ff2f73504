"""Where the binding's calls take memory from when they are given a stream (CPU: the library and torch's streams
are stand-ins)."""
from __future__ import annotations

import contextlib

import pytest

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Library:
    """Every call succeeds; every size is 4096."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith(("bytes", "bytes_path")) else 0


@pytest.fixture
def watch(monkeypatch):
    """(the call's stream, [(stream that an allocation was made on, tensor)], {id of a tensor: streams recorded})"""
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
    args = _arguments()
    for name in ("empty", "zeros", "full", "empty_like"):
        monkeypatch.setattr(torch, name, make(getattr(torch, name)))
    return current, side, made, used, args


def _arguments():
    h, i8, f, i = torch.float16, torch.int8, torch.float32, torch.int32
    z = lambda shape, t: torch.zeros(shape, dtype=t)  # noqa: E731
    return dict(X=z((4, 32), h), Wq=z((16, 32), i8), sW=z((16,), f), dY=z((4, 16), h), W=z((16, 32), h),
                q8=z((64,), i8), a8=z((1,), f), q4=z((256,), torch.uint8), a4=z((8,), f),
                cache=(z((3, 2, 16, 32), i8), z((3, 2, 32, 16), i8), z((3, 2), f), z((3, 2), f)),
                batch=(z((2,), i), z((1,), i), z((1, 3), i)), k=z((4, 2, 32), h))


def _kv(a):
    return m8.KVCache(*a["cache"]), m8.KVBatch(*a["batch"], 4)


CALLS = {
    "quantize_weight": lambda a, s: m8.llmint8_quantize_weight(a["W"], stream=s),
    "quantize_weight_ex": lambda a, s: m8.llmint8_quantize_weight_ex(a["W"], stream=s),
    "linear": lambda a, s: m8.llmint8_linear(a["X"], a["Wq"], a["sW"], stream=s),
    "linear_ex": lambda a, s: m8.llmint8_linear_ex(a["X"], a["Wq"], a["sW"], stream=s),
    "linear_noalloc": lambda a, s: m8.llmint8_linear_noalloc(a["X"], a["Wq"], a["sW"], stream=s),
    "linear_timed": lambda a, s: m8.llmint8_linear_timed(a["X"], a["Wq"], a["sW"], 6.0, None, None, [], stream=s),
    "linear_timed_ex": lambda a, s: m8.llmint8_linear_timed_ex(a["X"], a["Wq"], a["sW"], 6.0, None, None, [], stream=s),
    "linear_debug": lambda a, s: m8.llmint8_linear_debug(a["X"], a["Wq"], a["sW"], stream=s),
    "linear_debug_ex": lambda a, s: m8.llmint8_linear_debug_ex(a["X"], a["Wq"], a["sW"], stream=s),
    "dequantize_weight_t": lambda a, s: m8.llmint8_dequantize_weight_t(a["Wq"], a["sW"], stream=s),
    "dequantize_weight_t_ex": lambda a, s: m8.llmint8_dequantize_weight_t_ex(a["Wq"], a["sW"], stream=s),
    "backward": lambda a, s: m8.llmint8_linear_backward_input(a["dY"], a["Wq"], a["sW"], stream=s),
    "backward_ex": lambda a, s: m8.llmint8_linear_backward_input_ex(a["dY"], a["Wq"], a["sW"], stream=s),
    "backward_timed": lambda a, s: m8.llmint8_linear_backward_input_timed(a["dY"], a["Wq"], a["sW"], [], stream=s),
    "quantize_blockwise": lambda a, s: m8.llmint8_quantize_blockwise(a["W"], stream=s),
    "dequantize_blockwise": lambda a, s: m8.llmint8_dequantize_blockwise(a["q8"], a["a8"], stream=s),
    "quantize_4bit": lambda a, s: m8.llmint8_quantize_4bit(a["W"], stream=s),
    "dequantize_4bit": lambda a, s: m8.llmint8_dequantize_4bit(a["q4"], a["a4"], stream=s),
    "linear_4bit": lambda a, s: m8.llmint8_linear_4bit(a["X"], a["q4"], a["a4"], 16, stream=s),
    "rope_table": lambda a, s: m8.llmint8_rope_table([1.0, 0.5], 7, device="cpu", stream=s),
    "kv_append": lambda a, s: m8.llmint8_kv_append(*_kv(a), a["k"], a["k"], q=a["k"], stream=s),
    "kv_gather": lambda a, s: m8.llmint8_kv_gather(*_kv(a), stream=s),
    "kv_attention": lambda a, s: m8.llmint8_kv_attention(*_kv(a), a["k"], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_is_its_stream_s(watch, name):
    """A workspace of the current stream's pool goes back to the current stream when the call returns, while the
    call's own stream may still be writing to it."""
    current, side, made, used, args = watch
    CALLS[name](args, side)
    assert made
    for stream, t in made:
        assert stream is side
        assert used.get(id(t)) == [current]  # and the current stream may read it


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_the_current_stream(watch, name):
    current, _, made, used, args = watch
    for stream in (None, current):
        CALLS[name](args, stream)
    assert made and not used and all(stream is current for stream, _ in made)


WITH_WORKSPACE = {
    "linear": lambda a, w: m8.llmint8_linear(a["X"], a["Wq"], a["sW"], workspace=w),
    "linear_ex": lambda a, w: m8.llmint8_linear_ex(a["X"], a["Wq"], a["sW"], workspace=w),
    "linear_debug": lambda a, w: m8.llmint8_linear_debug(a["X"], a["Wq"], a["sW"], workspace=w),
    "linear_timed": lambda a, w: m8.llmint8_linear_timed(a["X"], a["Wq"], a["sW"], 6.0, None, w, []),
    "backward": lambda a, w: m8.llmint8_linear_backward_input(a["dY"], a["Wq"], a["sW"], workspace=w),
    "backward_ex": lambda a, w: m8.llmint8_linear_backward_input_ex(a["dY"], a["Wq"], a["sW"], workspace=w),
    "kv_attention": lambda a, w: m8.llmint8_kv_attention(*_kv(a), a["k"], workspace=w),
}


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces_that_are_not_the_call_s_memory_are_refused(watch, name):
    """Of another device, or with holes: the kernels would work in memory that is not the tensor's."""
    args = watch[-1]
    call = WITH_WORKSPACE[name]
    call(args, torch.zeros((4096,), dtype=torch.uint8))
    for bad in (torch.zeros((4096,), dtype=torch.uint8, device="meta"), torch.zeros((8192,), dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(args, bad)


def test_lse_of_another_device_is_refused(watch):
    a = watch[-1]
    m8.llmint8_kv_attention(*_kv(a), a["k"], lse=torch.zeros((4, 2)))
    with pytest.raises(ValueError, match="lse"):
        m8.llmint8_kv_attention(*_kv(a), a["k"], lse=torch.zeros((4, 2), device="meta"))
