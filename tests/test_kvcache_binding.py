"""Refusals of the key/value cache's Python calls that need no GPU (the library is a stand-in)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402


class _Library:
    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def setup(monkeypatch):
    monkeypatch.setattr(m8, "load_library", _Library)
    monkeypatch.setattr(m8, "_need", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 0}))
    z = lambda shape, t: torch.zeros(shape, dtype=t)  # noqa: E731
    c = m8.KVCache(z((3, 2, 16, 32), torch.int8), z((3, 2, 32, 16), torch.int8), z((3, 2), torch.float32),
                   z((3, 2), torch.float32))
    b = m8.KVBatch(z((2,), torch.int32), z((1,), torch.int32), z((1, 3), torch.int32), 4)
    return c, b, torch.zeros((4, 2, 32), dtype=torch.float16)


def test_tensors_that_require_a_gradient_are_refused(setup):
    c, b, x = setup
    g = torch.zeros_like(x).requires_grad_()
    calls = [lambda t: m8.llmint8_kv_append(c, b, t, x), lambda t: m8.llmint8_kv_append(c, b, x, t),
             lambda t: m8.llmint8_kv_append(c, b, x, x, q=t), lambda t: m8.llmint8_kv_append(c, b, x, x, q=x, q_out=t),
             lambda t: m8.llmint8_kv_attention(c, b, t), lambda t: m8.llmint8_kv_attention(c, b, x, out=t),
             lambda t: m8.llmint8_kv_gather(c, b, k=t), lambda t: m8.llmint8_kv_gather(c, b, v=t)]
    for call in calls:
        call(x)
        with pytest.raises(ValueError, match="gradient"):
            call(g)
        with pytest.raises(ValueError, match="gradient"):
            call(g * 2)  # not a leaf
        with torch.no_grad():
            call(g)
        call(g.detach())
