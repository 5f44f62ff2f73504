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


def test_positions_that_the_rope_table_has_no_row_for_are_refused(setup):
    c, _, _ = setup
    seqs = m8.PagedSequences(c)
    a, b = seqs.add(), seqs.add()
    x = torch.zeros((18, 2, 32), dtype=torch.float16)
    rope = torch.zeros((17, 32), dtype=torch.float32)
    m8.llmint8_kv_append(c, seqs.extend([a], [17]), x[:17], x[:17], rope=rope)
    with pytest.raises(ValueError, match="17 positions.*18"):
        m8.llmint8_kv_append(c, seqs.extend([a, b], [1, 2]), x[:3], x[:3], rope=rope)
    m8.llmint8_kv_append(c, seqs.extend([a, b], [0, 2]), x[:2], x[:2], rope=rope)  # only b has rows
    m8.llmint8_kv_append(c, seqs.extend([a], [1]), x[:1], x[:1])                    # nothing is rotated
    t = seqs.whole([a])
    m8.llmint8_kv_append(c, m8.KVBatch(t.cu, t.length, t.table, 19), torch.zeros((19, 2, 32)).half(),
                         torch.zeros((19, 2, 32)).half(), rope=rope)               # the host does not know
