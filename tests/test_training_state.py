"""What the training operators' binding keeps between calls, and what it makes of its inputs, without a GPU (the
library is a stand-in)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402
from mixed_precision_int8_amd import training  # noqa: E402


def test_a_contiguous_tensor_at_an_odd_place_is_copied():
    training._library()
    flat = torch.arange(8 + 6 * 4 * 16).half()
    for first in (1, 3):
        t = flat[first:first + 6 * 4 * 16].view(6, 4, 16)
        assert t.is_contiguous() and t.data_ptr() % 16 != 0
        fit = training._fit(t)
        assert fit.data_ptr() % 16 == 0 and fit.is_contiguous() and torch.equal(fit, t)
    # where the odd place comes from a gradient: that of a concatenation is a slice of the whole's
    aux, out = torch.zeros(3).half().requires_grad_(), torch.zeros((6, 4, 16)).half().requires_grad_()
    seen = []
    y = out * 1.0
    y.register_hook(seen.append)
    torch.cat([aux, y.flatten()]).backward(torch.ones(3 + y.numel()).half())
    assert seen[0].data_ptr() % 16 != 0 and training._fit(seen[0]).data_ptr() % 16 == 0
    even = flat[8:8 + 6 * 4 * 16].view(6, 4, 16)
    assert training._fit(even) is even


@pytest.fixture
def packed(monkeypatch):
    """PackedRows of memory that passes for a GPU's."""
    training._library()
    capturing = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))

    def filled(batch):
        """What an output's rows hold that no kernel wrote: memory comes as NaN."""
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", lambda shape, **kw: torch.full(shape, float("nan"), **kw))
            return training._empty_rows((batch.rows, 2), torch.zeros(0), batch)
    return filled, capturing


def test_rows_of_no_sequence_are_cleared_after_a_change_of_cu(packed):
    filled, capturing = packed
    b = m8.PackedRows.of([70, 50], rows=130, device="cpu")
    assert torch.isnan(filled(b)[:120]).all() and (filled(b)[120:] == 0).all()
    b.cu.copy_(torch.tensor([0, 30, 60], dtype=torch.int32))
    assert (filled(b)[60:] == 0).all()
    # a view of cu, and what cu is a view of, are cu
    for write in (lambda cu: cu[1:].sub_(1), lambda cu: cu.fill_(0)):
        base = torch.tensor([9, 0, 3, 5], dtype=torch.int32)
        b = m8.PackedRows(base[1:], 6, used=5)
        assert torch.isnan(filled(b)[:5]).all() and filled(b)[5:].tolist() == [[0, 0]]
        write(base)
        assert (filled(b) == 0).all()


def test_used_rows_of_a_captured_call_are_unknown(packed):
    filled, capturing = packed
    b = m8.PackedRows.of([3, 2], device="cpu")
    capturing.append(1)
    assert (filled(b) == 0).all()
    capturing.clear()
    assert torch.isnan(filled(b)).all()


def test_used_rows_in_inference_mode(packed):
    filled, _ = packed
    with torch.inference_mode():
        b = m8.PackedRows.of([3, 2], device="cpu")
        assert torch.isnan(filled(b)).all()
        b.cu.zero_()
        assert (filled(b) == 0).all()
        odd = m8.PackedRows(torch.tensor([0, 3, 5], dtype=torch.int32), 5, used=5)  # changes of which are not seen
        assert (filled(odd) == 0).all()


def test_used_rows_out_of_range(packed):
    cu = torch.tensor([0, 3, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="used"):
        m8.PackedRows(cu, 5, used=-1)
    assert m8.PackedRows(cu, 5, used=9).used_rows() == 5 and m8.PackedRows(cu, 5, used=0).used_rows() == 0


def test_the_longest_sequence_after_a_change_of_cu(packed):
    layer = object.__new__(m8.Int8SelfAttention)
    layer.rope, layer.axis, layer.norm = torch.zeros((100, 32)), None, None

    class Passed(Exception):
        pass

    def run(rows):
        def stop(X):
            raise Passed
        layer.qkv, layer.q_heads = stop, 4
        layer.packed(torch.zeros((rows.rows, 8)), rows)

    b = m8.PackedRows.of([60, 60], device="cpu")
    with pytest.raises(Passed):
        run(b)
    b.cu.copy_(torch.tensor([0, 110, 120], dtype=torch.int32))
    with pytest.raises(ValueError, match="max_len"):
        run(b)
    with pytest.raises(ValueError, match="max_len"):  # not known: up to 120
        run(m8.PackedRows(b.cu, 120))
    bound = m8.PackedRows(b.cu, 120, max_len=100)     # the caller's word, whatever cu holds
    b.cu.copy_(torch.tensor([0, 100, 120], dtype=torch.int32))
    for rows in (bound, m8.PackedRows(b.cu, 100), m8.PackedRows.of([], rows=300, device="cpu")):
        with pytest.raises(Passed):
            run(rows)
