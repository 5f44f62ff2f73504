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
