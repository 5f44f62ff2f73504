"""Calls of the training operators whose memory or metadata changes between them, inputs at odd places, and what is not
finite where the formula gives it no weight."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import training_oracle as ref

torch = pytest.importorskip("torch")
import mixed_precision_int8_amd as m8  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


def randn(seed, *shape, dtype=torch.float16, scale=1.0):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * scale
    return torch.from_numpy(x).cuda().to(dtype)


def leaf(t):
    return t.detach().clone().requires_grad_()


def at_odd_place(t, first):
    flat = torch.empty(first + t.numel(), dtype=t.dtype, device=t.device)
    flat[first:] = t.flatten()
    return flat[first:].view(t.shape)


@pytest.mark.parametrize("first", [1, 3, 4])
def test_attention_takes_tensors_that_begin_at_an_odd_place(first):
    print(f"[case] odd place {first}", flush=True)
    b = m8.PackedRows.of([50, 70])
    q, k, v, g = (randn(i, 120, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    want = [leaf(t) for t in (q, k, v)]
    m8.packed_attention(*want, b).backward(g)
    odd = [at_odd_place(t, first).requires_grad_() for t in (q, k, v)]
    aux = torch.zeros(first, dtype=torch.float16, device="cuda")
    # the concatenation's gradient for the output is contiguous and begins at an odd place
    z = torch.cat([aux, m8.packed_attention(*odd, b).flatten()])
    z.backward(torch.cat([aux, g.flatten()]))
    for a, t in zip(odd, want):
        assert torch.equal(a.grad, t.grad)
    qkv = torch.cat([q, k, v], 1)
    x, y = leaf(qkv), at_odd_place(qkv, first).requires_grad_()
    m8.qkv_attention(x, 2, b).backward(g)
    torch.cat([aux, m8.qkv_attention(y, 2, b).flatten()]).backward(torch.cat([aux, g.flatten()]))
    assert torch.equal(x.grad, y.grad)
