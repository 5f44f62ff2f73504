"""Attention over the int8 key/value cache against 64 bits within bounds that no 64 tokens fit into (kv_bounds):
the values of every tile, part and join count, not the weights alone."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import kv_bounds  # noqa: E402
import mixed_precision_int8_amd as m8  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m8.load_library()
    yield
    torch.cuda.synchronize()


def check(case, seed, bound="tol", **data):
    *args, kw = case
    d = kv_bounds.Data(seed, *args, **data)
    r = d.ref
    cache = m8.KVCache(*(torch.from_numpy(x).cuda() for x in (r.K, r.V, r.aK, r.aV)))
    batch = [torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (d.cu, d.lens, d.table)]
    want = list(d.groups(**kw))
    for hint in (0, 1, max(d.lens)):
        lse = torch.full((d.rows, d.q_heads), 3.0, device="cuda")
        o = m8.llmint8_kv_attention(cache, m8.KVBatch(*batch, d.rows, max_len=hint), d.q.cuda(), lse=lse, **kw)
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        worst = [0.0, 0.0]
        for at, heads, rows in want:
            err = np.abs(o[at, heads].reshape(rows.o.shape) - rows.o) / getattr(rows, bound)
            err_lse = np.abs(lse[at, heads].reshape(-1) - rows.lse) / rows.lse_tol
            worst = [max(worst[0], float(err.max())), max(worst[1], float(err_lse.max()))]
        print(f"[case] {kv_bounds.name(case)} max_len {hint}: {worst[0]:.3f} and {worst[1]:.3f} of the bounds", flush=True)
        assert max(worst) <= 1, worst


@pytest.mark.parametrize("case", kv_bounds.CASES, ids=kv_bounds.name)
def test_every_tile_s_values_count(case):
    check(case, 5)


DOMINANT = [([700, 90], [1, 1], 2, 4, 128, 64, "f16", {}), ([700, 90], [3, 1], 1, 5, 64, 16, "bf16", {}),
            ([2600], [1], 1, 2, 96, 64, "f16", {}), ([700, 90], [200, 90], 1, 2, 128, 64, "f16", {}),
            ([700, 90], [200, 90], 1, 2, 64, 16, "bf16", {})]


@pytest.mark.parametrize("case", DOMINANT, ids=kv_bounds.name)
def test_one_channel_of_q_far_above_the_others(case):
    """The others are held to 2^-16 of it by the 8-bit products, exactly by the 16-bit ones."""
    check(case, 6, bound="exact_q_tol" if max(case[1]) == 200 else "tol", dominant=1000.0)


@pytest.mark.parametrize("counts", [[1], [200]])
def test_pages_whose_values_differ_by_2_to_the_100(counts):
    """Two pages that weigh the same, the larger one's values 2^100 times the other's: half of the larger."""
    dim, page, n = 64, 64, 128
    for small, large in ((2.0 ** -50, 2.0 ** 50), (0.0, 2.0 ** 36)):
        codes = torch.full((2, 1, page, dim), 127, dtype=torch.int8, device="cuda")
        aV = torch.tensor([[large], [small]], device="cuda")
        cache = m8.KVCache(torch.zeros_like(codes), codes.clone(), torch.ones_like(aV), aV)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        batch = m8.KVBatch(ints([0, counts[0]]), ints([n]), ints([[0, 1]]), counts[0])
        q = torch.ones((counts[0], 1, dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((counts[0], 1), device="cuda")
        o = m8.llmint8_kv_attention(cache, batch, q, causal=False, lse=lse).double().cpu()
        assert ((o - large / 2).abs() <= 2.0 ** -8 * large / 2).all()
        assert (lse.cpu() - np.log(n)).abs().max() <= 2.0 ** -18
