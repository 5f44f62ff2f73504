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


def check(case, seed, **data):
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
            err = np.abs(o[at, heads].reshape(rows.o.shape) - rows.o) / rows.tol
            err_lse = np.abs(lse[at, heads].reshape(-1) - rows.lse) / rows.lse_tol
            worst = [max(worst[0], float(err.max())), max(worst[1], float(err_lse.max()))]
        print(f"[case] {kv_bounds.name(case)} max_len {hint}: {worst[0]:.3f} and {worst[1]:.3f} of the bounds", flush=True)
        assert max(worst) <= 1, worst


@pytest.mark.parametrize("case", kv_bounds.CASES, ids=kv_bounds.name)
def test_every_tile_s_values_count(case):
    check(case, 5)
