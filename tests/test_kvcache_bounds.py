"""The bounds that the GPU's attention is held to (kv_bounds) are small: any 64 tokens whose values had the wrong
sign, or were left out, would break them (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

pytest.importorskip("torch")
import kv_bounds  # noqa: E402


@pytest.mark.parametrize("case", kv_bounds.CASES, ids=kv_bounds.name)
def test_no_64_tokens_fit_into_the_bound(case):
    *args, kw = case
    least = np.inf
    for _, _, rows in kv_bounds.Data(5, *args).groups(**kw):
        for t in range(0, rows.p.shape[1], 64):
            whole = rows.see[:, t:t + 64].sum(1) >= 32
            if not whole.any():
                continue
            part, weight = rows.share(t)
            negated = -2 * part
            dropped = (rows.o - part) / np.maximum(1 - weight, 1e-300) - rows.o  # and not counted either
            lost = -part                                                       # but counted
            for wrong in (negated, dropped, lost):
                # rows that see nothing else keep their sign only in `negated`
                over = (np.abs(wrong) / rows.tol).max(1)[whole & (weight[:, 0] < 0.999)]
                if over.size:
                    least = min(least, float(over.min()))
    assert least > 2, least
