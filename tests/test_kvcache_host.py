"""The int8 key/value cache without a GPU: refusals of the C ABI, workspace sizes, the oracle against hand
values, the device code's instructions."""
from __future__ import annotations

import ctypes
import math
import os
import re
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

import mixed_precision_int8_amd as m8
import oracle
from mixed_precision_int8_amd.kvcache import _Batch, _Cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "mixed_precision_int8_amd")
KV_SOURCES = ("kvcache.hip", "kvattn.hip", "kvprompt.hip")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F16, F32, BF16 = m8.LLMINT8_DTYPE_F16, m8.LLMINT8_DTYPE_F32, m8.LLMINT8_DTYPE_BF16

P = 0x7f0000000000  # never dereferenced: every call below fails a check or is empty
MIS = P + 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m8.library_path()):
        pytest.skip("libllmint8.so not built")
    return m8.load_library()


def cache(K=P, V=P, aK=P, aV=P, pages=100, heads=8, page=64, dim=128):
    return _Cache(K, V, aK, aV, pages, heads, page, dim)


def batch(cu=P, length=P, table=P, seqs=4, rows=4, width=50, max_len=0):
    return _Batch(cu, length, table, seqs, rows, width, max_len)


def append(lib, c=None, b=None, dtype=F16, k=(P, 1024, 128), v=(P, 1024, 128), q=(None, 0, 0),
           qo=(None, 0, 0), heads=0, rope=None, rows=0, rot=0):
    return lib.llmint8_kv_append(ctypes.byref(c or cache()), ctypes.byref(b or batch()), dtype, *k, *v, *q,
                                 *qo, heads, rope, rows, rot, 0, None)


def attend(lib, c=None, b=None, dtype=F16, q=(P, 4096, 128), heads=32, scale=0.1, causal=1, window=0, sinks=0,
           out=(P, 4096, 128), lse=None, ws=P, size=None):
    c, b = c or cache(), b or batch()
    if size is None:
        size = 1 << 40
    return lib.llmint8_kv_attention(ctypes.byref(c), ctypes.byref(b), dtype, *q, heads, scale, causal, window,
                                    sinks, *out, lse, ws, size, None)


BAD_CACHES = [(dict(K=None), INVALID), (dict(V=None), INVALID), (dict(aK=None), INVALID), (dict(aV=MIS), INVALID),
              (dict(K=P + 8), INVALID), (dict(V=MIS), INVALID), (dict(pages=0), INVALID), (dict(heads=-1), INVALID),
              (dict(page=48), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
              (dict(dim=72), UNSUPPORTED), (dict(dim=272), UNSUPPORTED), (dict(heads=5000), UNSUPPORTED)]
BAD_BATCHES = [(dict(cu=None), INVALID), (dict(length=None), INVALID), (dict(table=MIS), INVALID),
               (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID),
               (dict(max_len=-1), INVALID), (dict(rows=(1 << 29) + 1), UNSUPPORTED),
               (dict(width=(1 << 23) + 1), UNSUPPORTED), (dict(seqs=1 << 23), UNSUPPORTED)]


def test_refusals_of_caches_and_batches(lib):
    k, v = (P, 1024, 128), (P, 1024, 128)
    for bad, want in [(dict(c=cache(**x)), w) for x, w in BAD_CACHES] + [(dict(b=batch(**x)), w) for x, w in BAD_BATCHES]:
        assert append(lib, **bad) == want, bad
        assert attend(lib, **bad) == want, bad
        c, b = bad.get("c") or cache(), bad.get("b") or batch()
        assert lib.llmint8_kv_gather(ctypes.byref(c), ctypes.byref(b), F16, *k, *v, None) == want, bad
    assert lib.llmint8_kv_append(None, ctypes.byref(batch()), F16, *k, *v, None, 0, 0, None, 0, 0, 0, None, 0,
                                 0, 0, None) == INVALID
    assert lib.llmint8_kv_gather(ctypes.byref(cache()), None, F16, *k, *v, None) == INVALID


def test_refusals_of_rows(lib):
    for bad in ((None, 1024, 128), (MIS, 1024, 128), (P, 100, 128), (P, 1028, 128), (P, 1024, 120), (P, 1024, 132),
                (P, -1024, 128), (P, 1 << 33, 128)):
        assert append(lib, k=bad) == INVALID, bad
        assert append(lib, v=bad) == INVALID, bad
        assert append(lib, q=bad, qo=(P, 4096, 128), heads=32) == INVALID, bad
        assert attend(lib, q=bad) == INVALID, bad
        assert attend(lib, out=bad) == INVALID, bad
        good = (P, 1024, 128)
        for rows in ((bad, good), (good, bad)):
            assert lib.llmint8_kv_gather(ctypes.byref(cache()), ctypes.byref(batch()), F16, *rows[0], *rows[1],
                                         None) == INVALID
    q = (P, 4096, 128)
    assert append(lib, q=q, heads=32) == INVALID                                  # q and no place for it
    assert append(lib, qo=q, heads=32) == INVALID
    assert append(lib, q=q, qo=(P, 8192, 128), heads=32) == INVALID               # in place, other strides
    assert append(lib, q=q, qo=q, heads=0) == INVALID
    assert append(lib, dtype=F32) == INVALID and attend(lib, dtype=F32) == INVALID


def test_refusals_of_rope_and_attention_options(lib):
    assert append(lib, rope=P, rows=10, rot=3) == INVALID
    assert append(lib, rope=P, rows=10, rot=0) == INVALID
    assert append(lib, rope=P, rows=10, rot=130) == INVALID
    assert append(lib, rope=P, rows=0, rot=128) == INVALID
    assert append(lib, rope=P + 4, rows=10, rot=128) == INVALID
    assert attend(lib, heads=0) == INVALID and attend(lib, heads=20) == INVALID
    assert attend(lib, scale=math.nan) == INVALID and attend(lib, scale=math.inf) == INVALID
    assert attend(lib, window=-1) == INVALID and attend(lib, sinks=-1) == INVALID
    assert attend(lib, window=8, causal=0) == INVALID
    assert attend(lib, lse=MIS) == INVALID
    assert attend(lib, ws=None) == INVALID and attend(lib, ws=P + 16) == INVALID
    need = lib.llmint8_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 32, 0, 0)
    assert need > 0 and attend(lib, size=need - 1) == WORKSPACE
    f = (ctypes.c_double * 2)(1.0, 0.5)
    t = lib.llmint8_rope_table
    assert t(None, 2, 5, 1.0, P, None) == INVALID and t(f, 0, 5, 1.0, P, None) == INVALID
    assert t(f, 2, -1, 1.0, P, None) == INVALID and t(f, 2, 5, math.nan, P, None) == INVALID
    assert t(f, 2, 5, 1.0, None, None) == INVALID and t(f, 2, 5, 1.0, P + 8, None) == INVALID
    assert t(f, 129, 5, 1.0, P, None) == UNSUPPORTED
    assert t((ctypes.c_double * 1)(math.inf), 1, 5, 1.0, P, None) == INVALID
    assert t(f, 2, 0, 1.0, None, None) == OK


def test_empty_calls_and_workspace_sizes(lib):
    for b in (batch(rows=0), batch(seqs=0, rows=0, cu=None, length=None, table=None)):
        none = (None, 0, 0)
        assert append(lib, b=b, k=none, v=none) == OK
        assert attend(lib, b=b, q=none, out=none, ws=None, size=0) == OK
    w = lambda **x: lib.llmint8_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch(**x)), 32, 0, 0)  # noqa: E731
    assert w(rows=0) == 0 and w(rows=-1) == 0
    assert w(seqs=4000, rows=4000, width=50) == 0         # enough rows to fill the chip: one part
    assert w(seqs=1, rows=1, width=2000) > 32 * 130 * 4
    assert w(seqs=1, rows=1, width=2000, max_len=64) == 0


def test_oracle_against_hand_values():
    """One page, one head: codes and their move to a larger scale, worked by hand."""
    z = oracle.KVOracle(np.zeros((1, 1, 16, 16), np.int8), np.zeros((1, 1, 16, 16), np.int8), [[9.0]], [[9.0]])
    x = np.zeros((2, 1, 16), np.float32)
    x[0, 0, 0], x[0, 0, 1] = 1.0, -0.5
    x[1, 0, 2] = 0.25
    table = np.zeros((1, 1), np.int32)
    z.append([0, 2], [2], table, x, 2 * x)
    assert z.aK[0, 0] == 1.0 and z.aV[0, 0] == 2.0          # the 9 of before the page began is gone
    assert z.K[0, 0, 0, :2].tolist() == [127, -64]           # -63.5 to even
    assert z.K[0, 0, 1, 2] == 32 and z.V[0, 0, 2, 1] == 32   # 31.75
    x[0, 0, 0] = 4.0
    z.append([0, 1], [3], table, x[:1], x[:1])
    assert z.aK[0, 0] == 4.0 and z.aV[0, 0] == 4.0
    assert z.K[0, 0, 0, :2].tolist() == [32, -16]            # 127 / 4, -64 / 4
    assert z.V[0, 0, :2, 0].tolist() == [64, -32]            # 127 / 2 to even, -64 / 2
    assert z.K[0, 0, 2, 0] == 127
    # rotation by a quarter turn
    y = oracle.KVOracle.rotate(np.arange(1.0, 5.0, dtype=np.float32)[None], oracle.rope_table([math.pi / 2, 0.0], 2), 1, False)
    assert np.allclose(y, [[-3, 2, 1, 4]], atol=1e-6)
    # two equal keys: the mean of the values; a window of one: the last
    z.K[:] = 0
    o, lse, _ = z.attention([0, 1], [2], table, np.ones((1, 1, 16), np.float32))
    v = z.tokens(table, 0, 0, 2)[1][:, 0].astype(np.float64)
    assert np.allclose(o[0, 0], v.mean(0)) and abs(lse[0, 0] - math.log(2)) < 1e-12
    o, lse, _ = z.attention([0, 1], [2], table, np.ones((1, 1, 16), np.float32), window=1)
    assert np.allclose(o[0, 0], v[1]) and lse[0, 0] == 0
    o, lse, _ = z.attention([0, 3], [2], table, np.ones((3, 1, 16), np.float32))
    assert (o[0] == 0).all() and lse[0, 0] == -np.inf and lse[1, 0] == 0


def test_rope_frequencies():
    f, mag = m8.rope_frequencies(8, 10000.0)
    assert mag == 1.0 and np.allclose(f, [1, 0.1, 0.01, 0.001])
    assert np.allclose(m8.rope_frequencies(8, 1e4, "linear", 4.0)[0], np.array(f) / 4)
    g = m8.rope_frequencies(8, 1e4, "ntk", 4.0)[0]
    assert g[0] == 1.0 and abs(g[3] - f[3] / 4) < 1e-9       # the slowest is divided by the factor
    y, mag = m8.rope_frequencies(128, 1e4, "yarn", 4.0, 4096)
    base = m8.rope_frequencies(128, 1e4)[0]
    assert y[0] == base[0] and abs(y[-1] - base[-1] / 4) < 1e-12 and abs(mag - (0.1 * math.log(4) + 1)) < 1e-12
    assert all(b / 4 - 1e-12 <= x <= b + 1e-12 for x, b in zip(y, base))
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, scaling="yarn", factor=2.0),
                dict(rot=8, scaling="other")):
        with pytest.raises(ValueError):
            m8.rope_frequencies(**bad)


def _hipcc():
    return next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)


def test_no_packed_fp32_or_scalar_writes_in_device_code():
    if _hipcc() is None:
        pytest.skip("hipcc not found")
    from mixed_precision_int8_amd import build
    flags = [f for f in build.FLAGS if f != "-fPIC"]
    with tempfile.TemporaryDirectory() as tmp:
        for src in KV_SOURCES:
            out = os.path.join(tmp, src + ".s")
            r = subprocess.run([_hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"),
                                "-I", os.path.join(PKG, "csrc"), os.path.join(PKG, "csrc", src), "-o", out],
                               capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-2000:]
            text = open(out).read()
            assert "s_endpgm" in text
            assert not re.search(r"^\s*v_pk_(add|mul|fma|mov)_(f32|b32)\b", text, re.M), src
            assert not re.search(r"^\s*s_(store|buffer_store|atomic|buffer_atomic|scratch_store|dcache_wb|dcache_discard)",
                                 text, re.M), src
            assert not re.search(r"\.vgpr_spill_count:\s*[1-9]", text), src


def test_refusal_of_more_rows_than_the_kernels_index(lib):
    assert attend(lib, b=batch(rows=1 << 26)) == UNSUPPORTED  # 2^31 rows of 32 heads
    w = lib.llmint8_kv_attention_workspace_bytes
    assert w(ctypes.byref(cache()), ctypes.byref(batch(rows=1 << 26)), 32, 0, 0) == 0
