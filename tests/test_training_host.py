"""The training operators without a GPU: refusals of the C ABI, workspace sizes, the tiles' layout, the device
code's instructions."""
from __future__ import annotations

import ctypes
import math
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import mixed_precision_int8_amd as m8
from mixed_precision_int8_amd.training import _Grad, _ROWS, _SHAPE

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "mixed_precision_int8_amd")
SOURCES = ("attn.hip", "attn_bwd.hip", "rope.hip", "norm.hip", "grads.hip")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F16, F32, BF16 = m8.LLMINT8_DTYPE_F16, m8.LLMINT8_DTYPE_F32, m8.LLMINT8_DTYPE_BF16

P = 0x7f0000000000  # never dereferenced: every call below fails a check or is empty


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m8.library_path()):
        pytest.skip("libllmint8.so not built")
    return m8.load_library()


def shape(cu=P, seqs=4, rows=100, q_heads=8, heads=2, dim=64, scale=0.1, causal=1, window=0, sinks=0):
    return _SHAPE(cu, seqs, rows, q_heads, heads, dim, scale, causal, window, sinks)


def rows_(data=P, token=4096, head=64):
    return _ROWS(data, token, head)


NAMES = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")


def forward(lib, s=None, dtype=F16, lse=P, **over):
    r = [over.get(n, rows_(P + 0x1000000 * i)) for i, n in enumerate(NAMES[:4])]
    return lib.llmint8_attention(s or shape(), dtype, *r, lse, None)


def backward(lib, s=None, dtype=F16, lse=P, ws=P, size=1 << 40, **over):
    r = [over.get(n, rows_(P + 0x1000000 * i)) for i, n in enumerate(NAMES)]
    return lib.llmint8_attention_backward(s or shape(), dtype, *r[:4], lse, *r[4:], ws, size, None)


BAD_SHAPES = [
    (dict(seqs=-1), INVALID), (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(q_heads=0), INVALID),
    (dict(q_heads=7), INVALID), (dict(dim=0), INVALID), (dict(dim=-8), INVALID), (dict(dim=12), UNSUPPORTED),
    (dict(dim=264), UNSUPPORTED), (dict(heads=4097, q_heads=4097), UNSUPPORTED),
    (dict(q_heads=65538, heads=2), UNSUPPORTED), (dict(rows=(1 << 29) + 1), UNSUPPORTED),
    (dict(rows=1 << 29, q_heads=4, heads=2), UNSUPPORTED), (dict(seqs=(1 << 24) + 1), UNSUPPORTED),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(window=5, causal=0), INVALID), (dict(window=1 << 30), UNSUPPORTED),
    (dict(sinks=1 << 30), UNSUPPORTED), (dict(cu=0), INVALID), (dict(cu=P + 2), INVALID),
]


@pytest.mark.parametrize("over,status", BAD_SHAPES)
def test_shapes_that_attention_refuses(lib, over, status):
    assert forward(lib, shape(**over)) == status
    assert backward(lib, shape(**over)) == status


def test_rows_that_attention_refuses(lib):
    bad = [(None, INVALID), (rows_(0), INVALID), (rows_(P + 8), INVALID), (rows_(token=56), INVALID),
           (rows_(token=4100), INVALID), (rows_(head=60), INVALID), (rows_(head=0), INVALID), (rows_(token=0), INVALID),
           (rows_(token=-4096), INVALID), (rows_(token=(1 << 23) + 8), UNSUPPORTED), (rows_(head=1 << 40), UNSUPPORTED)]
    for name in NAMES:
        for r, status in bad:
            if name in NAMES[:4]:
                assert forward(lib, **{name: r}) == status, name
            assert backward(lib, **{name: r}) == status, name
    for dtype in (F32, 3, -1):
        assert forward(lib, dtype=dtype) == INVALID and backward(lib, dtype=dtype) == INVALID
    assert forward(lib, lse=P + 2) == INVALID and backward(lib, lse=P + 2) == INVALID
    assert backward(lib, lse=None) == INVALID
    assert forward(lib, out=rows_(P)) == INVALID  # q's memory
    for name in ("dq", "dk", "dv"):
        assert backward(lib, **{name: rows_(P + 0x3000000)}) == INVALID  # out's
    assert backward(lib, dk=rows_(P + 0x5000000)) == INVALID  # dq's
    assert backward(lib, ws=None) == INVALID and backward(lib, ws=P + 128) == INVALID
    need = lib.llmint8_attention_backward_workspace_bytes(shape())
    assert need == 100 * 8 * 2 * 4 and backward(lib, size=need - 1) == WORKSPACE


def test_nothing_to_attend_to(lib):
    for over in (dict(seqs=0), dict(rows=0)):
        s = shape(**over)
        assert lib.llmint8_attention(s, F16, None, None, None, None, None, None) == OK
        assert lib.llmint8_attention_backward(s, F16, *[None] * 9, None, 0, None) == OK
        assert lib.llmint8_attention_backward_workspace_bytes(s) == 0
    assert lib.llmint8_attention_backward_workspace_bytes(shape(dim=12)) == 0


def rope(lib, dtype=F16, x=None, y=None, heads=4, x2=None, y2=None, heads2=0, rows=10, dim=64, pos=P, axes=2,
         axis=bytes([0, 1] * 16), table=P, table_rows=100, rot=64):
    return lib.llmint8_rope(dtype, x or rows_(), y or rows_(P + 0x1000000), heads, x2, y2, heads2, rows, dim, pos, axes,
                            axis, table, table_rows, rot, 0, 0, None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=F32), INVALID), (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(heads2=-1), INVALID),
    (dict(dim=0), INVALID), (dict(dim=63, rot=62), INVALID), (dict(rot=0), INVALID), (dict(rot=63), INVALID),
    (dict(rot=66), INVALID), (dict(axes=0), INVALID), (dict(axes=9), UNSUPPORTED), (dict(axis=None), INVALID),
    (dict(axis=bytes([0, 2] * 16)), INVALID), (dict(axis=bytes(31) + b"\xff"), INVALID), (dict(pos=None), INVALID),
    (dict(pos=P + 2), INVALID), (dict(table=None), INVALID), (dict(table=P + 2), INVALID), (dict(table_rows=0), INVALID),
    (dict(table_rows=1 << 30), UNSUPPORTED), (dict(rows=1 << 30), UNSUPPORTED), (dict(heads=65537), UNSUPPORTED),
    (dict(dim=65538), UNSUPPORTED), (dict(dim=512, rot=258, axis=bytes(129), x=rows_(token=4096, head=512)), UNSUPPORTED),
    (dict(x=rows_(0)), INVALID), (dict(x=rows_(P + 1)), INVALID), (dict(x=rows_(token=63)), INVALID),
    (dict(x=rows_(head=63)), INVALID), (dict(y=rows_(token=1 << 31)), UNSUPPORTED), (dict(y=rows_(head=1 << 40)), UNSUPPORTED),
    (dict(y=rows_(token=4160)), INVALID),  # in place with other strides
    (dict(x2=rows_()), INVALID), (dict(x2=rows_(), y2=rows_()), INVALID), (dict(heads2=2), INVALID),
    (dict(x2=rows_(), y2=rows_(0), heads2=2), INVALID),
])
def test_rotations_that_are_refused(lib, over, status):
    assert rope(lib, **over) == status
    assert rope(lib, rows=0) == OK


def norm(lib, x=P, x_row=64, dtype=F16, rows=10, K=64, w=P, b=P, w_dtype=F16, eps=1e-5, y=P + 0x1000000, y_row=64, stats=P):
    return lib.llmint8_layer_norm(x, x_row, dtype, rows, K, w, b, w_dtype, eps, y, y_row, stats, None)


def norm_bwd(lib, dy=P, dy_row=64, x=P, x_row=64, dtype=F16, rows=10, K=64, w=P, w_dtype=F16, stats=P, dx=P + 0x1000000,
             dx_row=64, dw=P, db=P + 0x1000, ws=P, size=1 << 40):
    return lib.llmint8_layer_norm_backward(dy, dy_row, x, x_row, dtype, rows, K, w, w_dtype, stats, dx, dx_row, dw, db, ws,
                                           size, None)


def test_norms_that_are_refused(lib):
    both = [(dict(dtype=3), INVALID), (dict(w_dtype=BF16), INVALID), (dict(dtype=F32), INVALID), (dict(rows=-1), INVALID),
            (dict(K=0), INVALID), (dict(K=65537), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED), (dict(x=None), INVALID),
            (dict(x=P + 1), INVALID), (dict(x_row=63), INVALID), (dict(w=P + 1), INVALID), (dict(stats=P + 2), INVALID)]
    for over, status in both:
        assert norm(lib, **over) == status, over
        assert norm_bwd(lib, **over) == status, over
    for over in (dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=None), dict(y_row=63),
                 dict(b=P + 1), dict(y=P, y_row=72)):
        assert norm(lib, **over) == INVALID, over
    for over in (dict(dy=None), dict(dx=None), dict(dx=P), dict(stats=None), dict(dw=P + 1), dict(db=P), dict(ws=None),
                 dict(ws=P + 16), dict(dx_row=63), dict(dy_row=63)):
        assert norm_bwd(lib, **over) == INVALID, over
    need = lib.llmint8_layer_norm_workspace_bytes(10, 64)
    assert need > 0 and need % (2 * 64 * 4) == 0 and norm_bwd(lib, size=need - 1) == WORKSPACE
    assert norm(lib, rows=0, x=None, y=None) == OK and norm_bwd(lib, rows=0, x=None, dw=None, db=None, ws=None) == OK
    assert lib.llmint8_layer_norm_workspace_bytes(10, 0) == 0


def grads(*items):
    arr = (_Grad * max(1, len(items)))()
    for a, it in zip(arr, items):
        a.data, a.out, a.n, a.dtype, a.out_dtype = it
    return arr, len(items)


def test_gradients_that_are_refused(lib):
    good = (P, P, 100, F16, F16)

    def calls(g, scale=1.0, norm_at=P, max_norm=1.0, ws=P, size=1 << 40):
        return (lib.llmint8_grad_norm(*g, scale, norm_at, ws, size, None),
                lib.llmint8_grad_clip(*g, norm_at, max_norm, scale, None))

    for item, status in (((0, P, 100, F16, F16), INVALID), ((P + 1, P, 100, F16, F16), INVALID),
                         ((P + 2, P + 2, 100, F32, F32), INVALID), ((P, P, -1, F16, F16), INVALID),
                         ((P, P, 100, 3, 3), INVALID), ((P, P, 1 << 40, F16, F16), UNSUPPORTED)):
        assert calls(grads(good, item)) == (status, status), item
    for item in ((P, 0, 100, F16, F16), (P, P + 1, 100, F16, F16), (P, P + 0x1000, 100, F16, BF16),
                 (P, P, 100, F16, F32), (P, P + 0x1002, 100, F16, F32)):
        assert calls(grads(good, item), size=0)[1] == INVALID, item
    for over in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(norm_at=None),
                 dict(norm_at=P + 2)):
        assert calls(grads(good), **over) == (INVALID, INVALID), over
    for bad in (0.0, -1.0, math.nan):
        assert calls(grads(good), max_norm=bad, ws=None)[1] == INVALID
    assert calls(grads(good), ws=None, max_norm=0.0) == (INVALID, INVALID)
    assert calls(grads(good), size=7, max_norm=0.0) == (WORKSPACE, INVALID)
    assert lib.llmint8_grad_norm_workspace_bytes(*grads(good, (P, P, 16385, F16, F16), (0, 0, 0, F16, F16))) == 3 * 8
    # half of 2^40 values: no more workgroups than 65536 and one for each tensor
    assert lib.llmint8_grad_norm_workspace_bytes(*grads((P, P, 1 << 39, F16, F16), good)) <= 65538 * 8
    assert lib.llmint8_grad_clip(*grads(), P, 1.0, 1.0, None) == OK
    assert lib.llmint8_grad_clip(*grads((0, 0, 0, F16, F16)), P, 1.0, 1.0, None) == OK
    assert lib.llmint8_grad_norm(None, 1, 1.0, P, P, 8, None) == INVALID


def _hipcc():
    c = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if c is None:
        pytest.skip("hipcc not found")
    return c


def test_attention_s_tiles(tmp_path):
    exe = str(tmp_path / "tiles")
    r = subprocess.run([_hipcc(), "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "attn_tile_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "tiles ok" in r.stdout, r.stdout


PACKED_FP32 = re.compile(r"^\s*v_pk_(add|mul|fma|mov)_(f32|b32)\b", re.M)
SCALAR_WRITE = re.compile(r"^\s*s_(store|buffer_store|atomic|buffer_atomic|scratch_store|dcache_wb|dcache_discard)", re.M)


def test_device_code(tmp_path):
    """No packed fp32, no scalar writes; no vector register spilled in attention of heads of up to 128 channels, nor
    anywhere else; and no copy to LDS inside a loop over the lanes (an address that is not in scalar registers)."""
    from mixed_precision_int8_amd import build
    cc, flags = _hipcc(), [f for f in build.FLAGS if f != "-fPIC"]

    def asm(src):
        out = str(tmp_path / (src + ".s"))
        r = subprocess.run([cc, *flags, "--cuda-device-only", "-S", "-I", os.path.join(ROOT, "include"),
                            os.path.join(PKG, "csrc", src), "-o", out], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return src, open(out).read()

    with ThreadPoolExecutor(max_workers=4) as ex:
        results = list(ex.map(asm, SOURCES))
    for src, text in results:
        assert "s_endpgm" in text
        for pattern in (PACKED_FP32, SCALAR_WRITE):
            m = pattern.search(text)
            assert m is None, f"{src}: {m.group(0).strip()}"
        meta = text[text.find(".amdgpu_metadata"):]
        names, spills = re.findall(r"\.symbol:\s+(\S+)\.kd", meta), re.findall(r"\.vgpr_spill_count:\s+(\d+)", meta)
        assert len(names) == len(spills) > 0
        for name, n in zip(names, spills):
            assert n == "0" or "Li256E" in name and "ka_" in name, (name, n)
        # a loop over lanes ends in a branch back on what is left of exec, right after the copy
        assert not re.search(r"offen lds\n\s+s_xor_b64 exec, exec", text), src
