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


@pytest.fixture(params=["table", "lists"])
def gradients(monkeypatch, request):
    """Either way of looking at tensors. [what the library was handed: (name, [(data, out, n, dtype, out_dtype)])], with tensors that pass for a GPU's."""
    training._library()
    calls = []
    if request.param == "lists":
        monkeypatch.setattr(training, "_TABLE", None)
    elif training._describe() is None:
        pytest.skip("no exchange table, or no library")

    class Library:
        def __getattr__(self, name):
            def call(*a):
                if name.endswith("bytes"):
                    return 8 * sum(a[0][i].n for i in range(a[1]))
                calls.append((name, [(e.data or 0, e.out or 0, e.n, e.dtype, e.out_dtype) for e in a[0][:a[1]]]))
                return 0
            return call

    monkeypatch.setattr(m8, "load_library", Library)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(training, "_handle", lambda stream, device: 0)
    return calls


CODE = {torch.float16: m8.LLMINT8_DTYPE_F16, torch.bfloat16: m8.LLMINT8_DTYPE_BF16, torch.float32: m8.LLMINT8_DTYPE_F32}


def entries(grads, outs):
    return [(g.data_ptr(), o.data_ptr(), g.numel(), CODE[g.dtype], CODE[o.dtype]) for g, o in zip(grads, outs)]


def handed(calls, gset, norm):
    """What both calls hand over; the workspace is of what they do."""
    calls.clear()
    m8.llmint8_grad_norm(gset, norm=norm)
    m8.llmint8_grad_clip(gset, norm, 1.0)
    (first, a), (second, b) = calls
    assert (first, second) == ("llmint8_grad_norm", "llmint8_grad_clip") and a == b
    assert gset.workspace_bytes() == 8 * sum(e[2] for e in a)
    return a


def test_a_set_follows_gradients_that_move(gradients):
    norm = torch.zeros(())
    model = torch.nn.Sequential(torch.nn.Linear(7, 5), torch.nn.Linear(5, 3))
    for p in model.parameters():
        p.grad = torch.ones_like(p)
    grads = [p.grad for p in model.parameters()]
    gset = m8.GradientSet(grads)
    assert handed(gradients, gset, norm) == entries(grads, grads)
    held = [g.detach() for g in grads]  # so that the new ones are elsewhere
    for change in (model.half, model.bfloat16, model.float):
        change()
        assert [p.grad.dtype for p in model.parameters()] == [grads[0].dtype] * 4
        held += [g.detach() for g in grads]
        assert handed(gradients, gset, norm) == entries(grads, grads), change
    grads[1].data = torch.zeros(5)          # the same type, other memory
    assert handed(gradients, gset, norm) == entries(grads, grads)
    grads[0].data = grads[0].data[:2]       # the same place, fewer values
    assert handed(gradients, gset, norm) == entries(grads, grads)
    grads[1].data = grads[1].data.view(torch.float16)  # the same place, another type
    assert handed(gradients, gset, norm) == entries(grads, grads)


def test_a_set_follows_outputs_that_move(gradients):
    norm = torch.zeros(())
    grads, outs = [torch.zeros(9).half(), torch.zeros(4).half()], [torch.zeros(9), torch.zeros(4)]
    gset = m8.GradientSet(grads, out=outs)
    assert handed(gradients, gset, norm) == entries(grads, outs)
    outs[1].data = torch.zeros(4)
    assert handed(gradients, gset, norm) == entries(grads, outs)
    outs[0].data = torch.zeros(9).half()
    assert handed(gradients, gset, norm) == entries(grads, outs)


def test_a_set_whose_tensors_no_longer_fit_is_refused(gradients):
    norm = torch.zeros(())
    grads, outs = [torch.zeros(9).half(), torch.zeros(4).half()], [torch.zeros(9), torch.zeros(4)]
    gset = m8.GradientSet(grads, out=outs)
    gradients.clear()
    for bad, good in ((torch.zeros(4).bfloat16(), outs[1].data), (torch.zeros(5), outs[1].data),
                      (outs[0].data[:4], outs[1].data)):
        outs[1].data = bad
        for _ in range(2):  # not only the first time
            with pytest.raises(ValueError):
                m8.llmint8_grad_norm(gset, norm=norm)
            with pytest.raises(ValueError):
                m8.llmint8_grad_clip(gset, norm, 1.0)
            with pytest.raises(ValueError):
                gset.workspace_bytes()
        assert not gradients
        outs[1].data = good
        assert handed(gradients, gset, norm) == entries(grads, outs)
        gradients.clear()


def test_the_list_that_is_returned_is_the_caller_s(gradients):
    norm = torch.zeros(())
    grads = [torch.zeros(9), torch.zeros(4)]
    gset = m8.GradientSet(grads)
    m8.llmint8_grad_clip(gset, norm, 1.0).append(torch.zeros(6))
    assert handed(gradients, gset, norm) == entries(grads, grads)
    with pytest.raises(AttributeError):  # the set's own do not change: as many entries as tensors
        gset.grads.append(torch.zeros(6))


def test_statistics_on_another_device_are_refused(monkeypatch):
    training._library()
    called = []
    monkeypatch.setattr(m8, "load_library", lambda: type("L", (), {"llmint8_layer_norm": lambda s, *a: called.append(a) or 0})())
    monkeypatch.setattr(m8, "_need", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(training, "_handle", lambda stream, device: 0)
    x = torch.zeros((6, 24)).half()
    m8.llmint8_layer_norm(x, stats=torch.zeros((6, 2)))
    assert len(called) == 1
    with pytest.raises(ValueError, match="stats"):
        m8.llmint8_layer_norm(x, stats=torch.zeros((6, 2), device="meta"))
    assert len(called) == 1


def test_rotations_of_host_memory_are_refused(monkeypatch):
    """Also on a stream of the caller's, where nothing else asks for the device."""
    training._library()
    called = []
    monkeypatch.setattr(m8, "load_library", lambda: type("L", (), {"llmint8_rope": lambda s, *a: called.append(a) or 0})())
    stream = type("Stream", (), {"cuda_stream": 5})()
    q, out = torch.zeros((6, 4, 16)).half(), torch.zeros((6, 4, 16)).half()
    with pytest.raises(ValueError, match="CUDA"):
        m8.llmint8_rope(torch.zeros((9, 16)), torch.zeros(6, dtype=torch.int32), bytes(8), q, q_out=out, stream=stream)
    assert not called


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(m8.library_path()):
        pytest.skip("libllmint8.so not built")
    return m8.load_library()


@pytest.mark.parametrize("seqs,rows,q_heads,heads,dim,forward", [
    (1 << 24, 1 << 24, 1, 1, 64, True), (1 << 21, 100, 8, 8, 64, True), ((1 << 24) - 8, 1 << 10, 1, 1, 64, True),
    (1 << 20, 1 << 26, 16, 16, 64, True),                # 2^20 + 2^19 for each of 16 heads
    (1 << 20, 100, 8, 8, 128, False), ((1 << 23) - 8, 1 << 10, 1, 1, 104, False), (1, 1 << 30, 1, 1, 128, True),
    (1 << 23, 1 << 29, 1, 1, 136, False),                # 2^23 tiles of 64 tokens
])
def test_more_work_items_than_a_launch_has_are_refused(lib, seqs, rows, q_heads, heads, dim, forward):
    P = 0x7f0000000000  # never read: every call is refused
    shape = training._SHAPE(P, seqs, rows, q_heads, heads, dim, 0.1, 1, 0, 0)
    other = [training._ROWS(P + 0x1000000 * i, q_heads * heads * 256, 256) for i in range(8)]
    if forward:
        assert lib.llmint8_attention(shape, m8.LLMINT8_DTYPE_F16, *other[:4], P, None) == -2
    assert lib.llmint8_attention_backward(shape, m8.LLMINT8_DTYPE_F16, *other[:4], P, *other[4:], P, 1 << 50, None) == -2


def test_rows_are_dealt_to_launches(tmp_path):
    import os
    import shutil
    import subprocess
    cc = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if cc is None:
        pytest.skip("hipcc not found")
    root, exe = os.path.dirname(os.path.dirname(os.path.abspath(__file__))), str(tmp_path / "rows")
    r = subprocess.run([cc, "-O1", "-std=c++17", "-I", os.path.join(root, "include"),
                        os.path.join(root, "tests", "train_rows_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "rows ok" in r.stdout, r.stdout


def test_a_set_of_tensors_of_every_kind(gradients):
    """That require a gradient, are parameters, empty, or not contiguous."""
    norm = torch.zeros(())
    grads = [torch.zeros(3).requires_grad_(), torch.nn.Parameter(torch.zeros(4, 2)), torch.zeros(0), torch.zeros(5, 3).t(),
             torch.zeros(()), torch.zeros(2, 3)[1:]]
    gset = m8.GradientSet(grads)
    assert handed(gradients, gset, norm) == entries(grads, grads)
    for g in grads:
        g.data = g.data.clone()
        assert handed(gradients, gset, norm) == entries(grads, grads)
    assert len(m8.GradientSet([])) == 0 and len(m8.GradientSet([])._current()) == 0


def test_used_rows_of_a_call_captured_on_another_device(packed, monkeypatch):
    """Asked of the device that the batch is on, whatever the current one is."""
    import contextlib
    filled, _ = packed
    b = m8.PackedRows.of([3, 2], device="cpu")
    b.device = torch.device("cuda", 1)
    at = [0]

    @contextlib.contextmanager
    def on(device):
        at.append(device.index)
        yield
        at.pop()

    monkeypatch.setattr(training, "_on", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at[-1] == 1)
    assert b.used_rows() is None and at == [0]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at[-1] == 0)
    assert b.used_rows() == 5


def test_one_parameter_is_clipped(gradients):
    p = torch.nn.Parameter(torch.zeros(4, 3))
    p.grad = torch.ones(4, 3)
    gradients.clear()
    m8.clip_grad_norm(p, 1.0)
    assert [c for c in gradients] == [(name, entries([p.grad], [p.grad])) for name in ("llmint8_grad_norm", "llmint8_grad_clip")]
    gradients.clear()
    m8.clip_grad_norm((x for x in [p, torch.nn.Parameter(torch.zeros(2))]), 1.0)
    assert [len(c[1]) for c in gradients] == [1, 1]


def test_what_the_host_knows_may_be_assigned(packed):
    """After a change of cu, by a program that keeps the batch."""
    filled, _ = packed
    b = m8.PackedRows.of([60, 60], device="cpu")
    b.cu.copy_(torch.tensor([0, 30, 90], dtype=torch.int32))
    assert b.used_rows() is None and b.longest() == 120
    b.used = 90
    assert b.used == 90 and torch.isnan(filled(b)[:90]).all() and (filled(b)[90:] == 0).all() and b.longest() == 120
    b.max_len = 60
    assert b.longest() == 60 and b.used_rows() == 90
    b.cu.copy_(torch.tensor([0, 60, 80], dtype=torch.int32))
    assert b.longest() == 60 and b.used_rows() is None and (filled(b) == 0).all()
    for name in ("used", "max_len"):
        with pytest.raises(ValueError, match=name):
            setattr(b, name, -1)
    b.used = None
    assert b.used_rows() is None
