"""Index arithmetic of the key/value cache's kernels, on the CPU: ``tests/kv_index_check.cpp`` sweeps the
functions that the kernels and it share (``csrc/kv_internal.h``)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    hipcc = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if hipcc is None:
        pytest.skip("hipcc not found")
    exe = str(tmp_path_factory.mktemp("kv") / "kv_index_check")
    r = subprocess.run([hipcc, "-O2", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "kv_index_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def run(what):
        r = subprocess.run([exe, what], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and f"{what} ok" in r.stdout, (r.stdout + r.stderr)[-3000:]

    return run


def test_every_row_of_a_batch_is_worked_on_once(check):
    """Also where the call has rows past the last sequence's."""
    check("items")


def test_a_note_of_any_content_names_rows_of_the_workspace(check):
    """A row that no run holds (cu that falls) has a note of whatever the workspace held."""
    check("notes")


def test_rows_keep_their_positions_whatever_the_length(check):
    """Tokens past the end of the table have no page; the rows before them stay where they are."""
    check("positions")
