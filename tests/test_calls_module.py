"""The compiled module of the speculative-decoding calls belongs to one Python and torch: it is
built anew when they change, and without it those calls alone fail, naming the build.  No GPU."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAME = "paged_kv_cache_31_gb300"

USE = """
import torch
from paged_kv_cache_31_gb300 import binding as b
assert b.version() >= 100 and b.status_string(b.PA_EINVAL) == "PA_EINVAL"
assert b.pa_varlen_forward_workspace_size(4, 27, 4, 2, 64, 4, 16) > 0
freq, factor = b.pa_rope_frequencies(64, device="cpu")
assert freq.numel() == 32
try:
    b.pa_copy_blocks(torch.zeros(1, 16, 1, 64), None, torch.zeros(1, 2, dtype=torch.int32))
except ImportError as e:
    print("refused:", e)
"""


@pytest.fixture
def copy(tmp_path):
    from paged_kv_cache_31_gb300 import _build

    _build.build()
    shutil.copytree(os.path.join(ROOT, NAME), tmp_path / NAME,
                    ignore=shutil.ignore_patterns("_build", "__pycache__", "csrc", "_calls*"))
    return tmp_path


def run(where):
    return subprocess.run([sys.executable, "-c", USE], cwd=where, capture_output=True, text=True,
                          env={**os.environ, "PYTHONPATH": str(where)})


def test_the_other_calls_do_not_need_it(copy):
    r = run(copy)
    assert r.returncode == 0, r.stderr
    assert "refused:" in r.stdout and "__graft_entry__.build()" in r.stdout


def test_a_file_that_cannot_be_loaded(copy):
    from paged_kv_cache_31_gb300 import _build

    (copy / NAME / os.path.basename(_build.calls_path())).write_bytes(b"not a library")
    r = run(copy)
    assert r.returncode == 0, r.stderr
    assert "refused:" in r.stdout and "__graft_entry__.build()" in r.stdout


def test_another_torch_is_not_up_to_date(monkeypatch):
    import torch

    from paged_kv_cache_31_gb300 import _build

    _build.build()
    assert _build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert _build.lib_up_to_date() and not _build.calls_up_to_date() and not _build.up_to_date()
