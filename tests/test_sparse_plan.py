"""Host side of the sparse attention's work split (no GPU), under sanitizers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_slots_fragments_and_grids(tmp_path):
    """Rows in blocks, slots of a selection, what the join reads, the largest grid of a selection."""
    if shutil.which(os.environ.get("CXX", "g++")) is None:
        pytest.skip("no host C++ compiler")
    from gated_deltanet_tree_amd import build_host_san  # not there where only GPU tests run
    exe = build_host_san.build_driver(os.path.join(ROOT, "tests", "host_sparse_work.cpp"), str(tmp_path))
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and out.strip().endswith("ok"), out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out
