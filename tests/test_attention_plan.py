"""Host side of the attention's work split (no GPU), under sanitizers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _drive(name, tmp_path):
    if shutil.which(os.environ.get("CXX", "g++")) is None:
        pytest.skip("no host C++ compiler")
    from gated_deltanet_tree_amd import build_host_san  # not there where only GPU tests run
    exe = build_host_san.build_driver(os.path.join(ROOT, "tests", name), str(tmp_path))
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and out.strip().endswith("ok"), out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out


def test_the_join_reads_the_fragments_its_unit_wrote(tmp_path):
    """Units that cost less than the parts they are cut into included."""
    _drive("host_attention_fragments.cpp", tmp_path)


def test_plans_and_the_workspace_query(tmp_path):
    """Refused sizes and offsets need no workspace; offsets without rows do not end the process."""
    _drive("host_attention_plans.cpp", tmp_path)
