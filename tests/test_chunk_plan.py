"""Host check of how chunk attention cuts a ragged batch into work (items, units, the
workers' snapped ranges): compiles tests/cpp/chunk_plan_check.cpp against the kernels' own
header with the host compiler and runs it. No GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "cpp", "chunk_plan_check.cpp")
CSRC = os.path.join(ROOT, "paged_decode_attention_02_gb300", "csrc")


def test_ranges_cover_every_key_tile_once(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "chunk_plan_check")
    subprocess.run([cxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC, SRC, "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
