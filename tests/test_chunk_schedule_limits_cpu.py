"""The work split of the int8 chunk attention at the longest contexts, compiled for the
host and checked against its definition by tests/chunk_schedule_limits_check.cu. No GPU
needed: nvcc compiles host code."""

import os
import subprocess

import pytest

from test_schedule_cpu import ROOT, _nvcc


def test_chunk_schedule_at_the_longest_contexts(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "chunk_schedule_limits_check")
    src = os.path.join(ROOT, "tests", "chunk_schedule_limits_check.cu")
    inc = os.path.join(ROOT, "paged_kv_cache_209_gb300", "csrc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", inc, src, "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok "), r.stdout
