"""Kernel timing of a pool whose calls come from several threads: no record is lost.  The launch wrapper is compiled from
the library's own header with stand-ins for the CUDA events."""
import os
import shutil
import subprocess

import pytest

from paged_kv_attention_25_gb300 import build as pkv_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_25_gb300", "csrc")


def test_records_of_calls_from_several_threads(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "profile_lists_check")
    cuda = os.path.join(os.path.dirname(os.path.dirname(pkv_build.nvcc())), "include")
    subprocess.run([cxx, "-O2", "-std=c++17", "-pthread", "-I", CSRC, "-I", os.path.join(ROOT, "include"), "-isystem", cuda,
                    os.path.join(ROOT, "tests", "native", "profile_lists_check.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
