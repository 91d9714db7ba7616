"""The rows kernel's records of cut groups: each is written by one CTA alone, which clears it first.  The kernel's own
index function is compiled for the host and checked for every shape of a launch."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_25_gb300", "csrc")


def test_no_record_has_two_writers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "cut_record_check")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "native", "cut_record_check.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_kernel_reaches_its_records_through_that_function():
    with open(os.path.join(CSRC, "tree.cu")) as f:
        body = f.read().split("rows_kernel(const TreeArgs a)")[1].split("__global__")[0]
    uses = [x.split("]")[0] for x in body.split("a.cuts[")[1:]]
    assert len(uses) == 2 and all(u.startswith("cut_record(blockIdx.x, W,") for u in uses)
