"""The driver's tensor-map function is looked up once, whichever threads call first."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = "/usr/local/cuda"


def test_first_calls_of_two_threads(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "tma_entry")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I",
                        os.path.join(ROOT, "paged_kv_attention_scatter_gb300", "csrc"), "-I",
                        os.path.join(CUDA, "include"), "-x", "c++",
                        os.path.join(ROOT, "tests", "c", "tma_entry.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
