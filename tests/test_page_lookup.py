"""The attention kernels' page lookups (qmm_pages.h) compiled for the host, against the table."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_lookups_on_the_host(tmp_path):
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("HIP's headers are not installed")
    exe = str(tmp_path / "page_lookup")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-D__HIP_PLATFORM_AMD__", "-isystem",
           os.path.join(rocm, "include"), os.path.join(ROOT, "tests", "host", "page_lookup.cpp"), "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and int(r.stdout) > 100000, r.stderr
