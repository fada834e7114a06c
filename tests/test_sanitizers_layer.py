"""The layer operators' host code under AddressSanitizer and UndefinedBehaviorSanitizer,
on the CPU: a build of libqmm whose host code is instrumented (the device code as
usual) answers every refusal of tests/sanitize/layer_driver.py."""
import os
import subprocess
import sys

import pytest

from tests.test_sanitizers import ENV, HIPCC, ROOT, _clang_asan


def test_layer_operators_validation_paths(tmp_path):
    runtime = _clang_asan()
    if runtime is None or not os.path.exists(HIPCC):
        pytest.skip("hipcc or clang's AddressSanitizer runtime is not installed")
    csrc = os.path.join(ROOT, "quant_q8_gemm_amd", "csrc")
    lib = str(tmp_path / "libqmm_san.so")
    sources = [os.path.join(csrc, f) for f in sorted(os.listdir(csrc))
               if f.endswith((".hip", ".cpp")) and f != "qmm_peak.hip"]
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-shared-libsan",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-I", os.path.join(ROOT, "include"), *sources, "-o", lib]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    env = dict(os.environ, LD_PRELOAD=runtime, **ENV)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "sanitize", "layer_driver.py"), lib],
                       env=env, capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "Sanitizer" not in out, out[-3000:]
