"""The host code of the paged cache's operators under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: a build
of libqmm whose host code is instrumented (the device code as usual) answers every call of
tests/sanitize/attention_driver.py."""
import concurrent.futures
import os
import subprocess
import sys

import pytest

from tests.test_sanitizers import ENV, HIPCC, ROOT, _clang_asan


def test_attention_validation_paths(tmp_path):
    runtime = _clang_asan()
    if runtime is None or not os.path.exists(HIPCC):
        pytest.skip("hipcc or clang's AddressSanitizer runtime is not installed")
    csrc = os.path.join(ROOT, "quant_q8_gemm_amd", "csrc")
    flags = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-shared-libsan", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-I", os.path.join(ROOT, "include")]

    def run(*args):
        r = subprocess.run([*flags, *args], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]

    sources = [f for f in sorted(os.listdir(csrc)) if f.endswith((".hip", ".cpp")) and f != "qmm_peak.hip"]
    objects = [str(tmp_path / (f + ".o")) for f in sources]
    with concurrent.futures.ThreadPoolExecutor(6) as pool:
        list(pool.map(lambda f, o: run("-c", os.path.join(csrc, f), "-o", o), sources, objects))
    lib = str(tmp_path / "libqmm_san.so")
    run("-shared", *objects, "-o", lib)
    env = dict(os.environ, LD_PRELOAD=runtime, **ENV)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "sanitize", "attention_driver.py"), lib], env=env,
                       capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "Sanitizer" not in out, out[-3000:]
