"""Calls from several threads at once.  On the CPU: what the library launches, recorded
by a program that answers the HIP runtime's calls itself (tests/host/launch_order.cpp).
On the GPU: two threads on one stream, every result bit for bit."""
import os
import shutil
import subprocess
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def launch_order(tmp_path_factory):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("g++ or HIP's headers are not installed")
    exe = str(tmp_path_factory.mktemp("host") / "launch_order")
    cmd = ["g++", "-std=c++20", "-O1", "-Wall", "-D__HIP_PLATFORM_AMD__", "-isystem", os.path.join(ROCM, "include"),
           os.path.join(ROOT, "tests", "host", "launch_order.cpp"), "-rdynamic", "-ldl", "-pthread", "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    return exe


@pytest.mark.parametrize("entry", ["mmq", "noalloc", "epilogue", "work"])
def test_a_split_products_kernels_stay_together_on_a_stream(launch_order, entry):
    env = dict(os.environ, LD_LIBRARY_PATH=os.path.join(ROCM, "lib") + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    r = subprocess.run([launch_order, qmm.LIB_PATH, entry, "stream"], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("entry", ["mmq", "epilogue"])
def test_every_threads_own_stream_has_its_own_scratch(launch_order, entry):
    env = dict(os.environ, LD_LIBRARY_PATH=os.path.join(ROCM, "lib") + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    r = subprocess.run([launch_order, qmm.LIB_PATH, entry, "per_thread"], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["mmq", "noalloc", "epilogue", "work"])
def test_two_threads_on_one_stream(entry):
    """A split tail (4352 x 2048, 509 tokens), called by two threads on one stream with inputs of their own."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    type_, od, id_, T = synth.Q6_K, 4352, 2048, 509
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    plan = qmm.mmq_plan(type_, od, id_, T, cus)
    assert cus != 256 or plan.n_tail > 0
    raw, x = synth.case(type_, od, id_, T, seed=4)
    w = qmm.register_weights(type_, od, id_, raw)
    x = torch.from_numpy(x).cuda()
    qacts = [qmm.quantize_activations(x), qmm.quantize_activations(x.flip(0).contiguous())]
    refs = [qmm.mmq(w, q, T) for q in qacts]
    outs = [[torch.full((T, od), float("nan"), device="cuda") for _ in range(40)] for _ in qacts]
    work = torch.empty(max(plan.scratch_bytes, 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def run(i):
        try:
            torch.cuda.set_device(0)
            start.wait(60)
            for out in outs[i]:
                if entry == "mmq":
                    qmm.mmq(w, qacts[i], T, out=out, stream=0)
                elif entry == "noalloc":
                    qmm.mmq_noalloc(w, qacts[i], T, out, stream=0)
                else:
                    qmm.mmq_epilogue(w, qacts[i], T, out=out, work=work if entry == "work" else None, stream=0)
        except Exception as e:  # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for ref, many in zip(refs, outs):
        for out in many:
            assert np.array_equal(out.cpu().numpy().view(np.uint32), ref.cpu().numpy().view(np.uint32))
    w.release()
