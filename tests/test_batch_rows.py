"""Starts that go down over several sequences: every entry point takes them as the highest start so far, so that no row
has two sequences.  The oracle is the same call with starts in order."""
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import paged  # noqa: E402

gpu = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rows_on_the_host(tmp_path):
    """The kernels' own arithmetic, with the maximum over the lanes written as a loop."""
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("HIP's headers are not installed")
    exe = str(tmp_path / "row_owners")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-D__HIP_PLATFORM_AMD__", "-isystem",
           os.path.join(rocm, "include"), os.path.join(ROOT, "tests", "host", "row_owners.cpp"), "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and int(r.stdout) > 100000, r.stderr


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def whole(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# starts, and the tokens of the call
STARTS = [([0, 20, 10, 37], 37), ([0, 37, 5], 37), ([30, 5, 12, 37], 37), ([0, 30, 3, 3, 20, 35, 36], 37), ([-5, 10 ** 9, 7, 30], 37),
          ([5] * 70 + [20] + [3] * 70 + [25, 30], 37), ([0, 9] + [4] * 700 + [15, 12, 37], 37),
          ([0] * 63 + [11] + [2] * 600 + [9, 30], 37), ([0, 400, 100, 395, 600], 500)]


@gpu
@pytest.mark.parametrize("length", [60, 2500])
@pytest.mark.parametrize("starts,n_tok", STARTS, ids=range(len(STARTS)))
def test_starts_that_go_down(device, starts, n_tok, length):
    n = len(starts) - 1
    in_order = np.maximum.accumulate(np.clip(starts, 0, n_tok)).tolist()
    g = torch.Generator(device="cuda").manual_seed(3)
    columns = -(-length // 32)
    pages = 5 * columns
    table = torch.stack([torch.randperm(pages, device="cuda", generator=g)[:columns] for _ in range(n)]).int()
    lengths = whole([length - i % 7 for i in range(n)])
    for dtype, dim in ((F16, 64), (BF16, 128), ("q8", 64)):
        kind = F16 if dtype == "q8" else dtype
        for max_new in (1, n_tok):
            good, down = (qmm.Batch(whole(s), lengths, table, max_new=max_new, max_length=length) for s in (in_order, starts))
            caches = [qmm.Cache(pages, 2, dim, page=32, dtype=dtype) for _ in range(2)]
            q, k, v = (torch.randn(n_tok, h, dim, device="cuda", generator=g).to(kind) for h in (4, 2, 2))
            freq, _ = qmm.rope_frequencies(dim)
            got = []
            for cache, batch in zip(caches, (good, down)):
                x = q.clone()
                qmm.rope_cache(cache, batch, q=x, frequencies=freq, out=x)
                # the pools' numbers, the same for both
                full = qmm.Batch(whole([0, pages * 32]), whole([pages * 32]), torch.arange(pages, device="cuda", dtype=torch.int32)[None])
                kv = torch.Generator(device="cuda").manual_seed(4)
                qmm.rope_cache(cache, full, k=torch.randn(pages * 32, 2, dim, device="cuda", generator=kv).to(kind),
                               v=torch.randn(pages * 32, 2, dim, device="cuda", generator=kv).to(kind))
                out = torch.full((n_tok, 4 * dim), 5.0, dtype=kind, device="cuda")
                qmm.attention(x, cache, batch, out=out)
                back = [t.clone() for t in qmm.cache_read(cache, batch, n_tok)]
                rows = slice(in_order[0], in_order[-1])
                got.append([x, out, *(b[rows] for b in back)])
            torch.cuda.synchronize()
            for a, b in zip(*got):
                assert torch.equal(a, b)
            outside = torch.ones(n_tok, dtype=torch.bool)
            outside[in_order[0]:in_order[-1]] = False
            assert torch.equal(got[1][0][outside.cuda()], q[outside.cuda()]) and bool((got[1][1][outside.cuda()] == 5).all())


@gpu
def test_keys_kept_by_starts_that_go_down(device):
    """Keys and values: each row's go to the slot of its one sequence."""
    starts, n_tok, dim = [0, 20, 10, 33, 37], 37, 64
    in_order = np.maximum.accumulate(starts).tolist()
    p = paged.Paged([40] * 4, [40] * 4, 2, 2, dim, F16, 32, junk=0.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n_tok, 2, dim, device="cuda", generator=g).half() for _ in range(2))
    pools = []
    for s in (in_order, starts):
        cache = qmm.Cache(p.n_pages, 2, dim, page=32)
        qmm.rope_cache(cache, qmm.Batch(whole(s), whole(p.lens), p.table.cuda()), k=k, v=v)
        pools.append((cache.k, cache.v))
    torch.cuda.synchronize()
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    assert int((pools[0][0].view(F16) != 0).sum()) == int((k != 0).sum())


@gpu
@pytest.mark.parametrize("n", [65, 67, 200, 1100, 2300])
def test_one_high_start_anywhere(device, n):
    """One start among many that is above the later ones: the rows behind it belong to those that it leaves in order."""
    n_tok, dim = 64, 64
    cache = qmm.Cache(1, 1, dim, page=32)
    lengths, table = whole([32] * n), torch.zeros((n, 1), dtype=torch.int32).cuda()
    q = torch.randn(n_tok, 1, dim, device="cuda").half()
    freq, _ = qmm.rope_frequencies(dim)
    for at in sorted({0, 1, 62, 63, 64, n // 2, n - 4, n - 2, n - 1} | set(range(255, n - 1, 256)) | set(range(64, n - 1, 256))):
        starts = [0] * at + [40] + [20] * (n - at - 1) + [50]
        in_order = np.maximum.accumulate(starts)
        got = [qmm.rope_cache(cache, qmm.Batch(whole(s), lengths, table), q=q, frequencies=freq, out=torch.full_like(q, 3.0))
               for s in (in_order.tolist(), starts)]
        torch.cuda.synchronize()
        assert torch.equal(*got), at
