"""qmm_attention: refusals on the CPU; on the GPU against the formula in 64 bits, with the tolerance that
tests/paged.py derives from the roundings (Paged.reference), plus half a step of the type an output is stored in."""
import ctypes
import itertools
import math
import os
import re
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import layouts, paged  # noqa: E402

gpu = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
CACHES = [F16, BF16, "q8"]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- on the CPU ----

from tests.test_rope_cache import BASE, BATCH_REFUSED, CACHE_REFUSED, batch_struct, cache_struct  # noqa: E402

N, H = 5, 4


def attn_struct(**kw):
    a = dict(heads=H, causal=1, out_type=1, scale=0.125, window=0, q=6 * BASE, q_stride=H * 64, q_head_stride=64, out=7 * BASE,
             out_stride=H * 64)
    a.update(kw)
    return qmm.Attn(**a)


def test_structs_match_header():
    hdr = open(os.path.join(ROOT, "include", "qmm.h")).read()
    for name, struct in (("qmm_attn", qmm.Attn), ("qmm_attn_plan", qmm.AttnPlan)):
        body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} %s;" % name, hdr, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        assert re.findall(r"(\w+)\s*[;,]", body) == [f[0] for f in struct._fields_]


REFUSED = [(dict(heads=0), "heads"), (dict(heads=3), "heads"), (dict(heads=8192), "heads"), (dict(causal=2), "causal"),
           (dict(out_type=0), "out_type"), (dict(out_type=2), "out_type"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"),
           (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=1e-31), "scale"),
           (dict(scale=2e30), "scale"), (dict(window=-1), "window"),
           (dict(window=4, causal=0), "window"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(out=7 * BASE + 8), "aligned"),
           (dict(q=6 * BASE + 2), "aligned"), (dict(q_stride=60), "q's strides"), (dict(q_stride=H * 64 + 4), "q's strides"),
           (dict(q_head_stride=32), "q's strides"), (dict(out_stride=H * 64 - 8), "out_stride"), (dict(out_stride=H * 64 + 4), "out_stride"),
           (dict(out_stride=1 << 25), "out_stride"), (dict(out_type=3), "qmm_qact_bytes"), (dict(out=6 * BASE), "overlaps"),
           (dict(out=BASE + 4096), "overlaps"), (dict(out=2 * BASE - 512), "overlaps"), (dict(out=3 * BASE), "overlaps")]


@pytest.mark.parametrize("kw,word", CACHE_REFUSED + BATCH_REFUSED + REFUSED)
def test_refused(kw, word):
    parts = [dict() for _ in range(3)]
    parts[1 if (kw, word) in CACHE_REFUSED else 2 if (kw, word) in BATCH_REFUSED else 0] = kw
    rc = qmm._lib.qmm_attention(attn_struct(**parts[0]), cache_struct(**parts[1]), batch_struct(**parts[2]), N, None, 0, None)
    assert rc == qmm.EINVAL and word in qmm.last_error(), qmm.last_error()


@pytest.mark.parametrize("work,size,word", [(None, 64, "work"), (8 * BASE, 0, "work"), (8 * BASE + 8, 64, "work"),
                                            (6 * BASE, 64, "overlaps"), (7 * BASE + 256, 64, "overlaps"), (BASE, 64, "overlaps")])
def test_work_memory_refused(work, size, word):
    assert qmm._lib.qmm_attention(attn_struct(), cache_struct(), batch_struct(), N, work, size, None) == qmm.EINVAL
    assert word in qmm.last_error()


def test_q8_output_refused():
    """heads * head_dim has to be whole rows of q8 blocks for the next product."""
    c = cache_struct(head_dim=96, heads=1)
    a = attn_struct(heads=2, out_type=3, q_stride=192, q_head_stride=96, out_stride=0)
    assert qmm._lib.qmm_attention(a, c, batch_struct(), N, None, 0, None) == qmm.EINVAL
    assert "256" in qmm.last_error()


@pytest.mark.parametrize("n_tok", [-1, (1 << 20) + 1])
def test_token_counts_refused(n_tok):
    assert qmm._lib.qmm_attention(attn_struct(), cache_struct(), batch_struct(), n_tok, None, 0, None) == qmm.EINVAL


def test_null_structs_and_empty_batch():
    L = qmm._lib
    assert L.qmm_attention(None, cache_struct(), batch_struct(), N, None, 0, None) == qmm.EINVAL
    assert L.qmm_attention(attn_struct(), None, batch_struct(), N, None, 0, None) == qmm.EINVAL
    assert L.qmm_attention(attn_struct(), cache_struct(), None, N, None, 0, None) == qmm.EINVAL
    assert L.qmm_attention(attn_struct(q=None, out=None), cache_struct(), batch_struct(), 0, None, 0, None) == qmm.OK


def _plan(heads, kv_heads, dim, n_seq, n_tok, max_new, max_length, cus=256, type_=1, window=0):
    plan = qmm.AttnPlan()
    rc = qmm._lib.qmm_attention_plan(cache_struct(type=type_, heads=kv_heads, head_dim=dim), batch_struct(n_seq=n_seq, max_new=max_new,
                                     max_length=max_length), heads, window, n_tok, cus, plan)
    return rc, plan


def test_plans():
    """Every plan's tiles cover the columns of max_new tokens, its splits fit the work memory, and it fits a launch."""
    rng = np.random.default_rng(0)
    for _ in range(3000):
        kv = int(rng.integers(1, 33))
        group, dim = int(rng.choice([1, 2, 4, 5, 8, 16, 71])), int(rng.choice([64, 96, 128, 192, 256]))
        n_seq, max_new = int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 12))
        n_tok = min(1 << 17, n_seq * max_new)
        length = int(2 ** rng.uniform(0, 20))
        cus = int(rng.choice([1, 64, 256, 304]))
        rc, p = _plan(kv * group, kv, dim, n_seq, n_tok, max_new, length, cus, int(rng.choice([1, 2, 3])))
        assert rc == qmm.OK, qmm.last_error()
        flats = min(max_new, n_tok) * group
        assert p.columns <= (32 if p.few else 128) and flats > (p.tiles - 1) * p.columns
        # every tile has a work-group, or there are very many and they take turns
        assert p.tiles * p.columns >= flats or (not p.few and n_seq * kv * (p.tiles + 1) > 1 << 18)
        assert p.work_groups < 1 << 30 and p.tiles * n_seq * kv <= max(1 << 18, 2 * n_seq * kv)
        assert p.work_groups == n_seq * kv * p.tiles * p.splits
        assert p.work_bytes == (0 if p.splits == 1 else p.splits * n_tok * kv * group * (dim * 4 + 8))
        assert p.splits == 1 or p.splits * 32 <= max(length, 32)
        assert p.splits * p.share * 32 >= length and (p.splits - 1) * p.share * 32 < length
        lds = 4 * (8 if dim <= 128 else 4) * (64 + p.columns * (dim + 4)) if p.few else 0
        assert lds <= 160 * 1024


@pytest.mark.parametrize("kw", [dict(heads=3), dict(n_seq=0), dict(max_new=-1), dict(max_length=-1), dict(cus=0), dict(type_=0),
                                dict(dim=80), dict(n_tok=-1), dict(n_tok=1 << 20, heads=4096)])
def test_plans_refused(kw):
    a = dict(heads=4, kv_heads=2, dim=64, n_seq=2, n_tok=5, max_new=5, max_length=100, cus=256, type_=1)
    a.update(kw)
    assert _plan(*a.values())[0] == qmm.EINVAL


def test_bounds_on_the_host(tmp_path):
    """The kernels' own lookups, compiled for the host: pages outside the pool and unfit batches lead nowhere."""
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("HIP's headers are not installed")
    exe = str(tmp_path / "cache_bounds")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover", "-D__HIP_PLATFORM_AMD__", "-isystem",
           os.path.join(rocm, "include"), os.path.join(ROOT, "tests", "host", "cache_bounds.cpp"), "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and int(r.stdout) > 100000, r.stderr


def test_binding_refuses_on_the_cpu():
    cache = qmm.Cache(4, 2, 64, page=32, device="cpu")
    with pytest.raises(qmm.QmmError):
        qmm.attention(torch.zeros(1, 2, 64, dtype=F16), cache, None)


# ---- on the GPU ----

@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def close(got, ref, off, type_):
    got = got.double().cpu()
    allowed = off + paged.HALF[type_] * (ref.abs() + off) + (2.0 ** -25 if type_ == F16 else 0)
    wrong = (got - ref).abs() - allowed
    assert bool((wrong <= 0).all()), f"{(wrong > 0).sum()} of {wrong.numel()} off, worst {wrong.max():.3e} at " \
        f"{np.unravel_index(int(wrong.argmax()), wrong.shape)}; nan {got.isnan().sum()}"


def check(p, causal=True, window=0, scale=None, **hints):
    cache, batch, q = p.cuda(qmm, **hints)
    out = qmm.attention(q, cache, batch, causal=causal, window=window, scale=scale)
    torch.cuda.synchronize()
    close(out, *p.reference(causal, window, scale), p.type)
    return out


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("new,length", [(1, 1), (1, 33), (1, 300), (5, 70), (70, 70), (150, 333)])
def test_one_sequence(device, dtype, dim, new, length):
    check(paged.Paged([new], [length], 4, 2, dim, dtype))


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (4, 1), (10, 2), (40, 8), (71, 1), (66, 2)])
def test_heads(device, dtype, heads, kv_heads):
    for new, length in ((1, 130), (9, 50)):
        check(paged.Paged([new], [length], heads, kv_heads, 64, dtype))


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 2, 3])
def test_whole_tiles_of_few_columns(device, dtype, dim, new):
    """32 heads of a cache head: 32 columns a token, in one, two and three tiles of the smallest kind; the last is the
    kernel's of many columns."""
    check(paged.Paged([new, 1], [300, 40], 32, 1, dim, dtype))


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [32, 64])
def test_either_side_of_two_groups_of_waves(device, dtype, dim, page):
    """Up to one work-group for a compute unit its keys are shared by two groups of waves, beyond by one: the same
    sequence by itself and among others."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    news, lens = [70], [333]
    check(paged.Paged(news, lens, 2, 2, dim, dtype, page))
    n = cus // 4 + 1
    many = paged.Paged(news + [65 + i % 9 for i in range(n)], lens + [90 + 3 * i for i in range(n)], 4, 4, dim, dtype, page)
    cache, batch, q = many.cuda(qmm)
    assert qmm.attention_plan(cache, batch, 4, q.shape[0], cus).work_groups > cus
    check(many)
    check(paged.Paged(news + [65] * n, lens + [90 + 3 * i for i in range(n)], 4, 4, dim, dtype, page), causal=False)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_many_work_groups(device, dtype, dim):
    """More work-groups than compute units, one group of waves each: a window, an output in q8 blocks, and a value that is
    no number, which reaches the tokens that see it and no others."""
    n = torch.cuda.get_device_properties(0).multi_processor_count // 4 + 1
    p = paged.Paged([150, 0] + [65 + i % 9 for i in range(n)], [333, 20] + [90 + 3 * i for i in range(n)], 4, 4, dim, dtype, 32)
    check(p, window=77)
    cache, batch, q = p.cuda(qmm)
    clean = qmm.attention(q, cache, batch).clone()
    if 4 * dim % 256 == 0:  # whole super-blocks
        blocks = qmm.attention(q, cache, batch, dtype="q8")
        torch.cuda.synchronize()
        q8_close(p, blocks, *p.reference())
    for slot in (200, 300):  # seen by all but 17 and by 33 of the 150 tokens
        pool, page, at = cache.v.clone(), p.where[0][slot // 32], slot - 183
        x = paged.unpacked(cache.v, dtype, "v", p.n_pages, 4, 32, dim) if dtype != "q8" else None
        if dtype == "q8":  # the first block's scale
            b, byte = cache.v.view(p.n_pages, 4, -1), 32 * dim + (slot % 32) * 2
            b[page, 2, byte], b[page, 2, byte + 1] = 0, 0x7e
        else:
            x[page, 2, slot % 32, 3] = float("nan")
            cache.v.copy_(paged.packed(x, dtype, "v").cuda())
        out = qmm.attention(q, cache, batch)
        torch.cuda.synchronize()
        cache.v.copy_(pool)
        width = slice(0, 32) if dtype == "q8" else slice(3, 4)
        assert bool(out[at:150, 2, width].isnan().all())
        out[at:150, 2, width] = clean[at:150, 2, width]
        assert torch.equal(out, clean)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
def test_shared_pages(device, dtype):
    """Two sequences whose tables begin with the same pages: a common prompt."""
    for new in (1, 40):
        p = paged.Paged([new, new], [150, 200], 4, 2, 64, dtype)
        p.where[1][:3] = p.where[0][:3]
        p.table[1, :3] = p.table[0, :3]
        for x in (p.k, p.v):
            x[1][:96] = x[0][:96]
        check(p)


@gpu
@pytest.mark.parametrize("page", [32, 64, 128, 512])
@pytest.mark.parametrize("dtype", CACHES, ids=str)
def test_pages_and_ragged_batches(device, page, dtype):
    news, lens = [1, 0, 40, 7, 130, 1, 3], [1, 90, 40, 300, 450, 700, 3]
    check(paged.Paged(news, lens, 4, 2, 64, dtype, page))
    check(paged.Paged([1] * 5, [1, 31, 32, 33, 200], 4, 2, 128, dtype, page))


@gpu
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (96, "q8"), (256, F16)], ids=str)
@pytest.mark.parametrize("window", [1, 5, 32, 33, 100, 1000])
def test_window(device, dim, dtype, window):
    check(paged.Paged([1, 70, 5], [200, 333, 5], 4, 2, dim, dtype), window=window)
    check(paged.Paged([1, 2], [200, 97], 4, 2, dim, dtype), window=window)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_cross(device, dtype, dim):
    """Lengths that have nothing to do with the tokens', none among them: rows of zeros."""
    for news in ([1, 1, 1, 1], [40, 3, 90, 17]):
        out = check(paged.Paged(news, [150, 0, 1, 33], 6, 3, dim, dtype), causal=False)
        assert not out[news[0]:news[0] + news[1]].any()


@gpu
def test_more_tokens_than_slots(device):
    """The first tokens have no slot and see nothing."""
    for new, group in ((3, 1), (50, 4)):
        p = paged.Paged([new], [2], 2 * group, 2, 64, F16)
        out = check(p)
        assert not out[:new - 2].any() and out[new - 2:].any()


@gpu
@pytest.mark.parametrize("scale", [1e-3, 0.125, 4.0])
def test_scales(device, scale):
    check(paged.Paged([1, 40], [90, 300], 2, 2, 64, F16), scale=scale)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("new", [1, 6, 33, 200])
def test_splits(device, dtype, new):
    """Long enough to be split over work-groups, at every alignment of the end."""
    for length in (2048, 4001):
        p = paged.Paged([new], [length], 2, 1, 64, dtype, 64)
        cache, batch, q = p.cuda(qmm)
        plan = qmm.attention_plan(cache, batch, 2, new, 256)
        assert plan.splits > 1
        check(p)
        check(paged.Paged([new, 0, new], [length, 50, 70], 2, 1, 64, dtype, 64))
        check(p, window=700)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [96, 128, 192, 256])
def test_splits_of_wide_heads(device, dtype, dim):
    for news, lens in (([1], [4001]), ([200, 0, 33], [4001, 50, 70]), ([61, 64], [2048, 3001])):
        p = paged.Paged(news, lens, 4, 2, dim, dtype, 64)
        assert qmm.attention_plan(*p.cuda(qmm)[:2], 4, sum(news), 256).splits > 1
        check(p)
        check(p, window=700)


@gpu
@pytest.mark.parametrize("hints", [dict(max_new=1, max_length=1), dict(max_new=0, max_length=0), dict(max_new=None, max_length=None),
                                   dict(max_new=500, max_length=100000)], ids=str)
def test_hints_only_size_the_launch(device, hints):
    for dim in (64, 256):
        check(paged.Paged([90, 3, 41, 1], [400, 200, 41, 1000], 4, 2, dim, F16), **hints)


def q8_close(p, qact, ref, off):
    n = p.heads * p.dim
    q, dh, s = layouts.read_qact(qact.cpu().numpy(), ref.shape[0], n)
    T = ref.shape[0]
    scale = dh.view(np.float16).astype(np.float64).repeat(32, 1)
    got = torch.from_numpy(q.astype(np.float64) * scale)[:T]
    ref, off = ref.reshape(T, n), off.reshape(T, n)
    top = (ref.abs() + off).unflatten(1, (-1, 32)).amax(2).repeat_interleave(32, 1)
    assert bool(((got - ref).abs() <= off + top / 127 * (0.5 + 2.0 ** -10) + top * 2.0 ** -11).all())
    assert not q[T:].any() and not dh[T:].any() and not s[T:].any()
    sums = (scale[:T, ::32] * q[:T].reshape(T, -1, 32).sum(2)).astype(np.float16)
    assert np.array_equal(sums.view(np.uint16), s[:T])


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_q8_output(device, dtype, dim):
    for news, lens in (([1], [40]), ([1, 0, 1], [40, 9, 3000]), ([70, 3], [90, 33]), ([129], [4000])):
        p = paged.Paged(news, lens, 8, 2, dim, dtype)
        cache, batch, q = p.cuda(qmm)
        nb = qmm.qact_bytes(sum(news), 8 * dim)
        out = torch.full((nb,), 0x55, dtype=torch.uint8, device="cuda")
        got = qmm.attention(q, cache, batch, dtype="q8", out=out)
        torch.cuda.synchronize()
        assert got is out
        q8_close(p, out, *p.reference())
        # the blocks are those of the numbers that the prepass would have
        assert torch.equal(out, qmm.attention(q, cache, batch, dtype="q8"))


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_where_it_is_not_seen(device, dtype, dim, bad):
    """A key and a value late in a sequence that are no numbers: tokens before them have the results that they had; the
    others have none, in the channels of the value and, for the key, in all."""
    for new, length, group in ((5, 50, 1), (70, 100, 2), (150, 400, 1), (20, 3000, 2)):
        for which in ("k", "v"):
            p = paged.Paged([new], [length], 2 * group, 2, dim, dtype)
            cache, batch, q = p.cuda(qmm)
            clean = qmm.attention(q, cache, batch).clone()
            at = new // 2  # the token whose slot is bad
            slot = length - new + at
            page, head = p.where[0][slot // 32], 1
            x = paged.unpacked(cache.k if which == "k" else cache.v, dtype, which, p.n_pages, 2, 32, dim)
            pool = cache.k if which == "k" else cache.v
            if dtype == "q8":  # the block's scale
                b = pool.view(p.n_pages, 2, -1)
                byte = 32 * dim + (0 * 32 + slot % 32) * 2
                bits = int(np.float16(bad).view(np.uint16))
                b[page, head, byte], b[page, head, byte + 1] = bits & 255, bits >> 8
            else:
                x[page, head, slot % 32, 3] = bad
                pool.copy_(paged.packed(x, dtype, which).cuda())
            out = qmm.attention(q, cache, batch)
            torch.cuda.synchronize()
            theirs = slice(group, 2 * group)  # the heads that share cache head 1
            assert torch.equal(out[:, :group], clean[:, :group])
            assert torch.equal(out[:at, theirs], clean[:at, theirs])
            after = out[at:, theirs].float()
            if which == "k":
                if not bad < 0 and not (bad > 0):  # NaN: every token that sees it
                    assert bool(after.isnan().all())
            else:
                width = 32 if dtype == "q8" else 1
                first = 0 if dtype == "q8" else 3
                assert not bool(after[:, :, first:first + width].isfinite().any())
                rest = torch.ones(dim, dtype=torch.bool)
                rest[first:first + width] = False
                assert torch.equal(after[:, :, rest.cuda()], clean[at:, theirs].float()[:, :, rest.cuda()])


@gpu
def test_scores_past_f32(device):
    """Finite inputs whose scores pass f32 in one direction: an infinite score is no number's row."""
    p = paged.Paged([2], [40], 1, 1, 64, BF16)
    p.k[0][:] = 1e30
    p.q[0], p.q[1] = 1e30, -1e30
    cache, batch, q = p.cuda(qmm)
    out = qmm.attention(q, cache, batch)
    torch.cuda.synchronize()
    assert bool(out[0].isnan().all())
    assert not out[1].any()  # every score is -infinity: as if nothing were seen


@gpu
@pytest.mark.parametrize("value", [0.0, 1e-7, 60000.0])
def test_sizes_of_values(device, value):
    """Zeros, f16's subnormal numbers and its largest ones."""
    p = paged.Paged([1, 40], [70, 90], 2, 2, 64, F16)
    for x in p.v:
        x.sign_().mul_(value)
    check(p)


@gpu
def test_rows_of_no_sequence_and_unfit_batches(device):
    p = paged.Paged([37], [100], 4, 2, 64, F16, junk=0.0)
    cache, batch, q = p.cuda(qmm)
    ref = qmm.attention(q, cache, batch)
    for starts, length, table in (([5, 30], 100, None), ([-7, 1000], 100, None), ([30, 5], 100, None), ([0, 37], 10 ** 9, None),
                                  ([0, 37], -5, None), ([0, 37], 100, [[99, -3, 1 << 30, -1]])):
        b = qmm.Batch(torch.tensor(starts, dtype=torch.int32).cuda(), torch.tensor([length], dtype=torch.int32).cuda(),
                      batch.table if table is None else torch.tensor(table, dtype=torch.int32).cuda(), max_new=37, max_length=100)
        out = torch.full((37, 256), 9.0, dtype=F16, device="cuda")
        qmm.attention(q, cache, b, out=out)
        torch.cuda.synchronize()
        rows = range(max(0, starts[0]), min(37, starts[1]))
        is_ = torch.zeros(37, dtype=torch.bool)
        is_[list(rows)] = True
        assert bool((out[~is_.cuda()] == 9).all())
        if starts == [-7, 1000] and length == 100:
            assert torch.equal(out.view(37, 4, 64), ref)
        if table is not None or length < 0:
            assert not out.any()


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
def test_a_page_outside_the_pool_is_not_seen(device, dtype):
    for new in (1, 40):
        p = paged.Paged([new], [160], 2, 2, 64, dtype)
        cache, batch, q = p.cuda(qmm)
        batch.table[0, 1] = 1000  # slots 32 .. 63
        out = qmm.attention(q, cache, batch)
        torch.cuda.synchronize()
        full = p.seen

        def seen(i, causal, window):
            m = full(i, causal, window)
            m[:, 32:64] = False
            return m

        p.seen = seen
        close(out, *p.reference(), p.type)


@gpu
def test_strides(device):
    p = paged.Paged([1, 50], [90, 120], 4, 2, 64, F16)
    cache, batch, q = p.cuda(qmm)
    want = qmm.attention(q, cache, batch)
    T = q.shape[0]
    wide = torch.zeros(T, 4, 128, dtype=F16, device="cuda")
    wide[:, :, :64] = q
    out = torch.full((T, 400), 3.0, dtype=F16, device="cuda")
    qmm.attention(wide[:, :, :64], cache, batch, out=out[:, 16:272])
    turned = qmm.attention(q.transpose(0, 1).contiguous().transpose(0, 1), cache, batch)
    torch.cuda.synchronize()
    assert torch.equal(out[:, 16:272], want.reshape(T, -1)) and torch.equal(turned, want)
    assert bool((out[:, :16] == 3).all()) and bool((out[:, 272:] == 3).all())


@gpu
@pytest.mark.parametrize("new,length", [(1, 4000), (100, 3000), (1, 40)])
def test_streams_and_replayed_graphs(device, new, length):
    """Two graphs that were captured with the same tensors, replayed side by side; what the batch's arrays hold at a replay
    counts."""
    p = paged.Paged([new], [length], 4, 2, 64, F16)
    cache, batch, q = p.cuda(qmm)
    want = qmm.attention(q, cache, batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = qmm.attention(q, cache, batch, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    q2 = torch.randn_like(q)
    want2 = qmm.attention(q2, cache, batch)
    graphs, outs = [], []
    for x in (q, q2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(qmm.attention(x, cache, batch))
    for _ in range(4):
        outs[0].zero_(), outs[1].zero_()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)
    batch.lengths.fill_(length - 7)
    graphs[0].replay()
    eager = qmm.attention(q, cache, batch)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager) and (length <= 7 or not torch.equal(eager, want))


@gpu
def test_work_memory(device):
    p = paged.Paged([1], [4000], 4, 2, 64, F16)
    cache, batch, q = p.cuda(qmm)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    need = qmm.attention_plan(cache, batch, 4, 1, cus).work_bytes
    assert need > 0
    want = qmm.attention(q, cache, batch)
    work = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    got = qmm.attention(q, cache, batch, work=work)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((work[need:] == 0xff).all())
    with pytest.raises(qmm.QmmError, match="work_bytes"):
        qmm.attention(q, cache, batch, work=work[:need - 16])


@gpu
def test_refused_tensors(device):
    p = paged.Paged([2], [40], 4, 2, 64, F16)
    cache, batch, q = p.cuda(qmm)
    for call in (lambda: qmm.attention(q.float(), cache, batch), lambda: qmm.attention(q.to(BF16), cache, batch),
                 lambda: qmm.attention(q[:, :3], cache, batch), lambda: qmm.attention(q[..., :32], cache, batch),
                 lambda: qmm.attention(q.cpu(), cache, batch), lambda: qmm.attention(q, cache, batch, dtype=torch.float32),
                 lambda: qmm.attention(q, cache, batch, out=q.view(2, 256)), lambda: qmm.attention(q[..., ::2], cache, batch),
                 lambda: qmm.attention(q, cache, batch, causal=False, window=3), lambda: qmm.attention(q, cache, batch, scale=-1.0)):
        with pytest.raises(qmm.QmmError):
            call()


@gpu
def test_largest_offsets(device):
    """A pool of more than 4 GiB: its last pages, and positions past 2^17."""
    heads, dim, page = 8, 256, 1024
    n = (9 << 29) // (heads * dim * page * 2) + 1
    cache = qmm.Cache(n, heads, dim, page=page, dtype=F16)
    length = 150_000
    table = torch.zeros(1, -(-length // page), dtype=torch.int32)
    table[0, -1], table[0, -2] = n - 1, n - 2
    batch = qmm.Batch(torch.tensor([0, 2000], dtype=torch.int32).cuda(), torch.tensor([length], dtype=torch.int32).cuda(), table.cuda(),
                      max_length=length)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(2000, heads, dim, device="cuda", generator=g).half()
    v = torch.randn(2000, heads, dim, device="cuda", generator=g).half()
    qmm.rope_cache(cache, batch, k=k, v=v)
    one = qmm.Batch(torch.tensor([0, 1], dtype=torch.int32).cuda(), batch.lengths, batch.table, max_length=length)
    q = torch.randn(1, heads, dim, device="cuda", generator=g).half()
    out = qmm.attention(q, cache, one, window=300)
    s = torch.einsum("hd,jhd->hj", q[0].float(), k[-300:].float()) / 16
    want = torch.einsum("hj,jhd->hd", s.softmax(1), v[-300:].float())
    torch.cuda.synchronize()
    assert float((out[0].float() - want).abs().max()) < 4e-3  # 2^-11 of p and of the result, of values up to about 4
