"""qmm_rope_frequencies, qmm_rope_cache and qmm_cache_read: formulas and refusals on the CPU; on the GPU against the
formula in 64 bits and the documented layout byte by byte.

Tolerance: with f = 2^-24, sine and cosine of the reduced angle are off by 2 ulp at most, and by 2 pi times half a step of the
reduced turn (f32, at most 1/2, times 2: 2^-24 pi): 8 f of the magnitude in all; their product with the magnitude, two
products and a sum add 3 f of |a| + |b|: 12 f (|a| + |b|) magnitude, and half a step of the type a result is stored in.  A q8
code is off by half a step of its block, dh/2, plus what dh's own rounding leaves out of the largest value."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import paged  # noqa: E402

gpu = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 20


# ---- on the CPU ----

def _fields(name):
    hdr = open(os.path.join(ROOT, "include", "qmm.h")).read()
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} %s;" % name, hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    return re.findall(r"\*?(\w+)\s*[;,]", body)


@pytest.mark.parametrize("name,struct", [("qmm_cache", qmm.CacheStruct), ("qmm_batch", qmm.BatchStruct), ("qmm_rope", qmm.Rope)])
def test_structs_match_header(name, struct):
    assert _fields(name) == [f[0] for f in struct._fields_]


def test_constants_match_header():
    hdr = open(os.path.join(ROOT, "include", "qmm.h")).read()
    c = {k: v for k, v in re.findall(r"#define (QMM_ROPE_[A-Z]+) (\d)", hdr)}
    assert [int(c["QMM_ROPE_" + n]) for n in ("HALF", "INTERLEAVED")] == [qmm.ROPE_LAYOUTS[n] for n in ("half", "interleaved")]
    assert [int(c["QMM_ROPE_" + n]) for n in ("PLAIN", "LINEAR", "BASE", "YARN", "TURNS")] == \
        [qmm.ROPE_SCALINGS[n] for n in ("none", "linear", "base", "yarn", "turns")]


@pytest.mark.parametrize("args,want", [((1, 8, 128, 64), 8 * 64 * 256), ((2, 1, 64, 32), 32 * 128), ((3, 5, 96, 256), 5 * 8 * 34 * 96),
                                       ((0, 8, 128, 64), 0), ((1, 0, 128, 64), 0), ((1, 8, 80, 64), 0), ((1, 8, 128, 48), 0),
                                       ((1, 8, 128, 16), 0), ((1, 4097, 128, 64), 0), ((1, 8, 128, 1 << 17), 0)])
def test_page_bytes(args, want):
    assert qmm._lib.qmm_cache_page_bytes(*args) == want


def _frequencies(n, base=10000.0, scaling=0, factor=1.0, original=4096.0, fast=32.0, slow=1.0):
    f, m = (ctypes.c_double * 128)(), ctypes.c_float()
    rc = qmm._lib.qmm_rope_frequencies(n, base, scaling, factor, original, fast, slow, f, ctypes.byref(m))
    assert rc == 0, qmm.last_error()
    return np.array(f[:n // 2]), m.value


@pytest.mark.parametrize("n", [16, 64, 128, 256])
def test_frequencies(n):
    i = np.arange(n // 2)
    plain = 10000.0 ** (-2 * i / n)
    same = dict(rtol=1e-14, atol=0)
    f, m = _frequencies(n)
    np.testing.assert_allclose(f, plain, **same)
    assert m == 1.0
    np.testing.assert_allclose(_frequencies(n, scaling=1, factor=8.0)[0], plain / 8, **same)
    f, m = _frequencies(n, scaling=2, factor=4.0)
    np.testing.assert_allclose(f[[0, -1]], plain[[0, -1]] / [1, 4], rtol=1e-13)  # the fastest stays, the slowest is divided
    f, m = _frequencies(n, scaling=3, factor=4.0)
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(f[turns >= 32 * 10000 ** (2 / n)], plain[turns >= 32 * 10000 ** (2 / n)], **same)
    np.testing.assert_allclose(f[turns <= 10000 ** (-2 / n)], plain[turns <= 10000 ** (-2 / n)] / 4, **same)
    assert np.all(f <= plain * (1 + 1e-14)) and np.all(f >= plain / 4 * (1 - 1e-14)) and np.all(np.diff(f) < 0)
    assert m == np.float32(0.1 * math.log(4) + 1)
    f, m = _frequencies(n, scaling=4, factor=4.0, original=8192.0, fast=4.0, slow=1.0)
    keep = np.clip((8192 * plain / (2 * math.pi) - 1) / 3, 0, 1)
    np.testing.assert_allclose(f, plain / 4 * (1 - keep) + plain * keep, rtol=1e-13)
    assert m == 1.0


@pytest.mark.parametrize("kw,word", [(dict(n=0), "n_rot"), (dict(n=24), "n_rot"), (dict(n=272), "n_rot"), (dict(base=1.0), "base"),
                                     (dict(base=float("inf")), "base"), (dict(scaling=5), "scaling"), (dict(scaling=-1), "scaling"),
                                     (dict(scaling=1, factor=0.0), "factor"), (dict(scaling=2, factor=float("nan")), "factor"),
                                     (dict(scaling=3, factor=2.0, original=0.0), "original"),
                                     (dict(scaling=4, factor=2.0, fast=1.0), "fast"), (dict(scaling=3, factor=2.0, slow=0.0), "slow")])
def test_frequencies_refused(kw, word):
    a = dict(n=64, base=10000.0, scaling=0, factor=1.0, original=4096.0, fast=32.0, slow=1.0)
    a.update(kw)
    f = (ctypes.c_double * 256)()
    assert qmm._lib.qmm_rope_frequencies(*a.values(), f, None) == qmm.EINVAL
    assert word in qmm.last_error()


def cache_struct(**kw):
    a = dict(type=1, heads=2, head_dim=64, page=32, n_pages=8, k=BASE, v=2 * BASE)
    a.update(kw)
    return qmm.CacheStruct(**a)


def batch_struct(**kw):
    a = dict(n_seq=2, columns=4, starts=3 * BASE, lengths=3 * BASE + 64, table=3 * BASE + 128, table_stride=4, max_new=5,
             max_length=100)
    a.update(kw)
    return qmm.BatchStruct(**a)


CACHE_REFUSED = [(dict(type=0), "type"), (dict(type=4), "type"), (dict(heads=0), "heads"), (dict(heads=5000), "heads"),
                 (dict(head_dim=80), "head_dim"), (dict(head_dim=0), "head_dim"), (dict(page=48), "page"), (dict(page=16), "page"),
                 (dict(page=0), "page"), (dict(n_pages=0), "n_pages"), (dict(n_pages=1 << 31), "n_pages"), (dict(k=None), "NULL"),
                 (dict(v=None), "NULL"), (dict(k=BASE + 8), "aligned")]
BATCH_REFUSED = [(dict(n_seq=0), "n_seq"), (dict(n_seq=1 << 16), "n_seq"), (dict(columns=0), "columns"),
                 (dict(columns=1 << 26, table_stride=1 << 26), "columns"), (dict(table_stride=3), "table_stride"),
                 (dict(table_stride=-4), "table_stride"), (dict(starts=None), "NULL"), (dict(lengths=None), "NULL"),
                 (dict(table=None), "NULL"), (dict(lengths=3 * BASE + 66), "aligned"), (dict(max_new=-1), "max_new"),
                 (dict(max_new=(1 << 20) + 1), "max_new"), (dict(max_length=-1), "max_length"), (dict(max_length=(1 << 30) + 1), "max_length")]
N, H = 5, 4


def rope_struct(**kw):
    a = dict(type=0, out_type=1, q_heads=H, layout=0, n_rot=64, magnitude=1.0, frequencies=4 * BASE, positions=5 * BASE,
             q=6 * BASE, q_stride=H * 64, q_head_stride=64, q_out=7 * BASE, q_out_stride=H * 64, q_out_head_stride=64,
             k=8 * BASE, k_stride=128, k_head_stride=64, v=9 * BASE, v_stride=128, v_head_stride=64)
    a.update(kw)
    return qmm.Rope(**a)


ROPE_REFUSED = [(dict(type=3), "type"), (dict(out_type=3), "out_type"), (dict(q_heads=0), "q_heads"), (dict(layout=2), "layout"),
                (dict(n_rot=24), "n_rot"), (dict(n_rot=80), "n_rot"), (dict(n_rot=-16), "n_rot"), (dict(magnitude=float("nan")), "magnitude"),
                (dict(frequencies=None), "frequencies"), (dict(frequencies=4 * BASE + 4), "aligned"), (dict(positions=5 * BASE + 2), "aligned"),
                (dict(q=None, k=None, v=None), "nothing"), (dict(q_out=None), "q_out"), (dict(q=6 * BASE + 8), "aligned"),
                (dict(q_stride=32), "q's strides"), (dict(q_stride=H * 64 + 4), "q's strides"), (dict(q_head_stride=56), "q's strides"),
                (dict(k_stride=1 << 25), "k's strides"), (dict(v_stride=-128), "v's strides"),
                (dict(q_out_stride=64, q_out_head_stride=64), "on one another"), (dict(q_out=8 * BASE), "overlaps"),
                (dict(q_out=6 * BASE), "overlaps"), (dict(q_out=BASE + 1024), "overlaps"), (dict(k=BASE), "overlaps"),
                (dict(v=2 * BASE + 64), "overlaps"), (dict(q_out=3 * BASE - 64), "overlaps"), (dict(positions=BASE), "overlaps"),
                (dict(frequencies=2 * BASE), "overlaps")]


@pytest.mark.parametrize("kw,word", CACHE_REFUSED + BATCH_REFUSED + ROPE_REFUSED)
def test_rope_refused(kw, word):
    parts = [dict() for _ in range(3)]
    names = [[f[0] for f in s._fields_] for s in (qmm.Rope, qmm.CacheStruct, qmm.BatchStruct)]
    which = 1 if (kw, word) in CACHE_REFUSED else 2 if (kw, word) in BATCH_REFUSED else 0
    assert set(kw) <= set(names[which])
    parts[which] = kw
    rc = qmm._lib.qmm_rope_cache(rope_struct(**parts[0]), cache_struct(**parts[1]), batch_struct(**parts[2]), N, None)
    assert rc == qmm.EINVAL and word in qmm.last_error(), qmm.last_error()


@pytest.mark.parametrize("kw,word", CACHE_REFUSED + BATCH_REFUSED)
def test_read_refused(kw, word):
    c, b = (kw, {}) if (kw, word) in CACHE_REFUSED else ({}, kw)
    rc = qmm._lib.qmm_cache_read(cache_struct(**c), batch_struct(**b), N, 0, 6 * BASE, 7 * BASE, None)
    assert rc == qmm.EINVAL and word in qmm.last_error(), qmm.last_error()


@pytest.mark.parametrize("type_,k,v,word", [(3, 6 * BASE, 7 * BASE, "type"), (0, None, None, "NULL"), (0, 6 * BASE + 4, None, "aligned"),
                                            (0, BASE, None, "overlaps"), (0, None, 2 * BASE, "overlaps"), (0, 3 * BASE, None, "overlaps"),
                                            (0, 6 * BASE, 6 * BASE + 16, "overlaps")])
def test_read_outputs_refused(type_, k, v, word):
    assert qmm._lib.qmm_cache_read(cache_struct(), batch_struct(), N, type_, k, v, None) == qmm.EINVAL
    assert word in qmm.last_error()


@pytest.mark.parametrize("n_tok", [-1, (1 << 20) + 1])
def test_token_counts_refused(n_tok):
    assert qmm._lib.qmm_rope_cache(rope_struct(), cache_struct(), batch_struct(), n_tok, None) == qmm.EINVAL
    assert qmm._lib.qmm_cache_read(cache_struct(), batch_struct(), n_tok, 0, 6 * BASE, None, None) == qmm.EINVAL


def test_null_structs_refused():
    assert qmm._lib.qmm_rope_cache(None, cache_struct(), batch_struct(), N, None) == qmm.EINVAL
    assert qmm._lib.qmm_rope_cache(rope_struct(), None, batch_struct(), N, None) == qmm.EINVAL
    assert qmm._lib.qmm_rope_cache(rope_struct(), cache_struct(), None, N, None) == qmm.EINVAL


def test_empty_batch():
    assert qmm._lib.qmm_rope_cache(rope_struct(q=None, k=None, v=None), cache_struct(k=None, v=None), batch_struct(), 0, None) == qmm.OK
    assert qmm._lib.qmm_cache_read(cache_struct(), batch_struct(), 0, 0, None, None, None) == qmm.OK


def test_binding_refuses_on_the_cpu():
    with pytest.raises(qmm.QmmError):
        qmm.Cache(4, 2, 80, device="cpu")
    with pytest.raises(qmm.QmmError):
        qmm.Cache(0, 2, 64, device="cpu")
    with pytest.raises(qmm.QmmError):
        qmm.rope_frequencies(64, scaling="other", device="cpu")
    f, m = qmm.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and m == 1.0
    cache = qmm.Cache(4, 2, 64, page=32, device="cpu")
    assert cache.k.numel() == 4 * 2 * 32 * 64 * 2
    with pytest.raises(qmm.QmmError):
        qmm.Batch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("page,dim", [(32, 64), (64, 96), (128, 256)])
def test_views_follow_the_layout(dtype, page, dim):
    n, heads = 3, 2
    x = torch.randn(n, heads, page, dim).to(dtype)
    cache = qmm.Cache(n, heads, dim, page=page, dtype=dtype, k=paged.packed(x, dtype, "k"), v=paged.packed(x, dtype, "v"))
    for view in cache.views():
        assert torch.equal(view.reshape(n, heads, page, dim), x)


# ---- on the GPU ----

@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def near(got, ref, size, type_, what):
    allowed = 12 * 2.0 ** -24 * size + paged.HALF[type_] * (ref.abs() + 12 * 2.0 ** -24 * size)
    if type_ == F16:
        allowed = allowed + 2.0 ** -25
    wrong = (got.double().cpu() - ref).abs() - allowed
    assert bool((wrong <= 0).all()), (what, float(wrong.max()))


def pairs_size(x, n, magnitude, layout):
    """|a| + |b| of each channel's pair, times the magnitude where it turns."""
    a = x.double().abs()
    y = torch.zeros_like(a)
    if layout == "half":
        both = a[..., :n // 2] + a[..., n // 2:n]
        y[..., :n] = torch.cat([both, both], -1)
    else:
        both = a[..., 0:n:2] + a[..., 1:n:2]
        y[..., :n] = both.repeat_interleave(2, -1)
    return y * abs(magnitude)


def run(device, news, lens, heads, kv_heads, dim, dtype, x_type, n_rot, layout, page=32, magnitude=1.0, far=None, out_type=None,
        q=True, k=True, v=True, seed=0, **hints):
    """One call against the formula; every other byte of the pools has to stay."""
    p = paged.Paged(news, lens, heads, kv_heads, dim, dtype, page, seed)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(news)
    xs = {"q": torch.randn(T, heads, dim, generator=g).to(x_type), "k": torch.randn(T, kv_heads, dim, generator=g).to(x_type),
          "v": torch.randn(T, kv_heads, dim, generator=g).to(x_type)}
    cache, batch, _ = p.cuda(qmm, **hints)
    before = cache.k.clone(), cache.v.clone()
    slots = torch.cat([torch.arange(n - m, n) for m, n in zip(news, lens)])
    pos = slots if far is None else torch.randint(far, far + 1000, (T,), generator=g)
    freq, _ = _frequencies(n_rot) if n_rot else (None, None)
    given = {n: xs[n].cuda() for n, is_ in (("q", q), ("k", k), ("v", v)) if is_}
    out = qmm.rope_cache(cache, batch, **given, frequencies=None if freq is None else torch.tensor(freq).cuda(), magnitude=magnitude,
                         layout=layout, positions=None if far is None else pos.to(torch.int32).cuda(), dtype=out_type)
    torch.cuda.synchronize()
    ref = {n: paged.rotated(x, pos, freq, magnitude, layout) if n != "v" and n_rot else x.double() for n, x in xs.items()}
    size = {n: pairs_size(x, n_rot, magnitude, layout) if n != "v" else torch.zeros_like(x, dtype=torch.float64) for n, x in xs.items()}
    if q:
        near(out, ref["q"], size["q"], out.dtype, "q")
    seq = torch.cat([torch.full((m,), i) for i, m in enumerate(news)])
    places = [(p.where[i][s // page], s % page) for i, s in zip(seq.tolist(), slots.tolist())]
    for n, pool, old, there in (("k", cache.k, before[0], k), ("v", cache.v, before[1], v)):
        got = paged.unpacked(pool, dtype, n, p.n_pages, kv_heads, page, dim)
        was = paged.unpacked(old, dtype, n, p.n_pages, kv_heads, page, dim)
        if there:
            at = torch.tensor(places, dtype=torch.long).reshape(-1, 2)
            new = got[at[:, 0], :, at[:, 1]]
            if dtype == "q8":
                off = 12 * 2.0 ** -24 * size[n]
                top = (ref[n].abs() + off).unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
                assert bool(((new.double() - ref[n]).abs() <= off + top / 127 * (0.5 + 2.0 ** -10) + top * 2.0 ** -10 / 2).all()), n
                if n == "v":  # nothing turns: the format's numbers exactly
                    qq, ss = paged.quantized(xs[n].float())
                    assert torch.equal(new, (qq.unflatten(-1, (-1, 32)).float() * ss.float().unsqueeze(-1)).flatten(-2))
            else:
                near(new, ref[n], size[n], dtype, n)
            got[at[:, 0], :, at[:, 1]] = was[at[:, 0], :, at[:, 1]]
        assert torch.equal(got.nan_to_num(7.0), was.nan_to_num(7.0)), "other slots of " + n
    return p, cache, batch, xs


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16, "q8"], ids=str)
@pytest.mark.parametrize("x_type", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,n_rot", [(64, 64), (96, 16), (128, 128), (128, 64), (192, 96), (256, 256), (64, 0)])
def test_types_layouts_and_parts(device, dtype, x_type, layout, dim, n_rot):
    run(device, [3, 1, 0, 37], [3, 50, 20, 70], 5, 2, dim, dtype, x_type, n_rot, layout, magnitude=1.0 if n_rot % 64 else 1.25)


@gpu
@pytest.mark.parametrize("page", [32, 64, 256])
def test_pages_and_odd_lengths(device, page):
    run(device, [1, 15, 16, 17, 33, 100], [1, 15, 300, 129, 257, 700], 3, 3, 64, F16, F16, 64, "half", page=page)
    run(device, [1, 15, 16, 17, 33, 100], [1, 15, 300, 129, 257, 700], 3, 3, 64, "q8", F16, 64, "half", page=page)


@gpu
@pytest.mark.parametrize("dtype", [F16, "q8"], ids=str)
@pytest.mark.parametrize("given", ["q", "k", "v", "kv", "qv"])
def test_parts_by_themselves(device, dtype, given):
    run(device, [5, 40], [9, 77], 4, 2, 128, dtype, F32, 128, "interleaved", **{n: n in given for n in "qkv"})


@gpu
@pytest.mark.parametrize("far", [5, 100_000, 2_000_000_000])
def test_positions(device, far):
    run(device, [7, 30], [40, 64], 2, 1, 128, F16, F32, 128, "half", far=far, out_type=F32)


@gpu
def test_many_heads_and_tokens(device):
    run(device, [700], [733], 33, 11, 64, BF16, BF16, 64, "half", page=64)
    run(device, [1], [1], 71, 1, 64, F16, F16, 64, "interleaved")


@gpu
@pytest.mark.parametrize("hints", [dict(max_new=1, max_length=1), dict(max_new=0, max_length=0), dict(max_new=None, max_length=None)])
def test_hints_only_size_the_launch(device, hints):
    run(device, [90, 3, 41], [100, 200, 41], 2, 2, 64, F16, F16, 32, "half", **hints)
    run(device, [90, 3, 41], [100, 200, 41], 2, 2, 64, "q8", F16, 32, "half", **hints)


def _call(device, T=37, heads=4, kv_heads=2, dim=64, dtype=F16):
    p = paged.Paged([T], [T + 5], heads, kv_heads, dim, dtype)
    cache, batch, _ = p.cuda(qmm)
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(T, h, dim, generator=g).half().cuda() for h in (heads, kv_heads, kv_heads)]
    f, _ = qmm.rope_frequencies(dim)
    return p, cache, batch, xs, f


@gpu
def test_strides_and_in_place(device):
    p, cache, batch, (q, k, v), f = _call(device)
    start = cache.k.clone(), cache.v.clone()
    want = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f)
    pools = cache.k.clone(), cache.v.clone()
    # q, k and v as columns of one joint product, tokens and heads exchanged, in place
    T = q.shape[0]
    joint = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], 1)
    jq, jk, jv = (joint[:, a:b].unflatten(1, (-1, 64)) for a, b in ((0, 256), (256, 384), (384, 512)))
    cache.k.copy_(start[0]), cache.v.copy_(start[1])
    before = joint.clone()
    out = qmm.rope_cache(cache, batch, q=jq, k=jk, v=jv, frequencies=f, out=jq)
    torch.cuda.synchronize()
    assert out is jq and torch.equal(jq, want) and torch.equal(joint[:, 256:], before[:, 256:])
    assert torch.equal(cache.k, pools[0]) and torch.equal(cache.v, pools[1])
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert turned.stride(0) == 64
    wide = torch.full((T, 4, 128), 5.0, dtype=F16, device="cuda")
    out = qmm.rope_cache(cache, batch, q=turned, frequencies=f, out=wide[:, :, :64])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool((wide[:, :, 64:] == 5).all())


@gpu
def test_rows_of_no_sequence_and_unfit_batches(device):
    p, cache, batch, (q, k, v), f = _call(device)
    want = qmm.rope_cache(cache, batch, q=q, frequencies=f)
    for starts, length, table, rows, kept in (
            ([5, 30], 42, None, range(5, 30), True),          # rows before and behind the sequence
            ([-7, 1000], 42, None, range(0, 37), True),       # taken within the call
            ([30, 5], 42, None, [], False),                   # going down: no tokens
            ([0, 37], 10, None, range(0, 37), True),          # tokens without a slot: 27 of them
            ([0, 37], 10 ** 9, None, range(0, 37), True),     # more than the table has
            ([0, 37], 42, [[99, -3]], range(0, 37), False)):  # pages outside the pool
        b = qmm.Batch(torch.tensor(starts, dtype=torch.int32).cuda(), torch.tensor([length], dtype=torch.int32).cuda(),
                      batch.table if table is None else torch.tensor(table, dtype=torch.int32).cuda(), max_new=37, max_length=42)
        cache.k.zero_(), cache.v.zero_()
        out = torch.full_like(q, 9.0)
        pos = torch.arange(5, 42, dtype=torch.int32).cuda()
        qmm.rope_cache(cache, b, q=q, k=k, v=v, frequencies=f, positions=pos, out=out)
        torch.cuda.synchronize()
        is_ = torch.zeros(37, dtype=torch.bool)
        is_[list(rows)] = True
        assert torch.equal(out[is_.cuda()], want[is_.cuda()]) and bool((out[~is_.cuda()] == 9).all())
        slots = paged.unpacked(cache.v, F16, "v", p.n_pages, 2, 32, 64).abs().amax((1, 3)) > 0
        assert int(slots.sum()) == (0 if not kept else min(len(list(rows)), length)), (starts, length)
        k2, v2 = qmm.cache_read(cache, b, 37, dtype=F16)
        torch.cuda.synchronize()
        if kept and length <= 42:
            has = torch.tensor([r for i, r in enumerate(rows) if length - len(rows) + i >= 0])
            assert torch.equal(v2[has.cuda()], v[has.cuda()])
            none = torch.tensor([r for i, r in enumerate(rows) if length - len(rows) + i < 0], dtype=torch.long)
            assert not v2[none.cuda()].any()
        elif table is not None:
            assert not v2.any() and not k2.any()


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16, "q8"], ids=str)
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=str)
def test_read(device, dtype, out):
    p, cache, batch, xs = run(device, [0, 33, 5], [10, 33, 60], 2, 3, 96, dtype, F32, 32, "half")
    k, v = qmm.cache_read(cache, batch, 38, dtype=out)
    torch.cuda.synchronize()
    for got, pool, n in ((k, cache.k, "k"), (v, cache.v, "v")):
        there = paged.unpacked(pool, dtype, n, p.n_pages, 3, 32, 96)
        want = torch.cat([there[p.where[i][s // 32], :, s % 32][None] for i, (m, l) in enumerate(zip(p.news, p.lens))
                          for s in range(l - m, l)])
        assert torch.equal(got.cpu(), want.to(out))


@gpu
def test_not_finite_stays_where_it_is(device):
    p, cache, batch, (q, k, v), f = _call(device, dtype="q8")
    q[3, 1, 7], k[4, 0, 9], v[5, 1, 40] = float("inf"), float("nan"), float("-inf")
    out = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f, dtype=F32)
    kk, vv = qmm.cache_read(cache, batch, 37)
    torch.cuda.synchronize()
    bad = (~out.isfinite()).nonzero().tolist()
    assert bad == [[3, 1, 7], [3, 1, 39]]
    for got, at in ((kk, (4, 0)), (vv, (5, 1))):
        fine = got.isfinite().all(2)
        assert not fine[at] and int((~fine).sum()) == 1


@gpu
def test_largest_offsets(device):
    """A pool of more than 4 GiB: its last page."""
    heads, dim, page = 8, 256, 1024
    n = (9 << 29) // (heads * dim * page * 2) + 1
    cache = qmm.Cache(n, heads, dim, page=page, dtype=F16)
    assert cache.k.numel() > 1 << 32
    batch = qmm.Batch(torch.tensor([0, 3], dtype=torch.int32).cuda(), torch.tensor([1024], dtype=torch.int32).cuda(),
                      torch.tensor([[n - 1]], dtype=torch.int32).cuda())
    x = torch.randn(3, heads, dim).half().cuda()
    qmm.rope_cache(cache, batch, k=x, v=x)
    k, v = qmm.cache_read(cache, batch, 3, dtype=F16)
    torch.cuda.synchronize()
    assert torch.equal(k, x) and torch.equal(v, x)
    tail = heads * dim * page * 2
    assert int(cache.k[:-tail].count_nonzero()) == 0 and int(cache.k[-tail:].count_nonzero()) > 0


@gpu
def test_other_stream_and_replayed_graph(device):
    p, cache, batch, (q, k, v), f = _call(device)
    want = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qmm.rope_cache(cache, batch, q=q, k=k, v=v, frequencies=f)
    for shift in (0, 1, 2):  # what the batch's arrays hold when it is replayed counts
        batch.lengths.fill_(42 - shift)
        cache.k.zero_(), cache.v.zero_(), out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        again = qmm.Cache(p.n_pages, 2, 64, page=32, dtype=F16)
        eager = qmm.rope_cache(again, batch, q=q, k=k, v=v, frequencies=f)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(cache.k, again.k) and torch.equal(cache.v, again.v)
        assert (shift == 0) == torch.equal(out, want)
