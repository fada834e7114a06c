"""qmm_attention where tiles, types and masks end: values that are no numbers beside pages outside the pool, leftovers of
a q8 pool, tokens whose scores are all -infinity, keys of small weight.  Tolerances: see each test."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import paged  # noqa: E402
from tests.test_attention import check  # noqa: E402

gpu = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
CACHES = [F16, BF16, "q8"]


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def put(p, pool, which, slot, head, channel, value):
    """Writes a number (q8: the scale of the channel's block) into the first sequence's slot; the channels it reaches."""
    page, at = p.where[0][slot // p.page], slot % p.page
    if p.dtype == "q8":
        byte = at // 32 * 34 * p.dim + 32 * p.dim + (channel // 32 * 32 + at % 32) * 2
        bits = int(np.float16(value).view(np.uint16))
        b = pool.view(p.n_pages, p.kv_heads, -1)
        b[page, head, byte], b[page, head, byte + 1] = bits & 255, bits >> 8
        return slice(channel // 32 * 32, channel // 32 * 32 + 32)
    x = paged.unpacked(pool, p.dtype, which, p.n_pages, p.kv_heads, p.page, p.dim)
    x[page, head, at, channel] = value
    pool.copy_(paged.packed(x, p.dtype, which).to(pool.device))
    return slice(channel, channel + 1)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("new,causal", [(5, True), (70, True), (64, False), (300, True)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite_beside_a_page_outside_the_pool(device, dtype, dim, new, causal, bad):
    """Of two neighbouring pages one is outside the pool, and the other holds a value that is no finite number, which every
    token sees: no token has a finite result in its channel, and all the others are as without it."""
    for missing in (0, 1, 2, 3):
        p = paged.Paged([new], [500], 4, 2, dim, dtype, 32, junk=0.0)
        cache, batch, q = p.cuda(qmm)
        batch.table[0, missing] = p.n_pages
        clean = qmm.attention(q, cache, batch, causal=causal).clone()
        wide = put(p, cache.v, "v", 32 * (missing ^ 1) + 5, 1, 3, bad)
        out = qmm.attention(q, cache, batch, causal=causal)
        torch.cuda.synchronize()
        assert bool(clean.isfinite().all())
        assert not bool(out[:, 2:, wide].isfinite().any()), (missing, out[:, 2:, wide].isfinite().sum())
        out[:, 2:, wide] = clean[:, 2:, wide]
        assert torch.equal(out, clean)


@gpu
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("junk", [60000.0, -600.0])
def test_leftovers_of_a_q8_pool(device, dim, junk):
    """Memory that nothing was stored to: scales whose products with the codes pass f16, in slots that no token sees.  The
    tolerance is that of Paged.reference."""
    for news, lens in (([1], [33]), ([1, 3, 1], [1, 40, 31]), ([1], [4001]), ([40], [90])):
        p = paged.Paged(news, lens, 4, 2, dim, "q8", junk=junk)
        check(p)
        check(p, window=7)
        check(p, causal=False)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 1.0])
def test_no_score_above_minus_infinity(device, dtype, dim, bad):
    """Every key that a token sees has a score of -infinity: zeros, whatever the values are, in every kernel."""
    for new, length in ((1, 40), (5, 70), (70, 100), (150, 333), (1, 4001), (100, 4001)):
        p = paged.Paged([new], [length], 4, 2, dim, dtype, junk=0.0)
        p.k[0][:, :, 0] = -math.inf
        p.q[:, :, 0] = p.q[:, :, 0].abs() + 0.25
        p.v[0][1::3, :, 5] = bad
        cache, batch, q = p.cuda(qmm)
        for causal in (True, False):
            assert not bool(qmm.attention(q, cache, batch, causal=causal).any())
        if 4 * dim % 256 == 0:
            assert not bool(qmm.attention(q, cache, batch, dtype="q8").any())


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("max_length", [30000, 1])
@pytest.mark.parametrize("far", [9.0, 13.0, 18.0, 71.4375, 142.875])
def test_keys_of_small_weight(device, dtype, new, max_length, far):
    """One key far above the many others, as the first of a long context often is, with values of zero: the result is the
    others' weights, exp(-far) each.  With max_length 1 a work-group takes all of the keys.

    Allowed, relative to the weight of the first key: half a step u of the products' type of each weight, and where the
    type's numbers get no finer (f16 below 2^-14 of its range, of which the largest weight takes at least 2^8) 2^-33 for
    each of the n keys; what is below f32's 2^-126 may be zero.  The scores are exact but for scale, its product with
    1/ln 2 and with the score (4 f, f = 2^-24) and their power's rounding (2^-22), n + 64 sums in f32 add
    (n + 64) f; then half a step of the stored result."""
    n, dim = 30000, 64
    p = paged.Paged([new], [n], 2, 1, dim, dtype, 64, junk=0.0)
    p.q[:] = 0.0
    p.q[:, :, 0] = 1.0
    p.k[0][:], p.v[0][:] = 0.0, 127.0 / 128.0  # whole codes of blocks with a scale that f16 holds
    p.k[0][0, :, 0], p.v[0][0] = 127.0 / 16.0, 0.0
    cache, batch, q = p.cuda(qmm, max_length=max_length)
    out = qmm.attention(q, cache, batch, scale=far * 16.0 / 127.0, causal=False).double().cpu()
    rest = (n - 1) * math.exp(-far)
    want, f, u = 127.0 / 128.0 * rest / (1.0 + rest), 2.0 ** -24, paged.HALF[p.type]
    off = want * (u + 2 * (far * 4 * f + 2.0 ** -22) + 2 * (n + 64) * f) + n * (2.0 ** -33 if p.type == F16 else 2.0 ** -126)
    off += paged.HALF[p.type] * (want + off) + (2.0 ** -25 if p.type == F16 else 0.0)
    assert float((out - want).abs().max()) <= off, (float((out - want).abs().max()), off, want)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_queries_that_are_no_numbers(device, dtype, dim, bad):
    """One query with a channel that is no finite number: its own row is no number, and all others keep their bits."""
    for news, lens in (([1, 3], [40, 33]), ([70], [75]), ([40, 5], [90, 3001])):
        p = paged.Paged(news, lens, 4, 2, dim, dtype, junk=3.0)
        cache, batch, q = p.cuda(qmm)
        clean = qmm.attention(q, cache, batch).clone()
        for row in (0, sum(news) - 1):
            x = q.clone()
            x[row, 2, 5] = bad
            out = qmm.attention(x, cache, batch)
            torch.cuda.synchronize()
            own = out[row, 2].clone()
            if bad != bad:
                assert bool(own.isnan().all())
            out[row, 2] = clean[row, 2]
            assert torch.equal(out, clean)
