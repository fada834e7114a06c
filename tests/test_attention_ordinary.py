"""qmm_attention with finite leftovers in the slots that are not in use, so that no result is anything but a finite number
and work-groups do their tiles once: partly filled tiles in every kernel, against the formula in 64 bits with the tolerance of
Paged.reference; and keys that are infinite, whose scores' signs say what comes of them."""
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import paged  # noqa: E402
from tests.test_attention import check, close, q8_close  # noqa: E402

gpu = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
CACHES = [F16, BF16, "q8"]
DIMS = [64, 96, 128, 192, 256]
LEFT = 3.0  # what unused slots hold: numbers, or in q8 blocks the scale of codes of 127


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_causal(device, dtype, dim):
    for news, lens in (([1], [33]), ([5, 1], [70, 31]), ([70], [75]), ([150, 0, 40], [333, 9, 41])):
        p = paged.Paged(news, lens, 4, 2, dim, dtype, junk=LEFT)
        check(p)
        check(p, window=37)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_cross(device, dtype, dim):
    for news in ([1, 1, 1, 1], [40, 3, 90, 17]):
        check(paged.Paged(news, [150, 0, 1, 33], 6, 3, dim, dtype, junk=LEFT), causal=False)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_one_group_of_waves(device, dtype, dim):
    """More work-groups than compute units."""
    n = torch.cuda.get_device_properties(0).multi_processor_count // 4 + 1
    p = paged.Paged([65 + i % 9 for i in range(n)], [90 + 3 * i for i in range(n)], 4, 4, dim, dtype, junk=LEFT)
    check(p)
    check(p, causal=False)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_splits(device, dtype, dim):
    for news, lens in (([1], [4001]), ([200, 0, 33], [4001, 50, 70])):
        p = paged.Paged(news, lens, 4, 2, dim, dtype, junk=LEFT)
        assert qmm.attention_plan(*p.cuda(qmm)[:2], 4, sum(news), 256).splits > 1
        check(p)


@gpu
@pytest.mark.parametrize("dtype", CACHES, ids=str)
@pytest.mark.parametrize("dim", DIMS)
def test_q8_output(device, dtype, dim):
    for news, lens in (([1, 1], [40, 3001]), ([70, 3], [90, 33])):
        p = paged.Paged(news, lens, 8, 2, dim, dtype, junk=LEFT)
        cache, batch, q = p.cuda(qmm)
        out = qmm.attention(q, cache, batch, dtype="q8")
        torch.cuda.synchronize()
        q8_close(p, out, *p.reference())


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("new,length", [(5, 50), (150, 400), (20, 3000)])
def test_infinite_keys(device, dtype, dim, bad, new, length):
    """One infinity in a key: a query whose score of it is +infinity has no numbers, one whose score is -infinity has the
    results of the other keys, and tokens before it have theirs."""
    slot = length - new + new // 2
    p = paged.Paged([new], [length], 2, 2, dim, dtype, junk=LEFT)
    p.q[:, :, 3] = torch.where(p.q[:, :, 3].abs() < 0.01, torch.ones_like(p.q[:, :, 3]), p.q[:, :, 3])  # no 0 times infinity
    cache, batch, q = p.cuda(qmm)
    page = p.where[0][slot // 32]
    x = paged.unpacked(cache.k, dtype, "k", p.n_pages, 2, 32, dim)
    x[page, 1, slot % 32, 3] = bad
    cache.k.copy_(paged.packed(x, dtype, "k").cuda())
    out = qmm.attention(q, cache, batch)
    torch.cuda.synchronize()
    want, off = p.reference()
    full = p.seen

    def seen(i, causal, window):
        m = full(i, causal, window)
        m[:, slot] = False
        return m

    p.seen = seen
    hidden, off_hidden = p.reference()
    sees = torch.arange(length - new, length) >= slot
    above = sees & (p.q[:, 1, 3].double() * bad > 0)
    below = sees & ~above
    assert bool(above.any()) and bool(below.any())
    close(out[:, 0], want[:, 0], off[:, 0], p.type)
    close(out[:, 1][~sees], want[:, 1][~sees], off[:, 1][~sees], p.type)
    close(out[:, 1][below], hidden[:, 1][below], off_hidden[:, 1][below], p.type)
    assert bool(out[:, 1][above].isnan().all())
