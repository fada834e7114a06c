"""What sizes a launch of qmm_attention: windows past the sequences."""
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
from tests.test_attention import _plan  # noqa: E402

SIZES = [(32, 32, 128, 1, 1, 1, 131072), (32, 8, 128, 1, 1, 1, 3314), (16, 4, 128, 1, 1000, 1000, 131072), (20, 20, 64, 16, 16, 1, 1500),
         (16, 4, 256, 9, 1500, 300, 5000), (8, 8, 96, 1, 1, 1, 1 << 30)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("type_", [1, 3])
def test_windows_past_the_length_plan_as_none(sizes, type_):
    """A window that no sequence reaches, the largest number among them, changes nothing."""
    rc, want = _plan(*sizes, type_=type_)
    assert rc == qmm.OK
    for window in (sizes[-1], sizes[-1] + 1, 1 << 31, 1 << 62, (1 << 63) - 200, (1 << 63) - 1):
        rc, p = _plan(*sizes, type_=type_, window=window)
        assert rc == qmm.OK and bytes(p) == bytes(want), (window, p.splits, want.splits)


@pytest.mark.parametrize("kw", [dict(max_new=-1), dict(max_new=(1 << 20) + 1), dict(max_new=(1 << 64) + 1), dict(max_length=-7),
                                dict(max_length=(1 << 30) + 1), dict(max_length=1 << 64)], ids=str)
def test_hints_out_of_range_are_refused(kw):
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(qmm.QmmError, match=next(iter(kw))):
        qmm.Batch(t, t[:1], t[None, :1], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [-1, 1 << 63, (1 << 64) + 3])
def test_windows_out_of_range_are_refused(window):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    t = torch.tensor([0, 1], dtype=torch.int32).cuda()
    cache, batch = qmm.Cache(1, 2, 64, page=32), qmm.Batch(t, t[1:], t[None, :1])
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    for call in (lambda: qmm.attention(q, cache, batch, window=window),
                 lambda: qmm.attention_plan(cache, batch, 2, 1, 256, window)):
        with pytest.raises(qmm.QmmError, match="window"):
            call()
    assert not bool(qmm.attention(q, cache, batch, window=(1 << 63) - 1).any())
