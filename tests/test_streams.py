"""New tensors of a call with a stream of its own belong to that stream."""
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402

pytestmark = pytest.mark.gpu


def test_new_tensors_belong_to_the_stream_they_are_written_on(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    h = torch.randn((3, 512), device="cuda")
    weight = torch.ones(512, device="cuda")
    ref = qmm.norm_quantize(h, weight, normed=True)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    seen, empty = [], torch.empty_strided

    def spy(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **k)

    monkeypatch.setattr(torch, "empty_strided", spy)
    for stream, handle in ((0, 0), (torch.cuda.default_stream(), 0), (side, side.cuda_stream),
                           (side.cuda_stream, side.cuda_stream), (None, other.cuda_stream)):
        with torch.cuda.stream(other):
            seen.clear()
            r = qmm.norm_quantize(h, weight, normed=True, stream=stream)
            assert seen == [handle] * 3, stream
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, ref))
