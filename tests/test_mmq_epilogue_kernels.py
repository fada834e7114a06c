"""qmm_mmq_epilogue on either side of the choice between its kernels: bit for bit
qmm_mmq's sums where the tiled kernel runs, within the few-token kernel's tolerance of
the oracle where that one does."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402
from tests.test_mmq_epilogue import U, device, make  # noqa: E402,F401


def few(od, id_, T, cus):
    """The header's "up to 64 tokens, or a launch that small": up to one round of row blocks by token blocks on the GPU's
    compute units, two with rows of up to 8192."""
    blocks = -(-od // 32) * -(-T // 32)
    return T <= 64 or blocks <= cus or (id_ <= 8192 and blocks <= 2 * cus)


CASES = [  # on 256 compute units: the few-token kernel?
    (synth.Q4_K, 2752, 8192, 160, True), (synth.Q4_K, 2752, 8448, 160, False),        # 430 blocks, the row length
    (synth.Q6_K, 1376, 8192, 320, True), (synth.Q6_K, 1376, 11008, 320, False),
    (synth.Q6_K, 4096, 768, 128, True), (synth.Q6_K, 4128, 768, 128, False),          # 512 and 516 blocks
    (synth.Q4_K_PACKED, 2048, 11008, 97, True), (synth.Q4_K_PACKED, 2080, 11008, 97, False),  # 256 and 260
    (synth.Q4_K_PACKED, 8224, 2304, 64, True), (synth.Q4_K_PACKED, 8224, 2304, 65, False),    # the tokens
    (synth.Q6_K, 8224, 8448, 33, True), (synth.Q4_K, 16416, 11008, 32, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("type_,od,id_,T,here", CASES)
def test_sums_of_either_kernel(device, type_, od, id_, T, here):  # noqa: F811
    print(f"{synth.TYPE_NAMES[type_]} {od}x{id_} T={T}", flush=True)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert cus != 256 or few(od, id_, T, cus) == here
    w, qact, raw, x = make(device, type_, od, id_, T, seed=od + T)
    sums = qmm.mmq_epilogue(w, qact, T)
    if not few(od, id_, T, cus):
        assert torch.equal(sums.view(torch.int32), qmm.mmq(w, qact, T).view(torch.int32))
    else:
        rows = min(od, 600)  # the first ones, and the last ones with the rest of the row blocks
        for lo in (0, od - rows):
            at = slice(lo * (raw.size // od), (lo + rows) * (raw.size // od))
            q, dh, s = oracle.quantize(x)
            ref, A = oracle.mmq_parallel(synth.block_format(type_), raw[at], rows, id_, q, dh, s)
            assert np.all(np.abs(sums[:, lo:lo + rows].cpu().numpy() - ref) <= (36 + 2 * (id_ // 256)) * U * A)
    w.release()
