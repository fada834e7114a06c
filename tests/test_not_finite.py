"""NaN and infinities: what they reach shows them, nothing else changes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu
ROWS = {synth.Q4_K: qmm.Q4_K_ROWS, synth.Q6_K: qmm.Q6_K_ROWS}
NAN, INF = float("nan"), float("inf")


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


# a product of each kernel: few tokens on the planes, tiles with a split tail, many tiles, few tokens on the rows form
PRODUCTS = [("few", synth.Q4_K, 96, 512, 40), ("tail", synth.Q6_K, 4352, 2048, 509), ("tiles", synth.Q4_K, 8192, 512, 600),
            ("rows", synth.Q4_K, 96, 512, 3), ("rows", synth.Q6_K, 96, 512, 11)]
IDS = [f"{p[0]}-{synth.TYPE_NAMES[p[1]]}" for p in PRODUCTS]


def product(dev, kind, type_, od, id_, T):
    """(the product as a function of its epilogue, its handle)"""
    raw, x = synth.case(type_, od, id_, T, seed=od + T)
    x = torch.from_numpy(x).to(dev)
    if kind == "rows":
        w = qmm.register_weights(ROWS[type_], od, id_, raw)
        return (lambda **ep: qmm.mmv(w, x, **ep)), w
    w, qact = qmm.register_weights(type_, od, id_, raw), qmm.quantize_activations(x)
    return (lambda **ep: qmm.mmq_epilogue(w, qact, T, **ep)), w


@pytest.mark.parametrize("case", PRODUCTS, ids=IDS)
def test_every_activation_keeps_nan_and_infinity(device, case):
    run, w = product(device, *case)
    od = case[2]
    bias = torch.randn(od, device=device, generator=torch.Generator(device=device).manual_seed(1))
    bad = bias.clone()
    bad[5], bad[od - 1], bad[40] = NAN, INF, -INF
    keep = torch.ones(od, dtype=torch.bool, device=device)
    keep[[5, od - 1, 40]] = False
    for act in qmm.ACTS:
        print(case[0], act, flush=True)
        ref, got = run(bias=bias, act=act), run(bias=bad, act=act)
        assert torch.equal(got[:, keep], ref[:, keep])
        assert torch.isnan(got[:, 5]).all(), act
        assert (got[:, od - 1] == INF).all(), act
        if act in ("none", "relu"):
            assert (got[:, 40] == (-INF if act == "none" else 0)).all(), act
    w.release()
