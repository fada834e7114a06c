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


def overflowing(T, id_, dtype, dev):
    """(rows, the same with rows 1 to 4 whose squares do not add up in f32: an infinity, 3e38, one of 3e19, NaN)"""
    h = torch.randn((T, id_), device=dev, generator=torch.Generator(device=dev).manual_seed(id_)).to(dtype)
    bad = h.clone()
    bad[1, 7] = INF
    bad[2] = torch.where(torch.arange(id_, device=dev) % 2 == 0, 3e38, -3e38).to(dtype)
    bad[3, id_ - 1] = -3e19
    bad[4, 100] = NAN
    return h, bad


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("id_", [256, 768, 9216, 33024])
def test_norm_of_a_row_whose_squares_overflow_is_nan(device, id_, dtype, kind):
    """Every element of it, of the norm before the next block and of the one after the block; other rows keep their
    bits, and a row whose squares just add up is right."""
    T = 7
    print(f"norm {id_} {dtype} {kind}", flush=True)
    h, bad = overflowing(T, id_, dtype, device)
    bad[6] = (bad[6].float() * (1.2e19 / id_ ** 0.5 / bad[6].float().abs().amax())).to(dtype)  # squares below 1.5e38
    weight = 1 + torch.randn(id_, device=device, generator=torch.Generator(device=device).manual_seed(1)) * 0.1
    ref, got = (qmm.norm_quantize(v, weight, kind=kind, normed=True) for v in (h, bad))
    assert torch.equal(got.normed[[0, 5]], ref.normed[[0, 5]])
    assert torch.isnan(got.normed[1:5]).all()
    v = bad[6].double()
    v = v - v.mean() if kind == "layer" else v
    want = v / (v ** 2).mean().sqrt() * weight.double()
    # a sum's roundings (below 120 units of 2^-24 of its terms, at most 10 of a layer norm's mean beside), then half a
    # step of the type
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    assert ((got.normed[6].double() - want).abs() <= 250 * 2.0 ** -24 * (want.abs() + 1) + half * want.abs()).all()
    y = torch.randn((T, id_), device=device, generator=torch.Generator(device=device).manual_seed(2)).to(dtype)
    ref, got = (qmm.norm_quantize(y, weight, y=v, post_weight=weight, kind=kind, normed=True) for v in (h, bad))
    assert torch.equal(got.h[[0, 5]], ref.h[[0, 5]]) and torch.equal(got.normed[[0, 5]], ref.normed[[0, 5]])
    assert torch.isnan(got.h[1:5]).all() and torch.isnan(got.normed[1:5]).all()


def dequantized_blocks(qact, T, n):
    return qmm.dequantize_activations(qact, T, n).reshape(T, -1, 32)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("id_", [256, 768, 9216, 33024])
def test_norm_blocks_of_a_row_that_is_nan(device, id_, kind):
    h, bad = overflowing(7, id_, torch.float32, device)
    weight = torch.ones(id_, device=device)
    ref, got = (dequantized_blocks(qmm.norm_quantize(v, weight, kind=kind).qact, 7, id_) for v in (h, bad))
    assert not torch.isfinite(got[1:5]).any()
    assert torch.equal(got[[0, 5, 6]], ref[[0, 5, 6]])


@pytest.mark.parametrize("value", [NAN, INF, -INF, 1e30], ids=["nan", "inf", "-inf", "1e30"])
@pytest.mark.parametrize("id_", [256, 4096])
def test_blocks_of_activations(device, id_, value):
    """A block with a value that is not finite, or too large for its scale, has a scale that is not finite; the others
    keep their bits; and so does a product of them, of every kernel."""
    T = 13
    x = torch.randn((T, id_), device=device, generator=torch.Generator(device=device).manual_seed(3))
    bad = x.clone()
    bad[4, 77] = value
    bad[12, id_ - 1] = value
    ref, got = (qmm.quantize_activations(v) for v in (x, bad))
    a, b = dequantized_blocks(ref, T, id_), dequantized_blocks(got, T, id_)
    hit = torch.zeros(a.shape[:2], dtype=torch.bool, device=device)
    hit[4, 77 // 32] = hit[12, -1] = True
    assert not torch.isfinite(b[hit]).any() and torch.equal(a[~hit], b[~hit])
    keep = [t for t in range(T) if t not in (4, 12)]
    for type_ in (synth.Q4_K, synth.Q6_K):
        raw = synth.weights(np.random.default_rng(1), type_, 300, id_)
        w, wr = qmm.register_weights(type_, 300, id_, raw), qmm.register_weights(ROWS[type_], 300, id_, raw)
        for name, f in (("mmq", lambda q, v: qmm.mmq(w, q, T)), ("few", lambda q, v: qmm.mmq_epilogue(w, q, T)),
                        ("rows, blocks", lambda q, v: qmm.mmv(wr, q, T)), ("rows", lambda q, v: qmm.mmv(wr, v)),
                        ("rows, f32 of 5", lambda q, v: qmm.mmv(wr, v[8:])),
                        ("rows, of 1", lambda q, v: qmm.mmv(wr, v[12:]))):
            print(id_, value, synth.TYPE_NAMES[type_], name, flush=True)
            r, g = f(ref, x), f(got, bad)
            first = T - r.shape[0]
            for t in range(first, T):
                if t in keep:
                    assert torch.equal(r[t - first], g[t - first]), (name, t)
                else:
                    assert not torch.isfinite(g[t - first]).any(), (name, t)
        w.release()
        wr.release()


@pytest.mark.parametrize("case", [("few", synth.Q4_K, 256, 512, 40), ("tail", synth.Q6_K, 4352, 2048, 509),
                                  ("tiles", synth.Q4_K, 8192, 512, 600), ("rows", synth.Q4_K, 256, 512, 3),
                                  ("rows", synth.Q6_K, 512, 512, 11)], ids=IDS)
def test_blocks_of_a_products_output(device, case):
    """NaN and infinities that an epilogue brings into values kept as q8 blocks show in their blocks, and only there."""
    run, w = product(device, *case)
    od, T = case[2], case[4]
    c = {"mul": torch.randn((T, od), device=device), "residual": torch.randn((T, od), device=device), "scale": 0.25}
    ref = dequantized_blocks(run(dtype="q8", **c), T, od)
    c["mul"][1, 40], c["residual"][T - 1, od - 1], c["residual"][0, 3] = NAN, INF, NAN
    got = dequantized_blocks(run(dtype="q8", **c), T, od)
    hit = torch.zeros(ref.shape[:2], dtype=torch.bool, device=device)
    hit[1, 1] = hit[T - 1, -1] = hit[0, 0] = True
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], ref[~hit])
    w.release()
