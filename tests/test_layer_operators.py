"""The operators of a layer run together, as a prefill and as decode steps run them:
norm -> gate and up products (the up one kept as q8 blocks) -> down product with the
residual -> norms after the block and before the next, against the same chain in 64
bits on the oracle's integers.

Tolerance: every stage is within f32 rounding of its formula, so the chains differ
where a rounding to fewer bits falls on the other side.  An f32 error of 1e-6 of a
value moves a q8 code (127 steps per block) for at most 2*127*1e-6 = 2.5e-4 of the
values, each by one step, about 3/127 of the values' size: 4e-4 in the 2-norm; an f16
value for 2*2^11*1e-6 = 4e-3 of them, by 2^-11: 3e-5.  Three roundings to q8 and two
to 16 bits follow one another: 2e-3, and one code's step, amplified by the largest
weight, for any single element: 0.05 of the 2-norm's size per element."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu

WIDTH, FFN = 768, 1280
ROWS = {synth.Q4_K: qmm.Q4_K_ROWS, synth.Q6_K: qmm.Q6_K_ROWS}


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def _weights(seed):
    rng = np.random.default_rng(seed)
    shapes = {"gate": (synth.Q4_K, FFN, WIDTH), "up": (synth.Q4_K, FFN, WIDTH), "down": (synth.Q6_K, WIDTH, FFN)}
    raw = {}
    for name, (t, od, id_) in shapes.items():
        b = synth.weights(rng, t, od, id_).reshape(-1, synth.BLOCK_BYTES[t]).copy()
        for at in ((0, 2) if t == synth.Q4_K else (208,)):  # weights of about 0.02
            d = np.abs(rng.standard_normal(b.shape[0]) * 8e-5).astype(np.float16)
            b[:, at:at + 2] = d.view(np.uint8).reshape(-1, 2)
        raw[name] = b.reshape(-1)
    vec = lambda n, by, at=0.0: (at + by * rng.standard_normal(n)).astype(np.float32)  # noqa: E731
    return shapes, raw, {"norm": vec(WIDTH, 0.1, 1), "post": vec(WIDTH, 0.1, 1), "next": vec(WIDTH, 0.1, 1),
                         "gate": vec(WIDTH, 0.5), "bias": vec(FFN, 0.3)}


def _reference(shapes, raw, v, h):
    """The chain in 64 bits; the stream and the gate's output are kept in f16, products' inputs as q8 blocks."""
    def norm(x, w):
        return x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-5) * w.astype(np.float64)

    def product(name, x):
        q, dh, s = oracle.quantize(np.ascontiguousarray(x.astype(np.float32)))
        t, od, id_ = shapes[name]
        return oracle.mmq(t, raw[name], od, id_, q, dh, s)[0]

    f16 = lambda x: x.astype(np.float16).astype(np.float64)  # noqa: E731
    h = h.astype(np.float64)
    n = norm(h, v["norm"])
    g = product("gate", n) + v["bias"]
    g = f16(g / (1 + np.exp(-g)))
    y = f16(product("down", product("up", n) * g))
    h = f16(0.5 * h + 0.8 * norm(y, v["post"]) * f16(v["gate"]))
    return h, norm(h, v["next"])


def _close(got, ref, what):
    got = got.double().cpu().numpy()
    rms = np.linalg.norm(ref) / np.sqrt(ref.size)
    rel, worst = np.linalg.norm(got - ref) / np.linalg.norm(ref), np.abs(got - ref).max() / rms
    print(f"{what}: rel {rel:.2e}, worst {worst:.2e} of the rms", flush=True)
    assert rel <= 2e-3 and worst <= 0.05


def _prefill(w, v, h, stream=None, out=None):
    T = h.shape[0]
    a = qmm.norm_quantize(h, v["norm"], h_out=False, stream=stream)
    g = qmm.mmq_epilogue(w["gate"], a.qact, T, bias=v["bias"], act="silu", dtype=torch.float16, stream=stream)
    u = qmm.mmq_epilogue(w["up"], a.qact, T, mul=g, dtype="q8", stream=stream)
    y = qmm.mmq_epilogue(w["down"], u, T, dtype=torch.float16, stream=stream)
    return qmm.norm_quantize(h, v["next"], y=y, post_weight=v["post"], gate=v["gate"].half(), residual_scale=0.5,
                             block_scale=0.8, normed=True, stream=stream)


def _decode(w, v, h, from_q8):
    T = h.shape[0]
    a = qmm.norm_quantize(h, v["norm"], h_out=False, normed=not from_q8, qact=from_q8)
    x = (a.qact, T) if from_q8 else (a.normed,)
    g = qmm.mmv(w["gate"], *x, bias=v["bias"], act="silu", dtype=torch.float16)
    if from_q8:  # q8 blocks from the first norm to the down product
        y = qmm.mmv(w["down"], qmm.mmv(w["up"], *x, mul=g, dtype="q8"), T, dtype=torch.float16)
    else:
        y = qmm.mmv(w["down"], qmm.mmv(w["up"], *x, mul=g), dtype=torch.float16)
    return qmm.norm_quantize(h, v["next"], y=y, post_weight=v["post"], gate=v["gate"].half(), residual_scale=0.5,
                             block_scale=0.8, normed=True, qact=False)


@pytest.mark.parametrize("T", [1, 5, 130, 700])
def test_prefill_chain(device, T):
    shapes, raw, v = _weights(1)
    h = np.random.default_rng(T).standard_normal((T, WIDTH)).astype(np.float16)
    ref_h, ref_n = _reference(shapes, raw, v, h)
    w = {k: qmm.register_weights(t, od, id_, raw[k]) for k, (t, od, id_) in shapes.items()}
    vt = {k: torch.from_numpy(x).to(device) for k, x in v.items()}
    r = _prefill(w, vt, torch.from_numpy(h).to(device))
    _close(r.h, ref_h, "stream")
    _close(r.normed, ref_n, "norm")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = _prefill(w, vt, torch.from_numpy(h).to(device), stream=side)  # the whole chain on another stream
    side.synchronize()
    for a, b in zip(r, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("from_q8", [True, False], ids=["q8", "numbers"])
@pytest.mark.parametrize("T", [1, 3, 8, 16])
def test_decode_chain(device, T, from_q8):
    """From q8 blocks the first products see the prefill's numbers.  From the stream's f16 numbers they see
    another rounding before the quantization: f16 moves a value by 2^-12 of itself in the mean, a code by
    127*2^-12 of a step, so about 3% of the codes fall on the other side: sqrt(0.03)*3/127 = 4e-3 more."""
    shapes, raw, v = _weights(2)
    h = np.random.default_rng(T).standard_normal((T, WIDTH)).astype(np.float16)
    ref_h, ref_n = _reference(shapes, raw, v, h)
    w = {k: qmm.register_weights(ROWS[t], od, id_, raw[k]) for k, (t, od, id_) in shapes.items()}
    vt = {k: torch.from_numpy(x).to(device) for k, x in v.items()}
    r = _decode(w, vt, torch.from_numpy(h).to(device), from_q8)
    if from_q8:
        _close(r.h, ref_h, "stream")
        _close(r.normed, ref_n, "norm")
    else:
        rel = np.linalg.norm(r.h.double().cpu().numpy() - ref_h) / np.linalg.norm(ref_h)
        assert rel <= 8e-3


def test_decode_step_in_a_graph(device):
    """A decode step captured once and replayed on new streams of numbers, the residual stream updated in place."""
    T = 4
    shapes, raw, v = _weights(3)
    w = {k: qmm.register_weights(ROWS[t], od, id_, raw[k]) for k, (t, od, id_) in shapes.items()}
    vt = {k: torch.from_numpy(x).to(device) for k, x in v.items()}
    gate = vt["gate"].half()
    h = torch.zeros((T, WIDTH), dtype=torch.float16, device=device)
    qact = torch.empty(qmm.qact_bytes(T, WIDTH), dtype=torch.uint8, device=device)
    g, y = (torch.empty((T, n), dtype=torch.float16, device=device) for n in (FFN, WIDTH))
    u = torch.empty((T, FFN), device=device)

    def step():
        qmm.norm_quantize(h, vt["norm"], h_out=False, qact=qact)
        qmm.mmv(w["gate"], qact, T, bias=vt["bias"], act="silu", out=g)
        qmm.mmv(w["up"], qact, T, mul=g, out=u)
        qmm.mmv(w["down"], u, out=y)
        qmm.norm_quantize(h, vt["next"], y=y, post_weight=vt["post"], gate=gate, residual_scale=0.5, block_scale=0.8,
                          h_out=h, qact=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        start = torch.randn((T, WIDTH), device=device, generator=torch.Generator(device=device).manual_seed(i)).half()
        h.copy_(start)
        step()
        step()  # two steps in a row on the updated stream
        want = h.clone()
        h.copy_(start)
        for t in (qact, g, u, y):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want), f"replay {i}"
    del graph
