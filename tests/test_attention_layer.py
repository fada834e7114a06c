"""A layer's attention block run together, as a prefill in chunks and as decode steps run it: norm -> q, k, v products ->
rotary positions and the cache -> attention to q8 blocks -> output product with the residual, against the same chain in 64
bits on the oracle's integers.

Tolerance: the chains differ where a rounding to fewer bits falls on the other side (as in test_layer_operators.py: an f32
error of 1e-6 moves 2.5e-4 of q8 codes by one step of about 3/127: 4e-4 in the 2-norm), and by the attention's 16-bit
operands: keys, values and queries rounded to f16 (2^-11 / sqrt(3) of each, as their rounding in the reference may fall
on the other side only rarely: they are rounded there too), probabilities rounded to f16 (2^-12 on average), which moves
q8 codes of the block's output: an error of 3e-4 of a value moves 127 * 2 * 3e-4 = 8% of codes by a step of 3/127, in the
2-norm 0.28 * 0.024 = 7e-3 of the attention's part of the stream, and with a q8 cache as much again from keys' and values' codes that
fall on the other side.  The residual stream's own part is exact: 1.5e-2 of the block's output bounds the sum."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402
from tests import paged  # noqa: E402

pytestmark = pytest.mark.gpu

WIDTH, HEADS, KV, DIM, PAGE = 512, 8, 2, 64, 32


@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def _weights():
    rng = np.random.default_rng(7)
    shapes = {"q": (synth.Q4_K, HEADS * DIM, WIDTH), "k": (synth.Q4_K, KV * DIM, WIDTH), "v": (synth.Q6_K, KV * DIM, WIDTH),
              "o": (synth.Q4_K, WIDTH, HEADS * DIM)}
    raw = {}
    for name, (t, od, id_) in shapes.items():
        b = synth.weights(rng, t, od, id_).reshape(-1, synth.BLOCK_BYTES[t]).copy()
        for at in ((0, 2) if t == synth.Q4_K else (208,)):  # weights of about 0.04
            d = np.abs(rng.standard_normal(b.shape[0]) * 1.6e-4).astype(np.float16)
            b[:, at:at + 2] = d.view(np.uint8).reshape(-1, 2)
        raw[name] = b.reshape(-1)
    return shapes, raw, (1 + 0.1 * rng.standard_normal(WIDTH)).astype(np.float32)


def _reference(shapes, raw, norm, x, dtype, freq):
    """One sequence at once; x [T][WIDTH] -> (x + block, block)"""
    def product(name, a):
        t, od, id_ = shapes[name]
        return oracle.mmq(t, raw[name], od, id_, *oracle.quantize(np.ascontiguousarray(a.astype(np.float32))))[0]

    x = x.astype(np.float64)
    n = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-5) * norm
    T = x.shape[0]
    q, k, v = (torch.from_numpy(product(s, n).astype(np.float32)).view(T, -1, DIM) for s in "qkv")
    pos = torch.arange(T)
    q = paged.rotated(q, pos, freq, 1.0, "interleaved").half().double()
    k = paged.held(paged.rotated(k, pos, freq, 1.0, "interleaved").float(), dtype)
    v = paged.held(v, dtype)
    out = torch.zeros(T, HEADS, DIM, dtype=torch.float64)
    for h in range(HEADS):
        s = q[:, h] @ k[:, h // (HEADS // KV)].t() / DIM ** 0.5
        s = s.masked_fill(torch.arange(T)[None] > torch.arange(T)[:, None], -np.inf)
        out[:, h] = s.softmax(1) @ v[:, h // (HEADS // KV)]
    y = product("o", out.reshape(T, -1).numpy())
    return x + y, y


class Block:
    def __init__(self, dtype):
        shapes, raw, norm = _weights()
        self.shapes, self.raw, self.norm = shapes, raw, norm
        rows = {synth.Q4_K: qmm.Q4_K_ROWS, synth.Q6_K: qmm.Q6_K_ROWS}
        self.w = {n: qmm.register_weights(t, od, id_, raw[n]) for n, (t, od, id_) in shapes.items()}
        self.rows = {n: qmm.register_weights(rows[t], od, id_, raw[n]) for n, (t, od, id_) in shapes.items()}
        self.gamma = torch.from_numpy(norm).cuda()
        self.freq, self.magnitude = qmm.rope_frequencies(DIM)
        self.cache = qmm.Cache(16, KV, DIM, page=PAGE, dtype=dtype)

    def __call__(self, x, batch):
        """x: cuda f32 [T][WIDTH] -> x + block(x)"""
        T = x.shape[0]
        qact = qmm.norm_quantize(x, self.gamma, h_out=False).qact
        if T <= qmm.MV_MAX_TOKENS:
            q, k, v = (qmm.mmv(self.rows[n], qact, T, dtype=torch.float32) for n in "qkv")
        else:
            q, k, v = (qmm.mmq_epilogue(self.w[n], qact, T) for n in "qkv")
        q = qmm.rope_cache(self.cache, batch, q=q.view(T, HEADS, DIM), k=k.view(T, KV, DIM), v=v.view(T, KV, DIM),
                           frequencies=self.freq, layout="interleaved", dtype=torch.float16)
        out = qmm.attention(q, self.cache, batch, dtype="q8")
        if T <= qmm.MV_MAX_TOKENS:
            return qmm.mmv(self.rows["o"], out, T, residual=x)
        return qmm.mmq_epilogue(self.w["o"], out, T, residual=x)


def _batch(news, lens, table):
    as_int = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    return qmm.Batch(as_int([0] + list(np.cumsum(news))), as_int(lens), table, max_new=max(news), max_length=max(lens))


def _near(got, ref, block):
    off = np.linalg.norm(got.double().cpu().numpy() - ref) / np.linalg.norm(block)
    assert off < 1.5e-2, off


@pytest.mark.parametrize("dtype", [torch.float16, "q8"], ids=str)
def test_prefill_chunks_and_decode_steps(device, dtype):
    b = Block(dtype)
    rng = np.random.default_rng(3)
    lens = [75, 41]
    xs = [rng.standard_normal((n, WIDTH)).astype(np.float32) for n in lens]
    table = torch.tensor([[5, 1, 9], [3, 0, 7]], dtype=torch.int32).cuda()
    refs = [_reference(b.shapes, b.raw, b.norm, x, dtype, b.freq.cpu().numpy()) for x in xs]
    done = [0, 0]
    for news in ([40, 33], [23, 0], [8, 4], [1, 1], [1, 1], [1, 1], [1, 1]):
        x = np.concatenate([x[d:d + n] for x, d, n in zip(xs, done, news)])
        got = b(torch.from_numpy(x).cuda(), _batch(news, [d + n for d, n in zip(done, news)], table))
        torch.cuda.synchronize()
        _near(got, np.concatenate([r[0][d:d + n] for r, d, n in zip(refs, done, news)]),
              np.concatenate([r[1][d:d + n] for r, d, n in zip(refs, done, news)]))
        done = [d + n for d, n in zip(done, news)]
    assert done == lens


def test_a_captured_decode_step(device):
    """One graph for every step: the batch's arrays and the input change between its replays."""
    b, eager = Block(torch.float16), Block(torch.float16)
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((50, WIDTH)).astype(np.float32)).cuda()
    table = torch.tensor([[2, 4]], dtype=torch.int32).cuda()
    prompt = _batch([44], [44], table)
    first = b(x[:44], prompt)
    assert torch.equal(first, eager(x[:44], prompt))
    step = _batch([1], [64], table)  # max_length: as long as it gets
    now = x[44:45].clone()
    step.lengths.fill_(45)
    b(now, step)  # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b(now, step)
    for t in range(44, 50):
        now.copy_(x[t:t + 1])
        step.lengths.fill_(t + 1)
        graph.replay()
        other = _batch([1], [64], table)
        other.lengths.fill_(t + 1)
        want = eager(x[t:t + 1], other)
        torch.cuda.synchronize()
        assert torch.equal(out, want), t
