"""qmm_norm_quantize and qmm_dequantize_activations: refusals on the CPU; on the GPU
against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32; a sum of m terms
added in a depth of D additions is off by at most D*u*sum|terms|):
  * the mean square is off by at most D + 3 roundings, 1/sqrt of it by half of that
    and rsqrt's own ulp; the three products add three: K = D/2 + 8 units of u on n;
  * the layer norm's mean is off by D + 2 units of mean|x|, and that times
    rstd*weight on n, beside the subtraction's own rounding;
  * a stored value is off by another half step of its type (f16: 2^-25 below its normal range).
D is 4 per group of four a thread adds, 6 over the wave, 16 over the waves."""
import ctypes
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
from tests import layouts  # noqa: E402

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half a step below the normal range
TYPES = [torch.float32, torch.float16, torch.bfloat16]
gpu = pytest.mark.gpu


# ---- on the CPU: structs and refusals ----

def test_norm_struct_matches_header():
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmm.h")).read()
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} qmm_norm;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    assert re.findall(r"(\w+)\s*;", body) == [f[0] for f in qmm.Norm._fields_]
    assert int(re.search(r"#define QMM_NORM_LAYER (\d)", hdr).group(1)) == qmm.NORM_KINDS["layer"]


BASE = 1 << 20


def _args(**kw):
    n, id_ = 4, 512
    a = dict(type=0, kind=0, eps=1e-5, residual_scale=1.0, block_scale=1.0, h=BASE, h_stride=id_, y=2 * BASE, y_stride=id_,
             weight=3 * BASE, h_out=4 * BASE, h_out_stride=id_, normed=5 * BASE, normed_stride=id_, qact=6 * BASE,
             qact_bytes=qmm.qact_bytes(n, id_))
    a.update(kw)
    return qmm.Norm(**a)


REFUSED = [
    (dict(type=3), "type"), (dict(type=-1), "type"), (dict(kind=2), "kind"), (dict(eps=0.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(residual_scale=float("inf")), "finite"),
    (dict(block_scale=float("nan")), "finite"), (dict(h=None), "NULL"), (dict(weight=None), "NULL"),
    (dict(h=BASE + 8), "aligned"), (dict(y=2 * BASE + 4), "aligned"), (dict(weight=3 * BASE + 4), "aligned"),
    (dict(qact=6 * BASE + 8), "aligned"), (dict(h_stride=508), "h_stride"), (dict(y_stride=0), "y_stride"),
    (dict(h_stride=514), "h_stride"), (dict(h_out_stride=-512), "h_out_stride"), (dict(normed_stride=1 << 25), "stride"),
    (dict(qact_bytes=16), "qact_bytes"), (dict(qact=None), "qact_bytes"),
    (dict(h_out=None, normed=None, qact=None, qact_bytes=0), "no output"),
    (dict(y=None, post_weight=7 * BASE), "need y"), (dict(y=None, gate=7 * BASE), "need y"),
    (dict(post_bias=7 * BASE), "post_weight"), (dict(gate=7 * BASE, gate_stride=256), "gate_stride"),
    (dict(normed=4 * BASE), "overlaps"), (dict(normed=4 * BASE + 64), "overlaps"),
    (dict(h_out=BASE + 16), "overlaps h"), (dict(h_out=BASE, h_out_stride=516), "overlaps h"),
    (dict(normed=BASE), "overlaps h"), (dict(h_out=2 * BASE + 2048), "overlaps y"), (dict(qact=BASE), "overlaps h"),
    (dict(qact=2 * BASE), "overlaps y"), (dict(h_out=3 * BASE - 2048), "overlaps weight"),
    (dict(gate=7 * BASE, gate_stride=0, normed=7 * BASE - 2048), "overlaps gate"),
]


@pytest.mark.parametrize("change,word", REFUSED, ids=[f"{i}-{c[1]}" for i, c in enumerate(REFUSED)])
def test_norm_refuses(change, word):
    a = _args(**change)
    assert qmm._lib.qmm_norm_quantize(ctypes.byref(a), 4, 512, None) == qmm.EINVAL
    assert word in qmm.last_error()


def test_norm_refuses_sizes_and_accepts_an_empty_batch():
    f = qmm._lib.qmm_norm_quantize
    assert f(None, 4, 512, None) == qmm.EINVAL
    assert f(ctypes.byref(_args()), -1, 512, None) == qmm.EINVAL
    assert f(ctypes.byref(_args()), (1 << 20) + 1, 512, None) == qmm.EINVAL
    for id_ in (0, 255, 300, 1 << 21):
        assert f(ctypes.byref(_args()), 4, id_, None) == qmm.EINVAL
    empty = qmm.Norm(type=0, kind=0, eps=1e-5, residual_scale=1.0, block_scale=1.0)
    assert f(ctypes.byref(empty), 0, 512, None) == qmm.OK
    assert f(ctypes.byref(_args()), 0, 512, None) == qmm.EINVAL  # qact_bytes of four tokens


def test_dequantize_refuses():
    f, nb = qmm._lib.qmm_dequantize_activations, qmm.qact_bytes(4, 512)
    good = (BASE, nb, 4, 512, 0, 2 * BASE, 512, None)
    for at, v in ((0, None), (0, BASE + 4), (1, nb - 1), (2, -1), (2, 3000), (3, 500), (4, 3), (5, None), (5, 2 * BASE + 4),
                  (6, 508), (6, 513), (6, 1 << 25), (5, BASE + nb - 16)):
        args = list(good)
        args[at] = v
        assert f(*args) == qmm.EINVAL, (at, v)
    assert f(None, 0, 0, 512, 0, None, 512, None) == qmm.OK


def test_binding_refuses_host_tensors_and_names():
    x = torch.zeros(2, 256)
    with pytest.raises(qmm.QmmError):
        qmm.norm_quantize(x, torch.ones(256))
    with pytest.raises(qmm.QmmError):
        qmm.norm_quantize(torch.zeros(2, 256, dtype=torch.float64), torch.ones(256))
    with pytest.raises(qmm.QmmError):
        qmm.norm_quantize(x, torch.ones(256), kind="batch")
    with pytest.raises(qmm.QmmError):
        qmm.norm_quantize(torch.zeros(256), torch.ones(256))


# ---- on the GPU ----

@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def _depth(id_):
    # four additions per group of four of a thread (at least 1/64 of the row's groups per thread is the worst case
    # of the shortest rows), the wave's six, the waves' sixteen
    return 4 * max(16, (id_ + 4095) // 4096) + 6 + 16


def _norm64(x, kind, weight, bias, eps):
    """(norm, its tolerance in f32 arithmetic) of x in 64 bits."""
    w = weight.double()
    b = bias.double() if bias is not None else torch.zeros_like(w)
    D = _depth(x.shape[1])
    K = D / 2 + 8
    if kind == "layer":
        mean = x.mean(1, keepdim=True)
        rstd = 1 / (((x - mean) ** 2).mean(1, keepdim=True) + eps).sqrt()
        off = (D + 4) * U * x.abs().mean(1, keepdim=True) + U * (x - mean).abs()
    else:
        mean = torch.zeros_like(x[:, :1])
        rstd = 1 / ((x ** 2).mean(1, keepdim=True) + eps).sqrt()
        off = torch.zeros_like(x)
    n = (x - mean) * rstd * w
    # the variance's error from the deviations' own: second order but for the mean's part, bounded by rstd*off
    tol = K * U * n.abs() + off * rstd * w.abs() + off.amax(1, keepdim=True) * rstd * n.abs() + U * (n + b).abs()
    return n + b, tol


def _make(dev, T, id_, dtype, seed, post=False, gate="", kind="rms", y=True, bias=False):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = lambda *s, by=1.0: torch.randn(s, device=dev, generator=g) * by  # noqa: E731
    c = {"h": (r(T, id_) * (1 + 9 * (torch.rand(id_, device=dev, generator=g) < 0.02))).to(dtype),
         "weight": 1 + r(id_, by=0.2), "kind": kind}
    if y:
        c["y"] = (r(T, id_) + 0.3).to(dtype)
    if post:
        c["post_weight"] = 1 + r(id_, by=0.2)
    if gate:
        c["gate"] = r(*((id_,) if gate == "row" else (T, id_))).to(dtype)
    if bias:
        c["bias"] = r(id_, by=0.2)
        if post:
            c["post_bias"] = r(id_, by=0.2)
    return c


def _check(c, r, rs=1.0, bs=1.0, eps=1e-5):
    dtype = c["h"].dtype
    s = rs * c["h"].double()
    tol = 2 * U * s.abs()
    if "y" in c:
        u, ut = c["y"].double(), torch.zeros_like(s)
        if "post_weight" in c:
            u, ut = _norm64(u, c["kind"], c["post_weight"], c.get("post_bias"), eps)
        if "gate" in c:
            u, ut = u * c["gate"].double(), ut * c["gate"].double().abs()
        s = s + bs * u
        tol = tol + abs(bs) * (ut + 4 * U * u.abs())
    T, id_ = s.shape
    assert torch.all((r.h.double() - s).abs() <= tol + (HALF[dtype] + U) * (s.abs() + tol) + TINY[dtype])
    n, nt = _norm64(r.h.double(), c["kind"], c["weight"], c.get("bias"), eps)
    if r.normed is not None:
        assert torch.all((r.normed.double() - n).abs() <= nt + HALF[dtype] * (n.abs() + nt) + TINY[dtype])
    if r.qact is None:
        return
    q, dh, sm = layouts.read_qact(r.qact.cpu().numpy(), T, id_)
    assert not q[T:].any() and not dh[T:].any() and not sm[T:].any(), "padding not zero"
    if dtype == torch.float32 and r.normed is not None:  # normed is what was quantized: bit for bit
        oq, odh, os_ = oracle.quantize(r.normed.cpu().numpy())
        assert np.array_equal(q[:T], oq) and np.array_equal(dh[:T], odh) and np.array_equal(sm[:T], os_)
    d = dh[:T].view(np.float16).astype(np.float64)
    n64, n_tol = n.cpu().numpy().reshape(T, -1, 32), nt.cpu().numpy().reshape(T, -1, 32)
    top = np.abs(n64).max(2)
    # dh = f16(amax/127): a quarter of an f16 step covers subnormals, half a step of the value the rest
    assert np.all(np.abs(d - top / 127) <= 2.0 ** -11 * top / 127 * (1 + 1e-3) + 2.0 ** -25 + n_tol.max(2) / 127)
    # codes: half a step, and what the clamp to 127 takes off the largest when dh was rounded down
    v = (q[:T].reshape(T, -1, 32) * d[:, :, None])
    assert np.all(np.abs(v - n64) <= d[:, :, None] * (0.5 + 127 * 2.0 ** -11) + n_tol + 127 * 2.0 ** -25)
    sums = (d.astype(np.float32) * q[:T].reshape(T, -1, 32).sum(2).astype(np.float32)).astype(np.float16)
    assert np.array_equal(sm[:T], sums.view(np.uint16).reshape(sm[:T].shape))


CASES = [  # tokens, id: registers of every depth, the last ones in passes over memory
    (1, 256), (3, 768), (64, 512), (65, 4096), (130, 1024), (509, 4096), (33, 5120), (200, 11008), (2, 16384), (3, 16640),
    (5, 32768), (2, 33024), (1, 1 << 20)]


@gpu
@pytest.mark.parametrize("dtype", TYPES, ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,id_", CASES)
def test_norm_against_the_formula(device, T, id_, dtype):
    print(f"norm {T}x{id_} {dtype}", flush=True)
    for i, (kind, post, gate, y, bias, rs, bs) in enumerate([
            ("rms", False, "", True, False, 1.0, 1.0), ("rms", True, "row", True, False, 0.75, -0.5),
            ("layer", True, "all", True, True, 1.25, 0.3), ("layer", False, "", False, True, 1.0, 1.0)]):
        c = _make(device, T, id_, dtype, 100 * i + T, post, gate, kind, y, bias)
        r = qmm.norm_quantize(residual_scale=rs, block_scale=bs, normed=True, **c)
        _check(c, r, rs, bs)


@gpu
@pytest.mark.parametrize("id_", [512, 33024])
def test_norm_outputs_do_not_depend_on_each_other_or_on_the_place(device, id_):
    """The same bits for every choice of outputs, for strided rows, in place, and on a repeat."""
    print(f"norm outputs {id_}", flush=True)
    T = 70
    c = _make(device, T, id_, torch.bfloat16, 7, True, "row", "layer", True, True)
    full = qmm.norm_quantize(normed=True, **c)
    again = qmm.norm_quantize(normed=True, **c)
    for a, b in zip(full, again):
        assert torch.equal(a, b)
    for want in ({"normed": True, "qact": False}, {"h_out": False}, {"qact": False}, {"h_out": False, "normed": True, "qact": False}):
        r = qmm.norm_quantize(**{**c, **want})
        for a, b in zip(r, full):
            assert a is None or torch.equal(a, b), want
    wide = {k: torch.full((T, id_ + 12), float("nan"), dtype=torch.bfloat16, device=device) for k in ("h", "y", "h_out", "normed")}
    for k in ("h", "y"):
        wide[k][:, :id_] = c[k]
    r = qmm.norm_quantize(**{**c, **{k: v[:, :id_] for k, v in wide.items()}})
    assert torch.equal(r.h, full.h) and torch.equal(r.normed, full.normed) and torch.equal(r.qact, full.qact)
    assert all(torch.isnan(v[:, id_:]).all() for v in wide.values()), "written behind the rows"
    h, y = c["h"].clone(), c["y"].clone()
    r = qmm.norm_quantize(**{**c, "h": h, "y": y, "h_out": h, "normed": y})  # both in place
    assert torch.equal(h, full.h) and torch.equal(y, full.normed) and torch.equal(r.qact, full.qact)
    y = c["y"].clone()
    r = qmm.norm_quantize(**{**c, "y": y, "h_out": y})
    assert torch.equal(y, full.h) and torch.equal(r.qact, full.qact)
    h = c["h"].clone()
    qmm.norm_quantize(**{**c, "h": h, "h_out": False, "normed": h, "qact": False})
    assert torch.equal(h, full.normed)
    for lo, hi in ((0, 1), (3, 64), (64, 70)):  # rows do not depend on their neighbours
        part = {k: (v[lo:hi] if k in ("h", "y") else v) for k, v in c.items()}
        r = qmm.norm_quantize(normed=True, **part)
        assert torch.equal(r.h, full.h[lo:hi]) and torch.equal(r.normed, full.normed[lo:hi])


@gpu
def test_norm_of_zeros_and_of_values_that_are_not_finite(device):
    """A zero row gives zeros; NaN, infinity and overflow stay in their own row."""
    T, id_ = 6, 768
    c = _make(device, T, id_, torch.float32, 3)
    ref = qmm.norm_quantize(normed=True, **c)
    c["h"][1] = 0
    c["y"][1] = 0
    c["h"][2, 5] = float("nan")
    c["h"][3, 700] = float("inf")
    c["h"][4] = 3e38
    r = qmm.norm_quantize(normed=True, **c)
    assert not r.h[1].any() and not r.normed[1].any()
    assert torch.isnan(r.normed[2]).all() and torch.isnan(r.normed[3, 700])
    for i in (0, 5):
        assert torch.equal(r.h[i], ref.h[i]) and torch.equal(r.normed[i], ref.normed[i])
    q, dh, s = layouts.read_qact(r.qact.cpu().numpy(), T, id_)
    rq, rdh, rs = layouts.read_qact(ref.qact.cpu().numpy(), T, id_)
    assert not q[1].any() and not dh[1].any() and not s[1].any()
    for i in (0, 5):
        assert np.array_equal(q[i], rq[i]) and np.array_equal(dh[i], rdh[i])


@gpu
def test_norm_of_a_long_stream_passes_32_bits(device):
    """Rows whose byte and element offsets pass 2^32: a strided batch whose last row lies 2^32 elements behind the first."""
    id_, stride = 256, 1 << 24
    T = 258  # 257 * 2^24 > 2^32 elements of two bytes
    big = torch.zeros(T * stride - stride + id_, dtype=torch.bfloat16, device=device)
    h = big.as_strided((T, id_), (stride, 1))
    g = torch.Generator(device=device)
    g.manual_seed(1)
    h.copy_(torch.randn((T, id_), device=device, generator=g))
    w = torch.ones(id_, device=device)
    r = qmm.norm_quantize(h, w, normed=True)
    ref = qmm.norm_quantize(h.contiguous(), w, normed=True)
    for a, b in zip(r, ref):
        assert torch.equal(a, b)


@gpu
def test_norm_on_a_stream_and_in_a_graph(device):
    """Another stream than the current one; a capture replayed with new inputs and eager work between the replays."""
    T, id_ = 130, 1024
    c = _make(device, T, id_, torch.float16, 5, True, "row")
    ref = qmm.norm_quantize(normed=True, **c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        r = qmm.norm_quantize(normed=True, stream=s, **c)
        side.synchronize()
        for a, b in zip(r, ref):
            assert torch.equal(a, b)
    out = [torch.empty_like(v) for v in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.norm_quantize(h_out=out[0], normed=out[1], qact=out[2], **c)
    for i in range(3):
        c["h"].copy_(_make(device, T, id_, torch.float16, 20 + i)["h"])
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = qmm.norm_quantize(normed=True, **c)
        for a, b in zip(out, ref):
            assert torch.equal(a, b), f"replay {i}"


@gpu
@pytest.mark.parametrize("T,id_", [(1, 256), (45, 768), (130, 11008)])
def test_read_back(device, T, id_):
    """The read-back values are dh * q rounded once to the type: equal to numpy's, strided rows kept."""
    x = torch.randn((T, id_), device=device, generator=torch.Generator(device=device).manual_seed(T)) * 3
    qact = qmm.quantize_activations(x)
    q, dh, _ = layouts.read_qact(qact.cpu().numpy(), T, id_)
    v = q[:T].reshape(T, -1, 32).astype(np.float32) * dh[:T].view(np.float16).astype(np.float32)[:, :, None]
    v = torch.from_numpy(v.reshape(T, id_))
    for dtype in TYPES:
        assert torch.equal(qmm.dequantize_activations(qact, T, id_, dtype).cpu(), v.to(dtype))
    wide = torch.full((T, id_ + 4), 7.0, device=device)
    qmm.dequantize_activations(qact, T, id_, out=wide[:, :id_])
    assert torch.equal(wide[:, :id_].cpu(), v) and torch.all(wide[:, id_:] == 7.0)


@gpu
def test_norm_binding_refuses_wrong_tensors(device):
    c = _make(device, 4, 512, torch.float16, 1)
    for change in ({"weight": c["weight"].half()}, {"weight": c["weight"][:256]}, {"y": c["y"].float()},
                   {"y": c["y"][:3]}, {"h_out": c["h"].float()}, {"normed": torch.empty(4, 512, device=device)},
                   {"gate": torch.ones(4, 256, device=device).half()}, {"qact": torch.empty(16, dtype=torch.uint8, device=device)},
                   {"y": c["y"].t().contiguous().t()}, {"h": c["h"][:, 1:257]}, {"y": c["y"][:1].expand(4, 512)}):
        with pytest.raises(qmm.QmmError) as e:
            qmm.norm_quantize(**{**c, **change})
        assert e.value.code == qmm.EINVAL
