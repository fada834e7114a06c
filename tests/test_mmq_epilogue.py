"""qmm_mmq_epilogue: refusals on the CPU; on the GPU its sums against the oracle (and
against qmm_mmq bit for bit where the tiled kernel runs), and the epilogue on those
sums against its formula in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32): a term of a sum meets
eight additions of its super-block (two roundings each), one per super-block and one
per wave that shares the row: K = 20 + 2*nsb + 16 units of the terms' magnitudes.  In
the epilogue the bias add, the
scale, the factor and the residual's fused add round once each; exp of an argument z
is off by |z| units of u and a few ulp, erfc of y by its ulps and 2*y^2 times the
argument's error; act' is below 1.2 everywhere.  A stored value adds half a step of
its type."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402
from tests import layouts  # noqa: E402

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 1e-35, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-35}  # below the normal range
TYPES = [torch.float32, torch.float16, torch.bfloat16]
ACTS = sorted(qmm.ACTS)
gpu = pytest.mark.gpu


# ---- on the CPU ----

def test_refusals_that_need_no_handle():
    """What does not depend on the handle is refused first, so without a GPU."""
    L, buf = qmm._lib, ctypes.c_void_p(1 << 20)

    def call(out_type=0, work=None, work_bytes=0, **kw):
        ep = qmm.Epilogue(**{"scale": 1.0, **kw})
        return L.qmm_mmq_epilogue(None, buf, 16, 4, ctypes.byref(ep), out_type, buf, 256, work, work_bytes, None)

    for change, word in (({"act": 5}, "act"), ({"act": -1}, "act"), ({"type": 3}, "type"), ({"out_type": 4}, "out_type"),
                         ({"out_type": -1}, "out_type"), ({"scale": float("nan")}, "finite"),
                         ({"residual_scale": float("inf")}, "finite"), ({"bias": (1 << 20) + 2}, "bias"),
                         ({"mul": (1 << 20) + 2}, "aligned"), ({"residual": (1 << 20) + 1, "type": 1}, "aligned"),
                         ({"work": ctypes.c_void_p(1 << 20)}, "work"), ({"work_bytes": 16}, "work"),
                         ({"work": ctypes.c_void_p((1 << 20) + 8), "work_bytes": 16}, "work"), ({}, "handle")):
        assert call(**change) == qmm.EINVAL, change
        assert word in qmm.last_error(), (change, qmm.last_error())


def test_epilogue_struct_matches_header():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qmm.h")).read()
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} qmm_epilogue;", hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    assert re.findall(r"(\w+)\s*;", body) == [f[0] for f in qmm.Epilogue._fields_]
    for name, value in qmm.ACTS.items():
        assert int(re.search(rf"#define QMM_ACT_{name.upper()} (\d)", hdr).group(1)) == value


# ---- on the GPU ----

@pytest.fixture
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield torch.device("cuda", 0)
    torch.cuda.synchronize()


def act64(kind, v):
    """(activation in 64 bits, error of its f32 form in units of u relative to it)"""
    if kind == "relu":
        return v.clamp(min=0), torch.zeros_like(v)
    if kind == "silu":
        return v * torch.sigmoid(v), 12 + 4 * v.abs()
    if kind == "gelu":
        return 0.5 * v * torch.special.erfc(-v / 2 ** 0.5), 24 + 4 * v * v
    if kind == "gelu_tanh":
        z = 2 * (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)
        return v * torch.sigmoid(z), 12 + 8 * z.abs()
    return v, torch.zeros_like(v)


def formula(sums, ep, dtype):
    """(the epilogue of f32 sums in 64 bits, its tolerance)"""
    v = sums.double()
    tol = torch.zeros_like(v)
    if ep.get("bias") is not None:
        v = v + ep["bias"].double()
        tol = U * v.abs()
    a, units = act64(ep.get("act", "none"), v)
    tol = 1.2 * tol + U * units * a.abs()
    v = a * ep.get("scale", 1.0)
    tol = tol * abs(ep.get("scale", 1.0)) + 2 * U * v.abs()
    if ep.get("mul") is not None:
        tol = (tol + U * v.abs()) * ep["mul"].double().abs()
        v = v * ep["mul"].double()
    if ep.get("residual") is not None:
        v = v + ep.get("residual_scale", 1.0) * ep["residual"].double()
        tol = tol + U * v.abs() + U * (ep.get("residual_scale", 1.0) * ep["residual"].double()).abs()
    return v, tol + HALF[dtype] * (v.abs() + tol) + TINY[dtype]


def check(got, sums, ep):
    ref, tol = formula(sums, ep, got.dtype)
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4], tol[bad][:4])


def check_q8(qact, values):
    """The q8 blocks are those of the f32 values, bit for bit, padding tokens zero."""
    T, od = values.shape
    q, dh, s = layouts.read_qact(qact.cpu().numpy(), T, od)
    oq, odh, os_ = oracle.quantize(values.cpu().numpy())
    assert np.array_equal(q[:T], oq) and np.array_equal(dh[:T], odh) and np.array_equal(s[:T], os_)
    assert not q[T:].any() and not dh[T:].any() and not s[T:].any(), "padding not zero"


def make(dev, type_, od, id_, T, seed):
    raw, x = synth.case(type_, od, id_, T, seed=seed)
    w = qmm.register_weights(type_, od, id_, raw)
    return w, qmm.quantize_activations(torch.from_numpy(x).to(dev)), raw, x


def sides(dev, T, od, dtype, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, device=dev, generator=g)  # noqa: E731
    return {"bias": r(od) * 4, "mul": r(T, od).to(dtype), "residual": (r(T, od) * 5).to(dtype)}


SHAPES = [  # every geometry, split tails, all-split launches, odd rows and tokens, one row, one token
    (synth.Q6_K, 256, 512, 64), (synth.Q4_K, 131, 768, 37), (synth.Q4_K, 1, 256, 1), (synth.Q6_K, 33, 1024, 129),
    (synth.Q6_K, 4097, 2048, 509), (synth.Q4_K, 512, 2816, 300), (synth.Q4_K_PACKED, 4160, 1024, 512),
    (synth.Q4_K, 8192, 1024, 560), (synth.Q6_K, 8192, 512, 600), (synth.Q4_K_PACKED, 8192, 512, 650),
    (synth.Q4_K, 4099, 256, 2111),
    # few tokens: one block of them, several, odd rows; one to sixteen waves per row, some with more super-blocks
    (synth.Q4_K, 300, 11008, 17), (synth.Q4_K_PACKED, 1000, 4096, 32), (synth.Q6_K, 515, 11008, 33), (synth.Q6_K, 97, 1280, 100),
    (synth.Q4_K, 2048, 2304, 129), (synth.Q4_K_PACKED, 70, 256, 200), (synth.Q6_K, 20001, 768, 9), (synth.Q4_K, 40000, 512, 5),
    # two blocks in a wave
    (synth.Q4_K, 8300, 768, 64), (synth.Q6_K, 4161, 2816, 33), (synth.Q4_K_PACKED, 20000, 512, 50)]


@gpu
@pytest.mark.parametrize("type_,od,id_,T", SHAPES)
def test_epilogue_against_the_formula(device, type_, od, id_, T):
    print(f"epilogue {synth.TYPE_NAMES[type_]} {od}x{id_} T={T}", flush=True)
    w, qact, raw, x = make(device, type_, od, id_, T, seed=od + T)
    sums = qmm.mmq_epilogue(w, qact, T)
    if od * T < 1_100_000:
        q, dh, s = oracle.quantize(x)
        ref, A = oracle.mmq_parallel(synth.block_format(type_), raw, od, id_, q, dh, s)
        assert np.all(np.abs(sums.cpu().numpy() - ref) <= (36 + 2 * (id_ // 256)) * U * A)
    if -(-od // 32) * -(-T // 32) > 768:  # more than three rounds of the GPU: the tiled kernel
        assert torch.equal(sums.view(torch.int32), qmm.mmq(w, qact, T).view(torch.int32)), "not qmm_mmq's sums"
    assert torch.equal(sums, qmm.mmq_epilogue(w, qact, T)), "a repeat differs"
    for i, act in enumerate(ACTS):
        side, out = TYPES[i % 3], TYPES[(i + 1) % 3]
        c = sides(device, T, od, side, i)
        ep = {**c, "act": act, "scale": 0.5, "residual_scale": -1.25}
        check(qmm.mmq_epilogue(w, qact, T, dtype=out, **ep), sums, ep)
        for part in ("bias", "mul", "residual"):
            ep = {part: c[part], "act": act}
            check(qmm.mmq_epilogue(w, qact, T, dtype=side, **ep), sums, ep)
    w.release()


@gpu
@pytest.mark.parametrize("type_,od,id_,T", [
    (synth.Q6_K, 256, 512, 64), (synth.Q4_K, 256, 256, 1), (synth.Q4_K, 512, 2816, 300), (synth.Q6_K, 4352, 2048, 509),
    (synth.Q4_K, 8192, 1024, 560), (synth.Q6_K, 8192, 512, 600), (synth.Q4_K_PACKED, 8192, 512, 650),
    (synth.Q4_K, 4096, 256, 2111), (synth.Q4_K_PACKED, 1024, 768, 130), (synth.Q6_K, 512, 2816, 1), (synth.Q4_K, 768, 4096, 31),
    (synth.Q4_K_PACKED, 20480, 512, 32), (synth.Q6_K, 1024, 1024, 97), (synth.Q4_K, 8192, 768, 40)])
def test_q8_output_is_the_prepass_of_the_values(device, type_, od, id_, T):
    """The output kept as q8 blocks equals the prepass's blocks of the f32 output, with and
    without the vector path, into a buffer that held other bytes."""
    print(f"q8 output {synth.TYPE_NAMES[type_]} {od}x{id_} T={T}", flush=True)
    w, qact, _, _ = make(device, type_, od, id_, T, seed=od + T)
    for side, act in ((torch.float16, "silu"), (torch.float32, "none"), (torch.bfloat16, "gelu")):
        c = sides(device, T, od, side, 3)
        ep = {**c, "act": act, "scale": 0.25}
        out = torch.full((qmm.qact_bytes(T, od),), 0x5A, dtype=torch.uint8, device=device)
        values = qmm.mmq_epilogue(w, qact, T, **ep)
        got = qmm.mmq_epilogue(w, qact, T, dtype="q8", out=out, **ep)
        assert got is out
        check_q8(out, values)
        wide = torch.empty((T, od + 1), dtype=side, device=device)  # rows that cannot be read in fours
        wide[:, 1:] = c["mul"]
        out2 = qmm.mmq_epilogue(w, qact, T, dtype="q8", **{**ep, "mul": wide[:, 1:]})
        assert torch.equal(out, out2)
    w.release()


@gpu
@pytest.mark.parametrize("type_,od,id_,T", [(synth.Q4_K, 260, 512, 70), (synth.Q6_K, 4097, 2048, 509), (synth.Q4_K, 1001, 1024, 20), (synth.Q6_K, 4225, 512, 64)])
def test_strides_places_and_repeats(device, type_, od, id_, T):
    """Strided rows at any alignment, columns of one tensor, in place, and nothing written outside."""
    w, qact, _, _ = make(device, type_, od, id_, T, seed=9)
    c = sides(device, T, od, torch.float16, 4)
    ep = {**c, "act": "silu"}
    ref = qmm.mmq_epilogue(w, qact, T, dtype=torch.float16, **ep)
    assert torch.equal(ref, qmm.mmq_epilogue(w, qact, T, dtype=torch.float16, **ep))
    for pad, at in ((3, 1), (8, 4), (5, 0)):
        wide = torch.full((3, T, od + pad), float("nan"), dtype=torch.float16, device=device)
        v = wide[:, :, at:at + od]
        v[0], v[1] = c["mul"], c["residual"]
        bias = torch.empty(od + 1, device=device)[1:]
        bias.copy_(c["bias"])
        qmm.mmq_epilogue(w, qact, T, out=v[2], **{**ep, "bias": bias, "mul": v[0], "residual": v[1]})
        assert torch.equal(v[2], ref)
        assert torch.isnan(wide[:, :, :at]).all() and torch.isnan(wide[:, :, at + od:]).all()
    cols = torch.zeros((T, 3 * od), dtype=torch.float16, device=device)  # mul | out | residual in one tensor
    cols[:, :od], cols[:, 2 * od:] = c["mul"], c["residual"]
    qmm.mmq_epilogue(w, qact, T, out=cols[:, od:2 * od], **{**ep, "mul": cols[:, :od], "residual": cols[:, 2 * od:]})
    assert torch.equal(cols[:, od:2 * od], ref)
    for name in ("mul", "residual"):
        place = c[name].clone()
        qmm.mmq_epilogue(w, qact, T, out=place, **{**ep, name: place})
        assert torch.equal(place, ref)
    w.release()


@gpu
def test_values_that_are_not_finite_stay_where_they_are(device):
    """NaN and infinities of mul and residual reach their own elements only; large sums
    through every activation give no NaN."""
    T, od = 40, 96
    w, qact, _, _ = make(device, synth.Q4_K, od, 512, T, seed=2)
    c = sides(device, T, od, torch.float32, 5)
    ref = qmm.mmq_epilogue(w, qact, T, **c)
    c["mul"][3, 7], c["residual"][39, 95], c["residual"][0, 0] = float("nan"), float("inf"), float("-inf")
    got = qmm.mmq_epilogue(w, qact, T, **c)
    assert torch.isnan(got[3, 7]) and got[39, 95] == float("inf") and got[0, 0] == float("-inf")
    got[3, 7], got[39, 95], got[0, 0] = ref[3, 7], ref[39, 95], ref[0, 0]
    assert torch.equal(got, ref)
    for big in (1e4, -1e4, 1e15, -1e15):
        bias = torch.full((od,), big, device=device)
        sums = qmm.mmq(w, qact, T)
        for act in ACTS:
            got = qmm.mmq_epilogue(w, qact, T, bias=bias, act=act)
            want = sums + bias if act == "none" or big > 0 else torch.zeros_like(sums)
            assert torch.allclose(got, want, rtol=1e-6, atol=1e-30), (act, big)
    w.release()


@gpu
def test_work_memory_streams_and_graphs(device):
    """A split tail with the caller's work memory on two streams at once; a captured chain of
    two products (q8 between them) replayed with new inputs and eager work between."""
    type_, od, id_, T = synth.Q6_K, 4352, 2048, 509
    w, qact, _, _ = make(device, type_, od, id_, T, seed=6)
    w2, _, _, _ = make(device, synth.Q4_K, 4160, od, 1, seed=7)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    need = max(qmm.mmq_plan(type_, od, id_, T, cus).scratch_bytes, qmm.mmq_plan(synth.Q4_K, 4160, od, T, cus).scratch_bytes)
    assert cus != 256 or need > 0
    works = [torch.empty(need, dtype=torch.uint8, device=device) for _ in range(3)]
    c = sides(device, T, od, torch.bfloat16, 8)
    ref = qmm.mmq_epilogue(w, qact, T, **c)
    if need:
        with pytest.raises(qmm.QmmError) as e:
            qmm.mmq_epilogue(w, qact, T, work=works[0][:16], **c)
        assert e.value.code == qmm.EINVAL
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = [qmm.mmq_epilogue(w, qact, T, work=k, stream=s, **c) for k, s in zip(works, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)

    mid = torch.empty(qmm.qact_bytes(T, od), dtype=torch.uint8, device=device)
    out = torch.empty((T, 4160), device=device)
    x = torch.randn((T, id_), device=device, generator=torch.Generator(device=device).manual_seed(1))
    q_in = torch.empty_like(qact)

    def chain(work):
        qmm.quantize_activations(x, q_in)
        qmm.mmq_epilogue(w, q_in, T, act="silu", mul=c["mul"], dtype="q8", out=mid, work=work)
        qmm.mmq_epilogue(w2, mid, T, out=out, work=work)

    chain(works[2])
    torch.cuda.synchronize()
    if need:  # without work memory of its own a split call is not captured
        refused = torch.cuda.CUDAGraph()
        with torch.cuda.graph(refused):
            out.zero_()
            with pytest.raises(qmm.QmmError) as e:
                qmm.mmq_epilogue(w, q_in, T, out=torch.empty((T, od), device=device))
        assert e.value.code == qmm.EINVAL
        del refused
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(works[2])
    for i in range(3):
        x.normal_()
        chain(works[0])
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(float("nan"))
        mid.zero_()
        works[2].fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
    del graph
    w.release()
    w2.release()


@gpu
def test_refusals_with_a_handle(device):
    T, od, id_ = 20, 130, 512
    w, qact, _, _ = make(device, synth.Q4_K, od, id_, T, seed=1)
    c = sides(device, T, od, torch.float32, 1)
    good = dict(qact=qact, n_tok=T, **c)

    def refused(code=qmm.EINVAL, **change):
        with pytest.raises(qmm.QmmError) as e:
            qmm.mmq_epilogue(w, **{**good, **change})
        assert e.value.code == code, e.value

    refused(qmm.ESHAPE, qact=qact[:-16])
    refused(dtype="q8")                                              # od % 256 != 0
    refused(n_tok=-1)
    for change in ({"bias": c["bias"][1:]}, {"bias": c["bias"].half()}, {"act": "tanh"}, {"mul": c["mul"][1:]},
                   {"mul": c["mul"].half()}, {"residual": c["residual"].double()}, {"dtype": torch.float64},
                   {"out": torch.empty((T, od + 1), device=device)}, {"out": torch.empty((T, od))},
                   {"mul": c["mul"][:1].expand(T, od)}, {"scale": float("inf")}):
        refused(**change)
    buf = torch.empty((T + 1, od), device=device)
    refused(out=buf[:T], mul=buf[1:])                                # overlap that is not in place
    refused(residual=c["residual"].t().contiguous().t())             # rows without adjacent elements
    half = torch.empty((T, 2 * od), dtype=torch.float16, device=device)
    refused(out=half[:, :od], mul=half.view(torch.float32), residual=None)  # the same place in another type
    flat = torch.empty(T * od + 4 * od, device=device)
    refused(out=flat[:T * od].view(T, od), bias=flat[od:2 * od])
    refused(out=qact[:T * od * 4].view(torch.float32).view(T, od))
    refused(work=qact[:4096])
    wide = qmm._lib.qmm_mmq_epilogue
    ep = qmm.Epilogue(scale=1.0, mul=c["mul"].data_ptr(), mul_stride=od - 1)
    args = [w.handle, qact.data_ptr(), qact.numel(), T, ctypes.byref(ep), 0, buf.data_ptr(), od, None, 0, None]
    assert wide(*args) == qmm.EINVAL and "mul_stride" in qmm.last_error()
    args[4], args[7] = None, od - 1
    assert wide(*args) == qmm.EINVAL and "out_stride" in qmm.last_error()
    args[6], args[7] = None, od
    assert wide(*args) == qmm.EINVAL and "out" in qmm.last_error()
    assert qmm.mmq_epilogue(w, torch.empty(0, dtype=torch.uint8, device=device), 0).shape == (0, od)
    w.release()


@gpu
def test_few_tokens_on_streams_and_in_a_graph(device):
    """The few-token kernel needs no work memory: two streams at once, and captured without any."""
    for type_, T in ((synth.Q4_K, 32), (synth.Q6_K, 90)):
        w, qact, _, _ = make(device, type_, 1100, 2816, T, seed=T)
        c = sides(device, T, 1100, torch.float16, 3)
        ref = qmm.mmq_epilogue(w, qact, T, **c)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            outs = [qmm.mmq_epilogue(w, qact, T, stream=s, **c) for s in streams]
            torch.cuda.synchronize()
            assert all(torch.equal(o, ref) for o in outs)
        out = torch.empty_like(ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qmm.mmq_epilogue(w, qact, T, out=out, **c)
        for i in range(3):
            c["residual"].normal_()
            want = qmm.mmq_epilogue(w, qact, T, **c)
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), f"replay {i}"
        del graph
        w.release()


@gpu
def test_outputs_past_32_bits(device):
    """Outputs of more than 2^32 elements (f16, in place of the residual) and of more than 2^32 bytes of q8
    blocks: the last tokens equal a call with only them."""
    od, id_, T, last = 1 << 20, 256, 4200, 130
    raw, x = synth.case(synth.Q4_K, od, id_, T, seed=3)
    w = qmm.register_weights(synth.Q4_K_PACKED, od, id_, raw)
    x = torch.from_numpy(x).to(device)
    qact, tail = qmm.quantize_activations(x), qmm.quantize_activations(x[-last:].contiguous())
    out = torch.zeros((T, od), dtype=torch.float16, device=device)
    out[-last:] = 0.5
    want = qmm.mmq_epilogue(w, tail, last, dtype=torch.float16, act="relu", residual=out[-last:].clone())
    qmm.mmq_epilogue(w, qact, T, act="relu", residual=out, out=out)
    assert torch.equal(out[-last:], want)
    del out, want
    q8 = qmm.mmq_epilogue(w, qact, T, dtype="q8", scale=0.125)
    assert q8.numel() > 1 << 32
    want = qmm.dequantize_activations(qmm.mmq_epilogue(w, tail, last, dtype="q8", scale=0.125), last, od, torch.float16)
    got = qmm.dequantize_activations(q8, T, od, torch.float16)
    assert torch.equal(got[-last:], want)
    w.release()
