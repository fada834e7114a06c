"""qmm_mmv and the rows forms: refusals on the CPU; on the GPU the registered bytes,
the sums against the oracle and the epilogue on them against its formula in 64 bits.

Tolerance of the sums: integer dots are exact; a term of the oracle's sum (a
32-block's scaled dot, its min) meets at most five roundings on its way into a
lane's sum and then one addition per term of that lane, at most eight per
super-block (of which a wave has every one in the worst case), two over the wave and
sixteen over the waves: K = 8*nsb + 23 units of 2^-24 of the sum of the terms'
magnitudes."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle  # noqa: E402
import quant_q8_gemm_amd as qmm  # noqa: E402
import synth  # noqa: E402
from tests import layouts  # noqa: E402
from tests.test_mmq_epilogue import ACTS, TYPES, U, check, check_q8, device, sides  # noqa: E402,F401

gpu = pytest.mark.gpu
ROWS = {synth.Q4_K: qmm.Q4_K_ROWS, synth.Q6_K: qmm.Q6_K_ROWS}


# ---- on the CPU ----

def test_refusals_that_need_no_handle():
    L, x, o = qmm._lib, 1 << 20, 1 << 21

    def call(n_tok=2, x_ptr=x, x_type=0, x_stride=512, out_type=0, **kw):
        ep = qmm.Epilogue(**{"scale": 1.0, **kw})
        return L.qmm_mmv(None, x_ptr, x_type, x_stride, n_tok, ctypes.byref(ep), out_type, o, 16, None)

    for change, word in (({"n_tok": -1}, "n_tok"), ({"n_tok": 17}, "n_tok"), ({"x_type": 4}, "x_type"), ({"x_type": 3, "x_ptr": x + 8}, "aligned"), ({"x_ptr": None}, "x is"),
                         ({"x_ptr": x + 8}, "aligned"), ({"x_ptr": x + 4, "x_type": 1}, "aligned"),
                         ({"x_stride": 514}, "aligned"), ({"out_type": 4}, "out_type"), ({"act": 7}, "act"),
                         ({"scale": float("inf")}, "finite"), ({}, "handle")):
        assert call(**change) == qmm.EINVAL, change
        assert word in qmm.last_error(), (change, qmm.last_error())


def test_rows_forms_have_no_plan():
    for t in (qmm.Q4_K_ROWS, qmm.Q6_K_ROWS):
        with pytest.raises(qmm.QmmError) as e:
            qmm.mmq_plan(t, 256, 256, 1, 256)
        assert e.value.code == qmm.EINVAL
    h = ctypes.c_void_p()
    buf = ctypes.create_string_buffer(840)
    f = qmm._lib.qmm_register_weights
    assert f(qmm.Q4_K_ROWS, 4, 256, buf, 4 * 210, None, ctypes.byref(h)) == qmm.EINVAL
    assert f(qmm.Q6_K_ROWS, 4, 256, buf, 4 * 144, None, ctypes.byref(h)) == qmm.EINVAL


# ---- on the GPU ----

def read_rows(buf, type_, od, id_, wd, sm):
    """The exported rows form back into block bytes, from the header's description."""
    nsb, tiles = id_ // 256, (od + 15) // 16
    nb = 16 * tiles * nsb
    out = np.zeros((tiles, nsb, 16, 144 if type_ == synth.Q4_K else 210), np.uint8)
    codes = buf[:nb * 128].reshape(tiles, nsb, 8, 16, 16).transpose(0, 1, 3, 2, 4).reshape(tiles, nsb, 16, 128)
    if type_ == synth.Q4_K:
        assert sm == buf.size
        head = buf[wd:wd + nb * 16].view("<u4").reshape(tiles, nsb, 16, 4).astype(np.int64)
        out[..., 0:4], out[..., 16:] = head >> 24, codes
        sc = np.stack([head & 63, head >> 12 & 63], -1).reshape(tiles, nsb, 16, 8)
        mn = np.stack([head >> 6 & 63, head >> 18 & 63], -1).reshape(tiles, nsb, 16, 8)
        out[..., 4:8] = sc[..., :4] | (sc[..., 4:] >> 4) << 6
        out[..., 8:12] = mn[..., :4] | (mn[..., 4:] >> 4) << 6
        out[..., 12:16] = (sc[..., 4:] & 15) | (mn[..., 4:] & 15) << 4
    else:
        out[..., :128] = codes
        high = buf[wd:wd + nb * 64].reshape(tiles, nsb, 4, 16, 2, 2, 4).astype(np.int64)  # [g][n][h][nibble][b]
        qh = np.zeros((tiles, nsb, 16, 2, 32), np.int64)
        real = (np.arange(tiles * 16) < od).reshape(tiles, 1, 16, 1)
        for g in range(4):
            for h in range(2):
                for nib in range(2):
                    for j in range(4):
                        bits = (high[:, :, g, :, h, nib] >> 2 * j & 3) ^ 2 * real
                        at = 16 * (g % 2) + 4 * j
                        qh[:, :, :, h, at:at + 4] |= bits << 2 * (g // 2 + 2 * nib)
        out[..., 128:192] = qh.reshape(tiles, nsb, 16, 64)
        out[..., 192:208] = (buf[sm:sm + nb * 16].reshape(tiles, nsb, 16, 16).astype(np.int64) - 128 * real).astype(np.int8).view(np.uint8)
        at = sm + (nb * 16 + 255) // 256 * 256
        out[..., 208:] = buf[at:at + nb * 2].reshape(tiles, nsb, 16, 2)
    out = out.transpose(0, 2, 1, 3).reshape(16 * tiles, nsb, -1)
    assert not out[od:].any(), "padding rows not zero"
    return out[:od]


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K])
@pytest.mark.parametrize("od,id_", [(1, 256), (7, 768), (130, 1024), (20001, 256)])
def test_registered_rows_are_the_blocks(device, type_, od, id_):  # noqa: F811
    """The rows form holds every bit of the blocks: read back, it is the input, byte for byte."""
    rng = np.random.default_rng(od)
    bb = synth.BLOCK_BYTES[type_]
    raw = rng.integers(0, 256, od * id_ // 256 * bb, dtype=np.uint8)
    w = qmm.register_weights(ROWS[type_], od, id_, raw)
    assert (w.type, w.od, w.id, w.od_pad, w.raw_bytes) == (ROWS[type_], od, id_, (od + 15) // 16 * 16, raw.size)
    assert w.plane_bytes <= raw.size // od * w.od_pad + 4 * 256
    assert np.array_equal(read_rows(w.export(), type_, od, id_, w.wd_offset, w.sm_offset).reshape(-1), raw)
    w.release()


def sums_ok(got, raw, type_, od, id_, x):
    q, dh, s = oracle.quantize(np.ascontiguousarray(x.float().cpu().numpy()))
    ref, A = oracle.mmq_parallel(type_, raw, od, id_, q, dh, s)
    K = 8 * (id_ // 256) + 23
    bad = ~(np.abs(got.cpu().numpy() - ref) <= K * U * A)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3])


SHAPES = [(1, 256), (3, 768), (64, 512), (131, 2048), (1030, 4096), (257, 11008), (4096, 2304), (20001, 512), (5, 65536)]


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K], ids=["q4_K", "q6_K"])
@pytest.mark.parametrize("od,id_", SHAPES)
def test_mmv_against_oracle_and_formula(device, type_, od, id_):  # noqa: F811
    print(f"mmv {synth.TYPE_NAMES[type_]} {od}x{id_}", flush=True)
    raw = synth.weights(np.random.default_rng(od), type_, od, id_)
    w = qmm.register_weights(ROWS[type_], od, id_, raw)
    for n_tok in (1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 16):
        x = synth.activations(np.random.default_rng(n_tok), n_tok, id_, outliers=n_tok % 2 == 0)
        x = torch.from_numpy(x).to(device).to(TYPES[n_tok % 3])
        got = qmm.mmv(w, x)
        sums_ok(got, raw, type_, od, id_, x)
        assert torch.equal(got, qmm.mmv(w, x)), "a repeat differs"
        qact = qmm.quantize_activations(x.float())
        assert torch.equal(got, qmm.mmv(w, qact, n_tok)), "from its q8 blocks it differs"
        for i, act in enumerate(ACTS[n_tok % 2::2]):
            c = sides(device, n_tok, od, TYPES[i % 3], i)
            ep = {**c, "act": act, "scale": 0.5, "residual_scale": -1.25}
            check(qmm.mmv(w, x, dtype=TYPES[(i + n_tok) % 3], **ep), got, ep)
            ep = {("bias", "mul", "residual")[i % 3]: c[("bias", "mul", "residual")[i % 3]], "act": act}
            check(qmm.mmv(w, x, **ep), got, ep)
    w.release()


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K], ids=["q4_K", "q6_K"])
@pytest.mark.parametrize("od,id_", [(256, 256), (512, 4096), (4096, 2304), (11008, 1024), (20480, 512), (256, 65536)])
def test_q8_output_is_the_prepass_of_the_values(device, type_, od, id_):  # noqa: F811
    """The output kept as q8 blocks: the next product's, from one to sixteen tokens, into a buffer that held other
    bytes; in the same order of sums as the numbers' where both share the waves per row tile."""
    print(f"mmv q8 {synth.TYPE_NAMES[type_]} {od}x{id_}", flush=True)
    raw = synth.weights(np.random.default_rng(od), type_, od, id_)
    w = qmm.register_weights(ROWS[type_], od, id_, raw)
    for n_tok in (1, 4, 6, 11, 16):
        x = torch.from_numpy(synth.activations(np.random.default_rng(n_tok), n_tok, id_)).to(device)
        c = sides(device, n_tok, od, torch.float16, 3)
        ep = {**c, "act": "silu", "scale": 2.0 ** -8}
        out = torch.full((qmm.qact_bytes(n_tok, od),), 0x5A, dtype=torch.uint8, device=device)
        assert qmm.mmv(w, x, dtype="q8", out=out, **ep) is out
        values = qmm.mmv(w, x, **ep)
        q, dh, s = layouts.read_qact(out.cpu().numpy(), n_tok, od)
        assert not q[n_tok:].any() and not dh[n_tok:].any() and not s[n_tok:].any(), "padding not zero"
        # the blocks' sums are f32 sums in another order where the waves per tile differ: K units of the terms
        # apart, far less than a step; codes may differ by one next to a border, rarely
        oq, odh, _ = oracle.quantize(values.cpu().numpy())
        d, od_ = (v[:n_tok].view(np.float16).astype(np.float64) for v in (dh, odh))
        assert np.all(np.abs(d - od_) <= 2.0 ** -10 * od_ + 2.0 ** -24)
        off = q[:n_tok].astype(int) != oq
        assert np.abs(q[:n_tok].astype(int) - oq).max() <= 1 and off.mean() <= 0.01
        sums = (d.astype(np.float32) * q[:n_tok].reshape(n_tok, -1, 32).sum(2).astype(np.float32)).astype(np.float16)
        assert np.array_equal(s[:n_tok], sums.view(np.uint16).reshape(s[:n_tok].shape))
        if od >= 20480:  # the same waves per tile: bit for bit
            check_q8(out, values)
    w.release()


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K], ids=["q4_K", "q6_K"])
def test_longest_rows_in_tiles(device, type_):  # noqa: F811
    """Rows whose activations do not fit the LDS at once: the inner dimension in tiles, the last one short."""
    for od, id_, n_tok in ((6, 1 << 20, 1), (37, 256 * 131, 8), (300, 256 * 61, 8), (50, 256 * 43, 16), (33, 256 * 29, 11),
                          (7, 256 * 300, 2), (21, 256 * 150, 3), (600, 256 * 70, 7)):
        raw, x = synth.case(type_, od, id_, n_tok, seed=od)
        w = qmm.register_weights(ROWS[type_], od, id_, raw)
        x = torch.from_numpy(x).to(device)
        got = qmm.mmv(w, x)
        sums_ok(got, raw, type_, od, id_, x)
        assert torch.equal(got, qmm.mmv(w, qmm.quantize_activations(x), n_tok))
        w.release()


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K], ids=["q4_K", "q6_K"])
@pytest.mark.parametrize("od,id_", [(4101, 256), (8197, 512), (12300, 256), (17000, 768), (24577, 256), (36865, 512)])
def test_any_share_of_row_tiles(device, type_, od, id_):  # noqa: F811
    """One to sixteen row tiles per work-group, odd numbers of them and a last group that is not full, as numbers and
    (the largest multiple of 256 rows) as q8 blocks."""
    od8 = od // 256 * 256
    raw = synth.weights(np.random.default_rng(od), type_, od, id_)
    w = qmm.register_weights(ROWS[type_], od, id_, raw)
    w8 = qmm.register_weights(ROWS[type_], od8, id_, raw[:raw.size // od * od8])
    scale = 2.0 ** -8  # the blocks' range
    for n_tok in (1, 2, 4, 7, 16):
        x = synth.activations(np.random.default_rng(n_tok), n_tok, id_)
        ref, A = oracle.mmq_parallel(type_, raw, od, id_, *oracle.quantize(x))
        E = (8 * (id_ // 256) + 23) * U * A
        x = torch.from_numpy(x).to(device)
        assert (np.abs(qmm.mmv(w, x).cpu().numpy() - ref) <= E).all()
        buf = torch.full((qmm.qact_bytes(n_tok, od8) + 4096,), 77, dtype=torch.uint8, device=device)
        qmm.mmv(w8, x, dtype="q8", out=buf[:-4096], scale=scale)
        assert (buf[-4096:] == 77).all(), "written behind the blocks"
        back = qmm.dequantize_activations(buf[:-4096], n_tok, od8).cpu().numpy().astype(np.float64)
        ref, E = ref[:, :od8] * scale, E[:, :od8] * scale
        # half a step of the block's largest value, or 0.07 steps where its stored scale (2^-11 off, or 2^-25 where
        # it is subnormal) is below a 127th of it
        top = (np.abs(ref) + E).reshape(n_tok, -1, 32).max(-1).repeat(32, -1)
        assert (np.abs(back - ref) <= 0.58 / 127 * top * (1 + 2.0 ** -10) + E + 127 * 2.0 ** -25).all()
    w.release()
    w8.release()


@gpu
@pytest.mark.parametrize("type_", [synth.Q4_K, synth.Q6_K], ids=["q4_K", "q6_K"])
def test_extreme_blocks(device, type_):  # noqa: F811
    """Full-range codes and scales, d and dmin of either sign, zero, subnormal and huge, activations with
    vanishing scales: within the same tolerance."""
    rng = np.random.default_rng(3)
    od, id_, T = 70, 1024, 4
    nb = od * id_ // 256
    blk = rng.integers(0, 256, (nb, synth.BLOCK_BYTES[type_]), dtype=np.uint8)
    halves = np.array([0x0000, 0x8000, 0x0001, 0x83FF, 0x7B53, 0xFB53, 0x1400, 0x9400], np.uint16)
    for at in ((0, 2) if type_ == synth.Q4_K else (208,)):
        blk[:, at:at + 2] = halves[rng.integers(0, 8, nb)].view(np.uint8).reshape(nb, 2)
    x = synth.activations(rng, T, id_)
    x[1] = 2046 * np.sign(x[1])
    x[2] *= 1e-6
    x[3, ::2] = 0
    w = qmm.register_weights(ROWS[type_], od, id_, blk.reshape(-1))
    x = torch.from_numpy(x).to(device)
    got = qmm.mmv(w, x)
    sums_ok(got, blk.reshape(-1), type_, od, id_, x)
    assert torch.equal(got, qmm.mmv(w, qmm.quantize_activations(x), T))  # the prepass's codes, ties and subnormals too
    w.release()


@gpu
def test_quantized_in_the_kernel_as_by_the_prepass(device):  # noqa: F811
    """Values a few ulps either side of half-integer quotients and on them, vanishing and subnormal scales: the
    same bits from the numbers and from the prepass's blocks of them."""
    rng = np.random.default_rng(11)
    T, id_ = 8, 1024
    x = np.zeros((T, id_), np.float32)
    xb = x.reshape(T, -1, 32)
    steps = (np.abs(rng.standard_normal(xb.shape[:2])) * 0.05 + 1e-3).astype(np.float16).astype(np.float32)
    steps[6] = np.float32(2.0 ** -24) * rng.integers(1, 40, steps.shape[1])  # subnormal scales
    steps[7, ::2] = 1e-9                                                      # vanishing ones
    xb[:, :, 0] = 127 * steps
    k = rng.integers(-126, 126, size=xb[:, :, 1:].shape).astype(np.float32)
    ulps = rng.integers(-3, 4, size=k.shape)
    target = ((k + 0.5) * steps[:, :, None]).astype(np.float32)
    xb[:, :, 1:] = np.nextafter(target, np.where(ulps > 0, np.inf, -np.inf).astype(np.float32))
    xb[:, :, 1:] = np.where(ulps == 0, target, xb[:, :, 1:])
    xb[6, :, 31] = 1.49 * 127 * steps[6]  # dh rounds down by up to a third: the clamp
    raw = synth.q6k_weights(rng, 200, id_)
    w = qmm.register_weights(qmm.Q6_K_ROWS, 200, id_, raw)
    xt = torch.from_numpy(x).to(device)
    got = qmm.mmv(w, xt)
    assert torch.equal(got, qmm.mmv(w, qmm.quantize_activations(xt), T))
    sums_ok(got, raw, synth.Q6_K, 200, id_, xt)
    r = qmm.norm_quantize(xt, torch.ones(id_, device=device), normed=True)  # the norm's blocks are made the same way
    assert torch.equal(r.qact, qmm.quantize_activations(r.normed))
    w.release()


@gpu
def test_mmv_numbers_are_the_mmqs(device):  # noqa: F811
    """The same product through the prefill path: both within f32 rounding of each other's terms."""
    for type_ in (synth.Q4_K, synth.Q6_K):
        raw, x = synth.case(type_, 515, 1280, 6, seed=11)
        w, wr = qmm.register_weights(type_, 515, 1280, raw), qmm.register_weights(ROWS[type_], 515, 1280, raw)
        x = torch.from_numpy(x).to(device)
        a, b = qmm.mmq(w, qmm.quantize_activations(x), 6), qmm.mmv(wr, x)
        q, dh, s = oracle.quantize(x.cpu().numpy())
        _, A = oracle.mmq(type_, raw, 515, 1280, q, dh, s)
        assert np.all(np.abs((a - b).cpu().numpy()) <= 2e-5 * A)


@gpu
def test_mmv_strides_places_streams_and_graphs(device):  # noqa: F811
    od, id_, T = 1030, 1024, 5
    raw, x = synth.case(synth.Q6_K, od, id_, T, seed=4)
    w = qmm.register_weights(qmm.Q6_K_ROWS, od, id_, raw)
    x = torch.from_numpy(x).to(device).half()
    c = sides(device, T, od, torch.bfloat16, 2)
    ep = {**c, "act": "gelu"}
    ref = qmm.mmv(w, x, dtype=torch.bfloat16, **ep)
    wx = torch.full((T, id_ + 8), float("nan"), dtype=x.dtype, device=device)
    wx[:, 4:-4] = x
    wo = torch.full((T, od + 7), float("nan"), dtype=torch.bfloat16, device=device)
    qmm.mmv(w, wx[:, 4:-4], out=wo[:, 3:-4], **ep)
    assert torch.equal(wo[:, 3:-4], ref) and torch.isnan(wo[:, :3]).all() and torch.isnan(wo[:, -4:]).all()
    for name in ("mul", "residual"):
        place = c[name].clone()
        qmm.mmv(w, x, out=place, **{**ep, name: place})
        assert torch.equal(place, ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = [qmm.mmv(w, x, dtype=torch.bfloat16, stream=s, **ep) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref) for o in outs)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.mmv(w, x, out=out, **ep)
    for i in range(3):
        x.normal_()
        want = qmm.mmv(w, x, dtype=torch.bfloat16, **ep)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
    del graph
    w.release()


@gpu
def test_mmv_refusals_with_a_handle(device):  # noqa: F811
    od, id_, T = 130, 512, 3
    raw, x = synth.case(synth.Q4_K, od, id_, T, seed=1)
    w, wm = qmm.register_weights(qmm.Q4_K_ROWS, od, id_, raw), qmm.register_weights(qmm.Q4_K, od, id_, raw)
    x = torch.from_numpy(x).to(device)
    c = sides(device, T, od, torch.float32, 1)

    def refused(h=w, xx=x, **kw):
        with pytest.raises(qmm.QmmError) as e:
            qmm.mmv(h, xx, **kw)
        assert e.value.code == qmm.EINVAL, e.value

    refused(h=wm)
    with pytest.raises(qmm.QmmError) as e:  # and the MMQ does not take a rows form
        qmm.mmq(w, qmm.quantize_activations(x), T)
    assert e.value.code == qmm.EINVAL
    with pytest.raises(qmm.QmmError):
        qmm.mmq_epilogue(w, qmm.quantize_activations(x), T)
    refused(xx=torch.zeros(17, id_, device=device))
    refused(xx=x[:, :256])
    refused(xx=x.double())
    refused(xx=x.cpu())
    refused(xx=torch.zeros(T, id_ + 4, device=device)[:, 1:-3])
    refused(xx=torch.zeros(T, id_ + 2, device=device)[:, :-2])
    refused(xx=x[:1].expand(T, id_))
    refused(dtype=torch.float64)
    refused(dtype="q8")                                              # od % 256 != 0
    with pytest.raises(qmm.QmmError) as e:
        qmm.mmv(w, qmm.quantize_activations(x)[:-16], T)
    assert e.value.code == qmm.ESHAPE
    refused(xx=x.view(-1))
    refused(mul=c["mul"].half(), residual=c["residual"])
    refused(out=torch.empty(T, od + 1, device=device))
    both = torch.zeros(T * id_ + 64, device=device)
    refused(xx=both[:T * id_].view(T, id_), out=both[64:64 + T * od].view(T, od))
    assert qmm.mmv(w, x[:0]).shape == (0, od)
    w.release()
    wm.release()


@gpu
def test_largest_matrices(device):  # noqa: F811
    """The most rows the ABI takes (the last ones against the oracle), and a wide row with sixteen tokens whose
    LDS is past 64 KiB, captured into a graph."""
    od, id_, T = 1 << 21, 256, 2
    raw, x = synth.case(synth.Q6_K, od, id_, T, seed=5)
    w = qmm.register_weights(qmm.Q6_K_ROWS, od, id_, raw)
    x = torch.from_numpy(x).to(device)
    got = qmm.mmv(w, x, dtype=torch.float32)
    for lo in (0, od - 100):
        sums_ok(got[:, lo:lo + 100], raw[lo * 210:(lo + 100) * 210], synth.Q6_K, 100, id_, x)
    w.release()
    raw, x = synth.case(synth.Q4_K, 600, 5120, 16, seed=6)
    w = qmm.register_weights(qmm.Q4_K_ROWS, 600, 5120, raw)
    x = torch.from_numpy(x).to(device)
    want = qmm.mmv(w, x)
    sums_ok(want, raw, synth.Q4_K, 600, 5120, x)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.mmv(w, x, out=out)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del graph
    w.release()


@gpu
def test_infinities_and_nan_stay_in_their_token(device):  # noqa: F811
    """Values outside the q8 range are not specified, but they do not reach the other tokens of the call."""
    for type_ in (synth.Q4_K, synth.Q6_K):
        for T in (3, 7, 12):
            raw, x = synth.case(type_, 100, 768, T, seed=T)
            w = qmm.register_weights(ROWS[type_], 100, 768, raw)
            x = torch.from_numpy(x).to(device)
            ref = qmm.mmv(w, x)
            bad = x.clone()
            bad[1, 5], bad[1, 700], bad[2, 300] = float("nan"), float("inf"), 1e30
            got = qmm.mmv(w, bad)
            keep = [t for t in range(T) if t not in (1, 2)]
            assert torch.equal(got[keep], ref[keep])
            w.release()
