"""Drives every validation path of the layer operators (qmm_norm_quantize,
qmm_dequantize_activations, qmm_mmq_epilogue, qmm_mmv) in the library named on the
command line, whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer; no GPU is used.  Exits 0 if every call is answered as
expected."""
import ctypes
import sys

EINVAL, OK = -1, 0
P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class Norm(ctypes.Structure):
    _fields_ = [("type", I32), ("kind", I32), ("eps", F), ("residual_scale", F), ("block_scale", F), ("h", P),
                ("h_stride", I64), ("y", P), ("y_stride", I64), ("post_weight", P), ("post_bias", P), ("gate", P),
                ("gate_stride", I64), ("weight", P), ("bias", P), ("h_out", P), ("h_out_stride", I64), ("normed", P),
                ("normed_stride", I64), ("qact", P), ("qact_bytes", SZ)]


class Epilogue(ctypes.Structure):
    _fields_ = [("bias", P), ("act", I32), ("type", I32), ("scale", F), ("residual_scale", F), ("mul", P),
                ("mul_stride", I64), ("residual", P), ("residual_stride", I64)]


def main():
    L = ctypes.CDLL(sys.argv[1])
    L.qmm_last_error.restype = ctypes.c_char_p
    L.qmm_qact_bytes.argtypes, L.qmm_qact_bytes.restype = [I64, I64], SZ
    L.qmm_norm_quantize.argtypes = [P, I64, I64, P]
    L.qmm_dequantize_activations.argtypes = [P, SZ, I64, I64, ctypes.c_int, P, I64, P]
    L.qmm_mmq_epilogue.argtypes = [P, P, SZ, I64, P, ctypes.c_int, P, I64, P, SZ, P]
    L.qmm_mmv.argtypes = [P, P, ctypes.c_int, I64, I64, P, ctypes.c_int, P, I64, P]
    L.qmm_register_weights.argtypes = [ctypes.c_int, I64, I64, P, SZ, P, P]
    bad = []

    def expect(what, got, want=EINVAL):
        if got != want:
            bad.append(f"{what}: got {got}, want {want} ({L.qmm_last_error().decode()})")

    def at(k):
        return k << 30

    big, top = (1 << 63) - 1, (1 << 64) - 64
    sizes = [(4, 512), (1, 256), (1 << 20, 1 << 20), (0, 512), (-1, 512), (big, 512), (4, 300), (4, big), (4, 0)]
    for n_tok, id_ in sizes:
        q = L.qmm_qact_bytes(n_tok, id_)
        for field, values in {"type": (-1, 3, 1 << 30), "kind": (2, -1), "eps": (0.0, -1.0, float("nan")),
                              "residual_scale": (float("inf"),), "h": (None, at(1) + 4),
                              "h_stride": (0, -4, big, big - 3, 1 << 25), "y_stride": (-big, 1), "weight": (None, 3),
                              "h_out": (at(1) + 64, at(2) + 64, at(3)), "h_out_stride": (big, 511), "normed": (at(4),),
                              "qact": (at(1), at(6) + 1, None), "qact_bytes": (0 if q else 16, (1 << 64) - 1),
                              "post_bias": (at(8),), "gate": (at(4), at(7) + 8), "gate_stride": (big, -8)}.items():
            for v in values:
                a = dict(type=1, kind=0, eps=1e-5, residual_scale=1, block_scale=1, h=at(1), h_stride=512, y=at(2), y_stride=512,
                         weight=at(3), h_out=at(4), h_out_stride=512, normed=at(5), normed_stride=512, qact=at(6),
                         qact_bytes=q, gate=at(7) if field == "gate_stride" else None)
                a[field] = v
                got = L.qmm_norm_quantize(ctypes.byref(Norm(**a)), n_tok, id_, None)
                if (n_tok, id_) == (0, 512):  # an empty batch: pointers and strides are not used
                    expect(f"norm empty {field}={v}", got, EINVAL if field in ("type", "kind", "eps", "residual_scale",
                                                                               "qact_bytes") else OK)
                else:
                    expect(f"norm {n_tok}x{id_} {field}={v}", got)
        for args in ((at(1), q + 1, 0, at(2), id_), (at(1) + 1, q, 0, at(2), id_), (at(1), q, 7, at(2), id_),
                     (at(1), q, 0, at(2), big), (at(1), q, 0, at(1) + 64, id_)):
            if n_tok != 0 or args[1] != q or args[2] != 0:
                expect(f"dequantize {n_tok}x{id_} {args}",
                       L.qmm_dequantize_activations(args[0], args[1], n_tok, id_, args[2], args[3], args[4], None))
    for change in (dict(act=9), dict(act=-9), dict(type=5), dict(scale=float("nan")), dict(residual_scale=float("-inf")),
                   dict(bias=3), dict(mul=1), dict(residual=top + 1), {}):
        ep = Epilogue(**{"scale": 1.0, **change})
        for out_type in (-1, 0, 3, 4):
            expect(f"epilogue {change}", L.qmm_mmq_epilogue(None, at(1), 16, 4, ctypes.byref(ep), out_type, at(2), 4, None, 0,
                                                            None))
            for n_tok, x_type, stride in ((1, 0, 256), (17, 0, 256), (-1, 1, 256), (1, 4, 256), (1, 0, big), (1, 3, -1)):
                expect(f"mmv {change}", L.qmm_mmv(None, at(1), x_type, stride, n_tok, ctypes.byref(ep), out_type, at(2), 4, None))
    h, buf = P(), ctypes.create_string_buffer(840)
    for t, n in ((24, 840), (26, 576), (25, 840), (24, 0)):
        expect(f"register {t}", L.qmm_register_weights(t, 4, 256, buf, n, None, ctypes.byref(h)))
    for t, n in ((24, 576), (26, 840)):  # valid: refused only for want of a GPU, nothing left held
        L.qmm_set_memory_cap(ctypes.c_size_t(1))
        expect(f"cap {t}", L.qmm_register_weights(t, 4, 256, buf, n, None, ctypes.byref(h)), -3)
        L.qmm_set_memory_cap(ctypes.c_size_t(0))
        rc = L.qmm_register_weights(t, 4, 256, buf, n, None, ctypes.byref(h))
        if rc not in (OK, -4) or (rc == OK) != bool(h.value):
            bad.append(f"valid registration {t}: {rc}")
    if bad:
        print("\n".join(bad))
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
