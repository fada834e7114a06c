"""Drives every validation path of qmm_rope_frequencies, qmm_rope_cache, qmm_cache_read, qmm_attention and
qmm_attention_plan in the library named on the command line, whose host code is built with AddressSanitizer and
UndefinedBehaviorSanitizer; no GPU is used.  Exits 0 if every call is answered as expected."""
import ctypes
import random
import sys

EINVAL, OK = -1, 0
P, I32, I64, SZ, F, D = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float, ctypes.c_double)


class Cache(ctypes.Structure):
    _fields_ = [("type", I32), ("heads", I32), ("head_dim", I32), ("page", I32), ("n_pages", I64), ("k", P), ("v", P)]


class Batch(ctypes.Structure):
    _fields_ = [("n_seq", I32), ("columns", I32), ("starts", P), ("lengths", P), ("table", P), ("table_stride", I64),
                ("max_new", I64), ("max_length", I64)]


class Rope(ctypes.Structure):
    _fields_ = [("type", I32), ("out_type", I32), ("q_heads", I32), ("layout", I32), ("n_rot", I32), ("magnitude", F),
                ("frequencies", P), ("positions", P), ("q", P), ("q_stride", I64), ("q_head_stride", I64), ("q_out", P),
                ("q_out_stride", I64), ("q_out_head_stride", I64), ("k", P), ("k_stride", I64), ("k_head_stride", I64), ("v", P),
                ("v_stride", I64), ("v_head_stride", I64)]


class Attn(ctypes.Structure):
    _fields_ = [("heads", I32), ("causal", I32), ("out_type", I32), ("scale", F), ("window", I64), ("q", P), ("q_stride", I64),
                ("q_head_stride", I64), ("out", P), ("out_stride", I64)]


class Plan(ctypes.Structure):
    _fields_ = [("work_bytes", SZ), ("work_groups", I64), ("few", I32), ("columns", I32), ("tiles", I32), ("splits", I32),
                ("share", I32)]


def main():
    L = ctypes.CDLL(sys.argv[1])
    L.qmm_last_error.restype = ctypes.c_char_p
    L.qmm_rope_frequencies.argtypes = [I64, D, ctypes.c_int, D, D, D, D, P, P]
    L.qmm_rope_cache.argtypes = [P, P, P, I64, P]
    L.qmm_cache_read.argtypes = [P, P, I64, ctypes.c_int, P, P, P]
    L.qmm_attention.argtypes = [P, P, P, I64, P, SZ, P]
    L.qmm_attention_plan.argtypes = [P, P, ctypes.c_int, I64, I64, ctypes.c_int, P]
    L.qmm_cache_page_bytes.argtypes, L.qmm_cache_page_bytes.restype = [ctypes.c_int] * 4, SZ
    bad = []

    def expect(what, got, want=EINVAL):
        if got != want:
            bad.append(f"{what}: got {got}, want {want} ({L.qmm_last_error().decode()})")

    def at(k):
        return k << 40

    wild32 = (-(1 << 31), -1, 0, (1 << 31) - 1)
    wild = (-(1 << 63), -1, (1 << 63) - 1, (1 << 62) + 8)
    cache = dict(type=1, heads=4, head_dim=128, page=64, n_pages=1000, k=at(1), v=at(2))
    batch = dict(n_seq=3, columns=10, starts=at(3), lengths=at(4), table=at(5), table_stride=10, max_new=7, max_length=600)
    rope = dict(type=0, out_type=1, q_heads=8, layout=1, n_rot=64, magnitude=1.0, frequencies=at(6), positions=at(7), q=at(8),
                q_stride=1024, q_head_stride=128, q_out=at(9), q_out_stride=1024, q_out_head_stride=128, k=at(10), k_stride=512,
                k_head_stride=128, v=at(11), v_stride=512, v_head_stride=128)
    attn = dict(heads=8, causal=1, out_type=1, scale=0.1, window=0, q=at(8), q_stride=1024, q_head_stride=128, out=at(9),
                out_stride=1024)
    changes = [("cache", {f: v}) for f, vs in {"type": wild32, "heads": wild32, "head_dim": wild32, "page": wild32, "n_pages": wild + (0,),
                                               "k": (None, at(1) + 8), "v": (None, at(2) + 1)}.items()
               for v in vs if not (f == "type" and v == 1)]
    changes += [("batch", {f: v}) for f, vs in {"n_seq": wild32, "columns": wild32, "starts": (None, 2), "lengths": (None, 1),
                                                "table": (None, 3), "table_stride": wild + (9,), "max_new": wild,
                                                "max_length": wild}.items() for v in vs]
    ropes = [{f: v} for f, vs in {"type": (-1, 3), "out_type": (3, -1), "q_heads": wild32, "layout": (-1, 2), "n_rot": (-16, 8, 144, 1 << 30),
                                  "magnitude": (float("nan"), float("inf")), "frequencies": (None, 4), "positions": (2,),
                                  "q": (1, at(9), at(1) + 64), "q_stride": wild + (64, 1028), "q_head_stride": wild + (64,),
                                  "q_out": (None, at(10), at(4)), "q_out_stride": wild + (128,), "k": (at(9), at(2)),
                                  "k_stride": wild, "v_head_stride": wild, "v": (at(1) + 16,)}.items() for v in vs]
    attns = [{f: v} for f, vs in {"heads": wild32 + (6,), "causal": (-1, 2), "out_type": (0, 2, 3, -1), "scale": (0.0, float("nan"), -1.0),
                                  "window": (-1, -(1 << 63)), "q": (None, 2), "q_stride": wild, "q_head_stride": wild,
                                  "out": (None, at(8), at(1), at(9) + 8), "out_stride": wild + (1016,)}.items() for v in vs]
    for n_tok in (1, 5, 1 << 20):
        for which, change in changes:
            c = Cache(**{**cache, **(change if which == "cache" else {})})
            b = Batch(**{**batch, **(change if which == "batch" else {})})
            what = f"{n_tok} {which} {change}"
            expect("rope " + what, L.qmm_rope_cache(ctypes.byref(Rope(**rope)), ctypes.byref(c), ctypes.byref(b), n_tok, None))
            expect("read " + what, L.qmm_cache_read(ctypes.byref(c), ctypes.byref(b), n_tok, 0, at(12), at(13), None))
            expect("attention " + what, L.qmm_attention(ctypes.byref(Attn(**attn)), ctypes.byref(c), ctypes.byref(b), n_tok, None, 0,
                                                        None))
        c, b = ctypes.byref(Cache(**cache)), ctypes.byref(Batch(**batch))
        for change in ropes:
            if n_tok == 1 and set(change) & {"q_stride", "k_stride", "q_out_stride"}:
                continue  # of one token: not used
            expect(f"rope {n_tok} {change}", L.qmm_rope_cache(ctypes.byref(Rope(**{**rope, **change})), c, b, n_tok, None))
        for change in attns:
            if n_tok == 1 and "q_stride" in change:
                continue
            expect(f"attention {n_tok} {change}", L.qmm_attention(ctypes.byref(Attn(**{**attn, **change})), c, b, n_tok, None, 0, None))
        for work, size in ((None, 1), (at(14), 0), (at(14) + 4, 64), (at(8), 64), (at(9), 1 << 50), (at(1) + 64, 16)):
            expect(f"work {work} {size}", L.qmm_attention(ctypes.byref(Attn(**attn)), c, b, n_tok, work, size, None))
    for n_tok in (-1, (1 << 20) + 1, -(1 << 63), (1 << 63) - 1):
        c, b = ctypes.byref(Cache(**cache)), ctypes.byref(Batch(**batch))
        expect("rope tokens", L.qmm_rope_cache(ctypes.byref(Rope(**rope)), c, b, n_tok, None))
        expect("read tokens", L.qmm_cache_read(c, b, n_tok, 0, at(12), None, None))
        expect("attention tokens", L.qmm_attention(ctypes.byref(Attn(**attn)), c, b, n_tok, None, 0, None))
    freq, rng = (D * 128)(), random.Random(1)
    for _ in range(3000):
        n = rng.choice([0, 8, 16, 24, 64, 128, 256, 272, -16, (1 << 63) - 1])
        base, factor = rng.choice([10000.0, 1.0, 0.0, -3.0, 1e300, float("nan"), 2.0]), rng.choice([1.0, 8.0, 0.0, -1.0, 1e-300, float("inf")])
        scaling = rng.randint(-1, 5)
        fast, slow, original = rng.choice([32.0, 1.0, 1e300, 0.0]), rng.choice([1.0, 0.0, 40.0, 1e-300]), rng.choice([4096.0, 0.0, 1e300])
        rc = L.qmm_rope_frequencies(n, base, scaling, factor, original, fast, slow, freq, None)
        ok = n in (16, 64, 128, 256) and base > 1 and 0 <= scaling <= 4 and (scaling == 0 or (factor > 0 and factor < float("inf"))) \
            and (scaling < 3 or (original > 0 and slow > 0 and fast > slow))
        expect(f"frequencies {n} {base} {scaling} {factor} {original} {fast} {slow}", rc, OK if ok else EINVAL)
    plan = Plan()
    for _ in range(20000):
        kv = rng.randint(1, 64)
        c = Cache(type=rng.choice([1, 2, 3]), heads=kv, head_dim=rng.choice([64, 96, 128, 192, 256]), page=64, n_pages=1)
        b = Batch(n_seq=rng.choice([1, 2, 100, 65535]), columns=1, max_new=rng.choice([0, 1, 7, 300, 1 << 20]),
                  max_length=rng.choice([0, 1, 31, 5000, 1 << 30]))
        rc = L.qmm_attention_plan(ctypes.byref(c), ctypes.byref(b), kv * rng.choice([1, 2, 8, 64]), rng.choice([0, 1, 128, 1 << 62]),
                                  rng.choice([0, 1, 5, 4096, 1 << 20]), rng.choice([1, 256, 65536]), ctypes.byref(plan))
        if rc not in (OK, EINVAL):
            bad.append(f"plan: {rc}")
    if bad:
        print("\n".join(bad[:50]))
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
