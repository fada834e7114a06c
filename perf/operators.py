"""The operators around the quantized products of a transformer layer, as cases to measure.

  norm     the norm after a block, its gate and the scales of the residual sum, the sum itself, and the norm before the
           next block, whose result is kept as q8 blocks (what the prefill product reads) or as numbers
  product  the prefill product of k-quant weights with bias, activation, a factor and the residual in its epilogue,
           stored as numbers or as the q8 blocks that the next product reads
  vector   the same product for one to eight tokens, straight from the activations

Weights are random q4_K / q6_K blocks, activations are quantized to q8 blocks of 32 with an f16 scale and an f16 scaled
sum.  With `own` false every operator is computed from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = {"q4_K": 144, "q4_K packed": 144, "q6_K": 210}
EPS = 1e-5


def _norm(tokens, width, dtype, kind="rms", post=False, gate=False, scales=False, out="q8", **more):
    return {"op": "norm", "tokens": tokens, "width": width, "dtype": dtype, "kind": kind, "post": post, "gate": gate,
            "scales": scales, "out": out, **more}


def _product(op, weights, rows, width, tokens, out, act="none", bias=False, mul="", residual="", x="f32", **more):
    return {"op": op, "weights": weights, "rows": rows, "width": width, "tokens": tokens, "out": out, "act": act,
            "bias": bias, "mul": mul, "residual": residual, "x": x, **more}


def listed():
    return [
        # one token of a decode step: the residual sum and the norm before the next product, all latency
        _norm(1, 4096, "f32", out="numbers", name="norm 1x4096 f32"),
        # a long prompt's layer: the norm feeds the prefill products
        _norm(3314, 4096, "f32", name="norm 3314x4096 f32 q8"),
        # norms on both sides of the block, with a per-channel gate and scaled residual, in 16 bits, a wider model
        _norm(512, 5120, "bf16", post=True, gate=True, scales=True, name="norm 512x5120 bf16 both q8"),
        # mean and variance, weight and bias, a wide row and an odd number of tokens
        _norm(509, 11008, "f16", kind="layer", out="numbers", name="norm 509x11008 f16 layer"),
        # the smallest product: one tile column, a bias and an activation
        _product("product", "q6_K", 256, 512, 64, "f32", act="gelu", bias=True, name="product q6_K 256x512 T64"),
        # the attention output of a 512-token prompt, added to the residual stream
        _product("product", "q4_K", 4096, 4096, 512, "f32", residual="f32", name="product q4_K 4096x4096 T512"),
        # the up projection of a long prompt, times the activated gate, kept as the down projection's q8 input
        _product("product", "q4_K", 11008, 4096, 3314, "q8", mul="f16", name="product q4_K 11008x4096 T3314 q8"),
        # an odd number of rows and of tokens, everything in the epilogue, 16-bit stream
        _product("product", "q6_K", 4097, 11008, 509, "bf16", act="gelu_tanh", bias=True, residual="bf16",
                 name="product q6_K 4097x11008 T509"),
        # one token through an attention projection: bound by latency and the weights' bytes
        _product("vector", "q4_K", 4096, 4096, 1, "f32", residual="f32", name="vector q4_K 4096x4096 T1"),
        # one token through the down projection, 16-bit stream
        _product("vector", "q6_K", 4096, 11008, 1, "f16", residual="f16", x="f16", name="vector q6_K 4096x11008 T1"),
        # a few sequences at once through the gate projection
        _product("vector", "q4_K", 11008, 4096, 5, "bf16", act="silu", bias=True, x="bf16",
                 name="vector q4_K 11008x4096 T5"),
        # the output head for eight sequences
        _product("vector", "q6_K", 32000, 4096, 8, "f32", name="vector q6_K 32000x4096 T8"),
    ]


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    width = 256 * _log(rng, 1, 56)
    if rng.random() < 1 / 3:
        tokens = _log(rng, 1, min(4096, 27_000_000 // width))
        return _norm(tokens, width, rng.choice(list(TYPES)), kind=rng.choice(["rms", "rms", "layer"]),
                     post=rng.random() < 0.4, gate=rng.random() < 0.4, scales=rng.random() < 0.5,
                     out=rng.choice(["q8", "numbers"]))
    op = rng.choice(["product", "vector"])
    rows = _log(rng, 24, min(32000, 131_072_000 // width))
    tokens = rng.randint(1, 8) if op == "vector" else _log(rng, 1, min(4096, max(1, 149_000_000_000 // (rows * width))))
    out = rng.choice(list(TYPES) + (["q8"] if op == "product" else []))
    if out == "q8":
        rows = max(256, rows // 256 * 256)
        tokens = max(1, min(tokens, 149_000_000_000 // (rows * width)))
    side = rng.choice(list(TYPES))
    return _product(op, rng.choice(["q4_K", "q6_K"] + (["q4_K packed"] if op == "product" else [])), rows, width, tokens,
                    out, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.5,
                    mul=side if rng.random() < 0.4 else "", residual=side if rng.random() < 0.5 else "",
                    x=rng.choice(list(TYPES)) if op == "vector" else "f32")


# ---- inputs ------------------------------------------------------------------------------------------------------

def _blocks(g, weights, rows, width):
    """Random k-quant blocks [rows * width/256][bytes]; the scales are those of weights of about 0.02."""
    n = rows * (width // 256)
    b = torch.randint(0, 256, (n, BLOCK[weights]), dtype=torch.uint8, device="cuda", generator=g)
    d = (torch.randn((n, 2), device="cuda", generator=g).abs() * 8e-5).half()
    if weights == "q6_K":
        b[:, 192:208] = torch.randint(-32, 32, (n, 16), dtype=torch.int8, device="cuda", generator=g).view(torch.uint8)
        b[:, 208:210] = d[:, :1].contiguous().view(torch.uint8)
    else:
        b[:, 0:4] = d.view(torch.uint8)
    return b


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, by=1.0, to=torch.float32):
        return (torch.randn(shape, device="cuda", generator=g) * by).to(to)

    tokens, width = case["tokens"], case["width"]
    if case["op"] == "norm":
        t = TYPES[case["dtype"]]
        loud = 1 + 19 * (torch.rand(width, device="cuda", generator=g) < 0.01).float()  # a few channels are far louder
        s = {"h": (normal(tokens, width) * loud).to(t), "y": normal(tokens, width, by=0.5, to=t),
             "weight": 1 + normal(width, by=0.1)}
        if case["kind"] == "layer":
            s["bias"] = normal(width, by=0.1)
        if case["post"]:
            s["post_weight"] = 1 + normal(width, by=0.1)
        if case["gate"]:
            s["gate"] = normal(width, by=0.5, to=t)
        return s
    rows = case["rows"]
    s = {"blocks": _blocks(g, case["weights"], rows, width), "x": normal(tokens, width, to=TYPES[case["x"]])}
    if case["bias"]:
        s["bias"] = normal(rows, by=0.5)
    if case["mul"]:
        s["mul"] = normal(tokens, rows, to=TYPES[case["mul"]])
    if case["residual"]:
        s["residual"] = normal(tokens, rows, to=TYPES[case["residual"]])
    return s


def _scales(case):
    """(scale of the residual, scale of the block)"""
    return (0.75, 0.5) if case["scales"] else (1.0, 1.0)


# ---- the plain form ----------------------------------------------------------------------------------------------

def _weights(kind, b, rows, width):
    """Blocks -> (factors of the codes [rows][width], mins [rows][width/32] or None), in 32 bits."""
    n = b.shape[0]
    if kind == "q6_K":
        ql = b[:, :128].view(n, 2, 1, 2, 32)
        qh = b[:, 128:192].view(n, 2, 1, 1, 32)
        low = torch.cat([ql & 15, ql >> 4], 2)  # [half][quarter / 2][quarter % 2][32]
        by = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=b.device).view(1, 1, 2, 2, 1)
        code = (low | (((qh >> by) & 3) << 4)).view(n, 16, 16).float() - 32
        d = b[:, 208:210].contiguous().view(torch.float16).float()
        return (code * (d * b[:, 192:208].view(torch.int8).float()).unsqueeze(2)).view(rows, width), None
    d = b[:, 0:4].contiguous().view(torch.float16).float()
    p = b[:, 4:16]
    scale = torch.cat([p[:, :4] & 63, (p[:, 8:12] & 15) | ((p[:, :4] >> 6) << 4)], 1).float()
    least = torch.cat([p[:, 4:8] & 63, (p[:, 8:12] >> 4) | ((p[:, 4:8] >> 6) << 4)], 1).float()
    qs = b[:, 16:144].view(n, 4, 1, 32)
    code = torch.cat([qs & 15, qs >> 4], 2).view(n, 8, 32).float()
    return (code * (d[:, :1] * scale).unsqueeze(2)).view(rows, width), (d[:, 1:] * least).view(rows, width // 32)


def _quantized(x):
    """Numbers [tokens][n] -> (the values that their q8 blocks stand for, the blocks' scaled sums); quotients in 64 bits,
    since they are next to the borders of a rounding."""
    v = x.view(x.shape[0], -1, 32)
    d = (v.abs().amax(2).double() / 127).float().half().float()
    q = (v.double() / d.double().unsqueeze(2)).float().round().clamp(-127, 127)
    q = torch.where(d.unsqueeze(2) > 0, q, torch.zeros_like(q))
    return (q * d.unsqueeze(2)).view(x.shape), (d * q.sum(2)).half().float()


def _act(kind, v):
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if kind == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_norm(kind, x, weight, bias=None):
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * weight
    return x if bias is None else x + bias


def _run_norm(s, case):
    t = TYPES[case["dtype"]]
    of_h, of_y = _scales(case)
    y = s["y"].float()
    if "post_weight" in s:
        y = _plain_norm(case["kind"], y, s["post_weight"])
    if "gate" in s:
        y = y * s["gate"].float()
    h = (s["h"].float() * of_h + y * of_y).to(t)
    n = _plain_norm(case["kind"], h.float(), s["weight"], s.get("bias"))
    if case["out"] == "q8":
        return {"h": h, "values": _quantized(n)[0].half()}
    return {"h": h, "normed": n.to(t)}


def _run_product(s, case):
    values, sums = _quantized(s["x"].float())
    v = values @ s["factors"].t()
    if s["mins"] is not None:
        v = v - sums @ s["mins"].t()
    if "bias" in s:
        v = v + s["bias"]
    v = _act(case["act"], v)
    if "mul" in s:
        v = v * s["mul"].float()
    if "residual" in s:
        v = v + s["residual"].float()
    return _quantized(v)[0].half() if case["out"] == "q8" else v.to(TYPES[case["out"]])


# ---- what is measured ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "norm":
        blocks = s.pop("blocks")
        if own:
            import quant_q8_gemm_amd as qmm
            kind = {"q4_K": qmm.Q4_K, "q4_K packed": qmm.Q4_K_PACKED, "q6_K": qmm.Q6_K}[case["weights"]]
            if case["op"] == "vector":
                kind = {qmm.Q4_K: qmm.Q4_K_ROWS, qmm.Q6_K: qmm.Q6_K_ROWS}[kind]
            s["w"] = qmm.register_weights(kind, case["rows"], case["width"], blocks.cpu().numpy())
        else:
            s["factors"], s["mins"] = _weights(case["weights"], blocks, case["rows"], case["width"])
    return s, case


def run(state):
    s, case = state
    if not own:
        return _run_norm(s, case) if case["op"] == "norm" else _run_product(s, case)
    import quant_q8_gemm_amd as qmm
    if case["op"] == "norm":
        of_h, of_y = _scales(case)
        q8 = case["out"] == "q8"
        r = qmm.norm_quantize(s["h"], s["weight"], bias=s.get("bias"), y=s["y"], post_weight=s.get("post_weight"),
                              gate=s.get("gate"), residual_scale=of_h, block_scale=of_y, kind=case["kind"], eps=EPS,
                              normed=not q8, qact=q8)
        if q8:
            return {"h": r.h, "values": qmm.dequantize_activations(r.qact, case["tokens"], case["width"],
                                                                  dtype=torch.float16)}
        return {"h": r.h, "normed": r.normed}
    epilogue = {"bias": s.get("bias"), "act": case["act"], "mul": s.get("mul"), "residual": s.get("residual")}
    if case["op"] == "vector":
        return qmm.mmv(s["w"], s["x"], dtype=TYPES[case["out"]], **epilogue)
    qact = qmm.quantize_activations(s["x"])
    if case["out"] == "q8":
        qact = qmm.mmq_epilogue(s["w"], qact, case["tokens"], dtype="q8", **epilogue)
        return qmm.dequantize_activations(qact, case["tokens"], case["rows"], dtype=torch.float16)
    return qmm.mmq_epilogue(s["w"], qact, case["tokens"], dtype=TYPES[case["out"]], **epilogue)


def work(case):
    tokens, width = case["tokens"], case["width"]
    if case["op"] == "norm":
        n, b = tokens * width, SIZE[case["dtype"]]
        # h and y read, h written; q8 blocks written and what they stand for, or numbers; the vectors
        vectors = width * (4 * (1 + (case["kind"] == "layer") + case["post"]) + b * case["gate"])
        return {"bytes": n * (3 * b + (1.125 + 2 if case["out"] == "q8" else b)) + vectors,
                "flops": n * (20 if case["out"] == "q8" else 10)}
    rows = case["rows"]
    b = rows * (width // 256) * BLOCK[case["weights"]] + tokens * width * SIZE[case["x"]] + 4 * rows * case["bias"]
    b += tokens * rows * ((SIZE[case["mul"]] if case["mul"] else 0) + (SIZE[case["residual"]] if case["residual"] else 0))
    b += tokens * rows * (1.125 + 2 if case["out"] == "q8" else SIZE[case["out"]])
    return {"bytes": b, "flops": 2 * tokens * rows * width}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------

def _exact_weights(kind, b, rows, width):
    """One 32-block after the other, from the blocks' definition: (weights without mins, mins)."""
    n = b.shape[0]
    v = b.to(torch.int64)

    def f16(at):
        bits = (v[:, at] + 256 * v[:, at + 1]).to(torch.int32).to(torch.int16)
        return bits.view(torch.float16).double()

    w = torch.empty((n, 256), dtype=torch.float64, device=b.device)
    least = torch.zeros((n, 8), dtype=torch.float64, device=b.device)
    for c in range(8):
        if kind == "q6_K":
            half, quarter = divmod(c, 4)
            ql = v[:, 64 * half + 32 * (quarter % 2):][:, :32]
            code = (ql // 16 if quarter > 1 else ql % 16) + 16 * (v[:, 128 + 32 * half:][:, :32] // 4 ** quarter % 4) - 32
            scale = v[:, 192 + 2 * c:194 + 2 * c]
            scale = (scale - 256 * (scale > 127)).repeat_interleave(16, 1)
            w[:, 32 * c:32 * c + 32] = f16(208)[:, None] * (scale * code)
        else:
            p = v[:, 4:16]
            if c < 4:
                scale, m = p[:, c] % 64, p[:, c + 4] % 64
            else:
                scale = p[:, c + 4] % 16 + 16 * (p[:, c - 4] // 64)
                m = p[:, c + 4] // 16 + 16 * (p[:, c] // 64)
            code = v[:, 16 + 32 * (c // 2):][:, :32] // (16 if c % 2 else 1) % 16
            w[:, 32 * c:32 * c + 32] = f16(0)[:, None] * (scale[:, None] * code)
            least[:, c] = f16(2) * m
    return w.view(rows, width), least.view(rows, -1)


def _exact_q8(x):
    """64-bit numbers -> (values, scaled sums) of their q8 blocks; the scale and the quotient are rounded as the format says."""
    v = x.reshape(x.shape[0], x.shape[1] // 32, 32)
    scale = (torch.maximum(v.amax(2), -v.amin(2)).float().double() / 127).float().to(torch.float16).double()[..., None]
    q = torch.nan_to_num((v / scale).float().double(), nan=0.0, posinf=0.0, neginf=0.0)
    q = torch.round(q).clamp(-127, 127)
    return (q * scale).reshape(x.shape), (q.sum(2) * scale[..., 0]).to(torch.float16).double()


def _exact_norm(kind, x, weight, bias):
    mean = x.sum(1, keepdim=True) / x.shape[1] if kind == "layer" else torch.zeros((), dtype=x.dtype, device=x.device)
    power = ((x - mean) ** 2).sum(1, keepdim=True) / x.shape[1]
    n = (x - mean) / (power + EPS).sqrt() * weight.double()
    return n + bias.double() if bias is not None else n


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        of_h, of_y = _scales(case)
        y = s["y"].double()
        if case["post"]:
            y = _exact_norm(case["kind"], y, s["post_weight"], None)
        if case["gate"]:
            y = y * s["gate"].double()
        h = of_h * s["h"].double() + of_y * y
        # the next norm reads the stream as it is kept
        n = _exact_norm(case["kind"], h.to(TYPES[case["dtype"]]).double(), s["weight"], s.get("bias"))
        return {"h": h, "values": _exact_q8(n)[0]} if case["out"] == "q8" else {"h": h, "normed": n}
    w, least = _exact_weights(case["weights"], s["blocks"], case["rows"], case["width"])
    values, sums = _exact_q8(s["x"].double())
    v = values @ w.t().contiguous() - sums @ least.t().contiguous()
    if case["bias"]:
        v = v + s["bias"].double()
    if case["act"] == "relu":
        v = torch.where(v > 0, v, torch.zeros_like(v))
    elif case["act"] == "silu":
        v = v * torch.sigmoid(v)
    elif case["act"] == "gelu":
        v = v * (1 + torch.erf(v / 2 ** 0.5)) / 2
    elif case["act"] == "gelu_tanh":
        v = v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))) / 2
    if case["mul"]:
        v = v * s["mul"].double()
    if case["residual"]:
        v = v + s["residual"].double()
    return _exact_q8(v)[0] if case["out"] == "q8" else v
