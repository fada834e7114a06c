"""The operators between a layer's q, k, v products and its output product, as cases to measure.

  rope    rotary positions of the new tokens' queries and keys, and the keys and values kept in a paged cache
  attend  attention of the sequences' new tokens (one of a decode step, a chunk of a prompt, a whole prompt) over the cache
  cross   attention of the new tokens to an encoder's states, of another length than theirs, kept in a cache

A cache has pages of a power of two of slots, taken in any order by a table for each sequence; it holds f16, bf16 or q8 blocks of 32
channels with an f16 scale.  With `own` false every operator is computed from elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "q8": 1.0625}


def _rope(sequences, new, length, heads, kv_heads, dim, cache, x, rotated, layout, scaling="none", far=0, page=64,
          ragged=0, **more):
    return {"op": "rope", "sequences": sequences, "new": new, "length": length, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "cache": cache, "x": x, "rotated": rotated, "layout": layout, "scaling": scaling, "far": far, "page": page,
            "ragged": ragged, **more}


def _attend(op, sequences, new, length, heads, kv_heads, dim, cache, out="same", window=0, page=64, ragged=0, **more):
    return {"op": op, "sequences": sequences, "new": new, "length": length, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "cache": cache, "out": out, "window": window, "page": page, "ragged": ragged, **more}


def listed():
    return [
        # a decode step of one sequence: three short rows and a cache slot, all latency
        _rope(1, 1, 3314, 32, 32, 128, "f16", "f16", 128, "interleaved", name="rope 1 token 32+32x128 f16"),
        # a long prompt, straight from the f32 products
        _rope(1, 3314, 3314, 32, 32, 128, "f16", "f32", 128, "half", name="rope 3314 tokens 32+32x128 f32"),
        # chunks of several sequences, half of each head rotated, a scaled context, the cache in 8 bits
        _rope(24, 150, 900, 40, 8, 128, "q8", "f16", 64, "interleaved", scaling="yarn", ragged=1, page=32,
              name="rope 24 chunks 40+8x128 q8"),
        # far positions of a long context, an odd number of tokens each, wide heads
        _rope(7, 129, 300, 16, 4, 256, "bf16", "bf16", 256, "half", scaling="linear", far=1000000, page=128,
              name="rope 7x129 far 16+4x256 bf16"),
        # one token of one sequence behind a long prompt: latency and the cache's bytes
        _attend("attend", 1, 1, 3314, 32, 32, 128, "f16", name="decode 1 of 3314 32/32x128 f16"),
        # a batch of sequences of all lengths, the cache in 8 bits, kept as the output product's q8 input
        _attend("attend", 32, 1, 8192, 32, 8, 128, "q8", out="q8", ragged=1, name="decode 32 of 8192 32/8x128 q8"),
        # one token over a very long context: the work of few rows split over a long axis
        _attend("attend", 1, 1, 131072, 64, 8, 128, "bf16", page=256, name="decode 1 of 131072 64/8x128 bf16"),
        # a whole prompt, kept as the output product's q8 input
        _attend("attend", 1, 3314, 3314, 32, 32, 128, "f16", out="q8", name="prompt 3314 32/32x128 f16 q8"),
        # a chunk of a long prompt over what is cached of it; the largest case
        _attend("attend", 1, 2048, 32768, 40, 8, 128, "bf16", page=128, name="chunk 2048 of 32768 40/8x128 bf16"),
        # prompts, chunks and single tokens in one batch, a sliding window, wide heads
        _attend("attend", 9, 300, 5000, 16, 4, 256, "f16", window=1024, ragged=1, page=32, name="mixed 9 of 5000 16/4x256 f16"),
        # a decode step over encoder states; some sequences have few of them or none
        _attend("cross", 16, 1, 1500, 20, 20, 64, "f16", ragged=1, page=32, name="cross 16x1 to 1500 20/20x64 f16"),
        # a decoder's prompt over encoder states, heads of 96
        _attend("cross", 4, 448, 1501, 16, 16, 96, "bf16", name="cross 4x448 to 1501 16/16x96 bf16"),
    ]


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "cross"])
    kv_heads, group = rng.choice([1, 2, 4, 5, 8, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 8])
    if kv_heads > 8:
        group = rng.choice([1, 1, 2])
    heads, dim = kv_heads * group, rng.choice([64, 96, 128, 128, 192, 256])
    cache, page, ragged = rng.choice(["f16", "bf16", "q8"]), rng.choice([32, 64, 128, 256]), rng.choice([0, rng.randint(1, 999)])
    if op == "rope":
        new = rng.choice([1, _log(rng, 2, 4096)])
        sequences = _log(rng, 1, max(1, min(64, 30_000_000 // (new * heads * dim))))
        new = max(1, min(new, 30_000_000 // (sequences * heads * dim)))
        return _rope(sequences, new, new + rng.randint(0, 1000), heads, kv_heads, dim, cache,
                     "bf16" if cache == "bf16" else rng.choice(["f16", "f32"]), rng.choice([dim, dim, dim // 2, 16]),
                     rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "yarn"]),
                     rng.choice([0, _log(rng, 1000, 1000000)]), page, ragged)
    length = _log(rng, 1, 65536)
    sequences = _log(rng, 1, max(1, min(64, 200_000_000 // (length * kv_heads * dim))))
    length = max(1, min(length, 200_000_000 // (sequences * kv_heads * dim)))
    most = max(1, min(4096, 1_000_000_000 // (sequences * length * heads)))
    most = max(1, min(most, 60_000_000 // (sequences * heads * dim)))
    if op == "attend":
        most = min(most, length)
    new = rng.choice([1, _log(rng, 1, min(8, most)), _log(rng, 1, most)])
    return _attend(op, sequences, new, length, heads, kv_heads, dim, cache,
                   "q8" if heads * dim % 256 == 0 and rng.random() < 0.3 else "same",
                   rng.choice([0, 0, _log(rng, 1, length)]) if op == "attend" else 0, page, ragged)


def _sizes(case):
    """(new tokens, slots in use with them) of each sequence; the first has the most of both."""
    n, new, length = case["sequences"], case["new"], case["length"]
    if not case["ragged"]:
        return [new] * n, [length] * n
    rng = random.Random(case["ragged"])
    news = [new] + [rng.randint(1 if new == 1 else 0, new) for _ in range(n - 1)]
    low = [0] * n if case["op"] == "cross" else news
    return news, [length] + [rng.randint(a, length) for a in low[1:]]


# ---- inputs ------------------------------------------------------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, by=1.0, to=torch.float32):
        return (torch.randn(shape, device="cuda", generator=g) * by).to(to)

    news, lens = _sizes(case)
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    tokens = sum(news)
    columns = [-(-n // page) for n in lens]
    pages = max(1, sum(columns))
    s = {"news": news, "lens": lens, "pages": pages}

    def whole(v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.zeros((len(news), max(1, max(columns))), dtype=torch.int32)
    at = 0
    for i, c in enumerate(columns):
        table[i, :c] = order[at:at + c]
        at += c
    s["table"] = table.cuda()
    s["starts"] = whole([sum(news[:i]) for i in range(len(news) + 1)])
    s["lengths"] = whole(lens)
    if case["op"] == "rope":
        t = TYPES[case["x"]]
        loud = 1 + 9 * (torch.rand(dim, device="cuda", generator=g) < 0.02).float()  # keys have a few loud channels
        s["q"] = normal(tokens, heads, dim, to=t)
        s["k"] = (normal(tokens, kv_heads, dim) * loud).to(t)
        s["v"] = normal(tokens, kv_heads, dim, by=0.5, to=t)
        if case["far"]:  # positions that do not go by the slots
            s["positions"] = whole([case["far"] + seed % 1000 + j for n in news for j in range(n)])
        return s
    # what the cache holds of the sequences, one behind the other; keys with a common part, as after a norm and a product
    held = sum(lens)
    t = torch.bfloat16 if case["cache"] == "bf16" else torch.float16
    s["q"] = normal(tokens, heads, dim, by=1.5, to=t)
    s["k"] = (normal(held, kv_heads, dim) + normal(kv_heads, dim)).to(t)
    s["v"] = (normal(held, kv_heads, dim) + 0.2 * normal(kv_heads, dim)).to(t)
    s["held"] = whole([sum(lens[:i]) for i in range(len(lens) + 1)])
    return s


def _frequencies(case):
    """(angle per position of each pair, in 64 bits, and the factor of what is rotated)"""
    n, base = case["rotated"], 10000.0
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":
        return [x / 4.0 for x in f], 1.0
    if case["scaling"] == "yarn":  # 4 times the context of 4096: pairs of few turns are slowed, of many are not
        def pair(turns):
            return n * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(0, math.floor(pair(32.0))), min(n - 1, math.ceil(pair(1.0)))
        keep = [1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(n // 2)]
        return [x / 4.0 * (1 - k) + x * k for x, k in zip(f, keep)], 0.1 * math.log(4.0) + 1.0
    return f, 1.0


# ---- the plain form ----------------------------------------------------------------------------------------------

def _quantized(x):
    """Numbers [...][n] -> (codes, f16 scales) of their q8 blocks; quotients in 64 bits, since they are next to the borders of
    a rounding."""
    v = x.unflatten(-1, (-1, 32))
    d = (v.abs().amax(-1).double() / 127).float().half()
    q = (v.double() / d.double().unsqueeze(-1)).float().round().clamp(-127, 127)
    q = torch.where(d.unsqueeze(-1) > 0, q, torch.zeros_like(q))
    return q.flatten(-2).to(torch.int8), d


def _values(codes, scales):
    return (codes.unflatten(-1, (-1, 32)).float() * scales.float().unsqueeze(-1)).flatten(-2)


def _places(s, starts, news, lens, page):
    """(page, slot) of each token of sequences whose tokens are the last ones of their slots."""
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(news)] or [torch.zeros(0)]).long().cuda()
    slot = torch.cat([torch.arange(length - n, length) for n, length in zip(news, lens)]).long().cuda()
    return s["table"].long()[seq, slot // page], slot % page, slot


def _turned(x, cos, sin, layout, n):
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if layout == "interleaved" else (x[..., :n // 2], x[..., n // 2:n])
    c, d = a * cos - b * sin, a * sin + b * cos
    both = torch.stack([c, d], -1).flatten(-2) if layout == "interleaved" else torch.cat([c, d], -1)
    return torch.cat([both, x[..., n:]], -1)


def _run_rope(s, case):
    page, slot, place = s["places"]
    angle = s.get("positions", place).double()[:, None] * s["frequencies"]
    cos, sin = ((f(angle) * s["magnitude"]).float().unsqueeze(1) for f in (torch.cos, torch.sin))
    n = case["rotated"]
    q = _turned(s["q"].float(), cos, sin, case["layout"], n)
    k = _turned(s["k"].float(), cos, sin, case["layout"], n)
    v = s["v"].float()
    if case["cache"] == "q8":
        out = {"q": q.half()}
        for name, x in (("k", k), ("v", v)):
            codes, scales = _quantized(x)
            s["pool_" + name][page, :, slot] = codes
            s["scale_" + name][page, :, slot] = scales
            out[name] = _values(s["pool_" + name][page, :, slot], s["scale_" + name][page, :, slot]).half()
        return out
    t = TYPES[case["cache"]]
    s["pool_k"][page, :, slot] = k.to(t)
    s["pool_v"][page, :, slot] = v.to(t)
    pages, heads, slots, dim = s["pool_k"].shape
    # the whole cache, in the order of the views that the framework gives of its own
    return {"q": q.to(t), "k": s["pool_k"].view(pages, heads, slots // 32, 2, 2, 2, 4, dim // 16, 2, 8),
            "v": s["pool_v"].view(pages, heads, slots // 32, 2, 2, 8, dim // 32, 32)}


def _gathered(s, name, case):
    """[sequence][head][slot][channel] in 32 bits"""
    table = s["table"].long()
    x = s["pool_" + name][table]
    x = _values(x, s["scale_" + name][table]) if case["cache"] == "q8" else x.float()
    return x.transpose(1, 2).flatten(2, 3)


def _run_attend(s, case):
    n, new, heads, kv_heads, dim = case["sequences"], case["new"], case["heads"], case["kv_heads"], case["dim"]
    k, v = _gathered(s, "k", case), _gathered(s, "v", case)
    seq, row = s["rows"]
    q = torch.zeros((n, new, heads, dim), device=k.device)
    q[seq, row] = s["q"].float()
    q = q.view(n, new, kv_heads, -1, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = q @ k.transpose(2, 3).contiguous() * dim ** -0.5
    key = torch.arange(k.shape[2], device=k.device)
    lengths = s["lengths"].long()
    seen = (key < lengths[:, None])[:, None, :]
    if case["op"] == "attend":
        news = s["starts"].long().diff()
        at = (lengths - news)[:, None] + torch.arange(new, device=k.device)
        seen = seen & (key <= at[:, :, None])
        if case["window"]:
            seen = seen & (key > at[:, :, None] - case["window"])
    seen = seen.expand(n, new, -1).repeat(1, heads // kv_heads, 1).unsqueeze(1)
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(3, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(3, keepdim=True)
    o = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.view(n, kv_heads, -1, new, dim).permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, row]
    if case["out"] == "q8":
        return _values(*_quantized(o.flatten(1))).half()
    return o.to(s["q"].dtype)


# ---- what is measured ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    s = _inputs(case, seed)
    heads, dim, page, news, lens = case["kv_heads"], case["dim"], case["page"], s["news"], s["lens"]
    rope, q8 = case["op"] == "rope", case["cache"] == "q8"
    if rope:
        s["frequencies"], s["magnitude"] = _frequencies(case)
        s["frequencies"] = torch.tensor(s["frequencies"], dtype=torch.float64).cuda()
    if own:
        import quant_q8_gemm_amd as qmm
        dtype = "q8" if q8 else TYPES[case["cache"]]
        s["cache"] = qmm.Cache(s["pages"], heads, dim, page=page, dtype=dtype)
        s["batch"] = qmm.Batch(s["starts"], s["lengths"], s["table"], max_new=max(news), max_length=max(lens))
        if not rope:  # what is in the cache when the call comes
            held = qmm.Batch(s["held"], s["lengths"], s["table"], max_new=max(lens), max_length=max(lens))
            qmm.rope_cache(s["cache"], held, k=s.pop("k"), v=s.pop("v"))
        return s, case
    shape = (s["pages"], heads, page, dim)
    for name in ("k", "v"):
        s["pool_" + name] = torch.zeros(shape, dtype=torch.int8 if q8 else TYPES[case["cache"]], device="cuda")
        if q8:
            s["scale_" + name] = torch.zeros((*shape[:3], dim // 32), dtype=torch.float16, device="cuda")
    if rope:
        s["places"] = _places(s, s["starts"], news, lens, page)
        return s, case
    at, slot, _ = _places(s, s["held"], lens, lens, page)
    for name in ("k", "v"):
        x = s.pop(name)
        if q8:
            codes, scales = _quantized(x.float())
            s["pool_" + name][at, :, slot] = codes
            s["scale_" + name][at, :, slot] = scales
        else:
            s["pool_" + name][at, :, slot] = x
    s["rows"] = (torch.cat([torch.full((n,), i) for i, n in enumerate(news)]).long().cuda(),
                 torch.cat([torch.arange(n) for n in news]).long().cuda())
    return s, case


def run(state):
    s, case = state
    if not own:
        return _run_rope(s, case) if case["op"] == "rope" else _run_attend(s, case)
    import quant_q8_gemm_amd as qmm
    cache, batch = s["cache"], s["batch"]
    if case["op"] == "rope":
        q8 = case["cache"] == "q8"
        q = qmm.rope_cache(cache, batch, q=s["q"], k=s["k"], v=s["v"], frequencies=s["frequencies"], magnitude=s["magnitude"],
                           layout=case["layout"], positions=s.get("positions"),
                           dtype=torch.float16 if q8 else TYPES[case["cache"]])
        k, v = qmm.cache_read(cache, batch, s["q"].shape[0], dtype=torch.float16) if q8 else cache.views()
        return {"q": q, "k": k, "v": v}
    out = qmm.attention(s["q"], cache, batch, causal=case["op"] == "attend", window=case["window"],
                        dtype="q8" if case["out"] == "q8" else None)
    if case["out"] == "q8":
        return qmm.dequantize_activations(out, s["q"].shape[0], case["heads"] * case["dim"], dtype=torch.float16)
    return out


def work(case):
    news, lens = _sizes(case)
    heads, kv_heads, dim, cache = case["heads"], case["kv_heads"], case["dim"], SIZE[case["cache"]]
    tokens = sum(news)
    if case["op"] == "rope":
        x = SIZE[case["x"]]
        # q, k and v read, q and the cache written; with q8 blocks the numbers that they stand for
        b = tokens * dim * (heads * (x + (2 if case["cache"] == "q8" else cache)) + 2 * kv_heads * (x + cache))
        if case["cache"] == "q8":
            b += tokens * dim * 2 * kv_heads * 2
        return {"bytes": b, "flops": tokens * (heads + kv_heads) * case["rotated"] * 3}
    pairs = slots = 0
    for new, length in zip(news, lens):
        if case["op"] == "cross":
            pairs += new * length
            slots += length if new else 0
        else:
            window = case["window"] or length
            pairs += sum(min(window, length - new + j + 1) for j in range(new))
            slots += min(length, new + window - 1) if new else 0
    out = 1.125 + 2 if case["out"] == "q8" else 2
    return {"bytes": 2 * slots * kv_heads * dim * cache + tokens * heads * dim * (2 + out), "flops": 4 * pairs * heads * dim}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------

def _exact_rope(s, case):
    """Each pair as a complex number times its turn."""
    f, magnitude = _frequencies(case)
    if "positions" in s:
        at = s["positions"].double()
    else:
        at = torch.cat([torch.arange(b - a, b) for a, b in zip(s["news"], s["lens"])]).double().cuda()
    turn = torch.polar(torch.full((), magnitude, dtype=torch.float64, device="cuda"),
                       torch.outer(at, torch.tensor(f, dtype=torch.float64, device="cuda")))[:, None]
    n = case["rotated"]

    def turned(x):
        x = x.double()
        part = x[..., :n]
        if case["layout"] == "half":
            z = torch.complex(part[..., :n // 2], part[..., n // 2:]) * turn
            part = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.complex(part[..., ::2], part[..., 1::2]) * turn
            part = torch.view_as_real(z).reshape(part.shape)
        return torch.cat([part, x[..., n:]], -1)

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
    if case["cache"] == "q8":
        return {"q": q, "k": _exact_q8(k), "v": _exact_q8(v)}
    page, dim, heads = case["page"], case["dim"], case["kv_heads"]
    pools = []
    for x in (k, v):
        pool = torch.zeros((s["pages"], page, heads, dim), dtype=torch.float64, device="cuda")
        t = 0
        for i, (new, length) in enumerate(zip(s["news"], s["lens"])):
            slots = torch.arange(length - new, length, device="cuda")
            pool[s["table"][i].long()[slots // page], slots % page] = x[t:t + new]
            t += new
        pools.append(pool.permute(0, 2, 1, 3).contiguous())
    k, v = pools
    return {"q": q, "k": k.view(s["pages"], heads, page // 32, 2, 2, 2, 4, dim // 16, 2, 8),
            "v": v.view(s["pages"], heads, page // 32, 2, 2, 8, dim // 32, 32)}


def _exact_q8(x):
    """What the q8 blocks of 64-bit numbers stand for; the scale and the quotient are rounded as the format says."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    scale = (torch.maximum(b.amax(-1), -b.amin(-1)).float().double() / 127).float().to(torch.float16).double()[..., None]
    q = torch.nan_to_num((b / scale).float().double(), nan=0.0, posinf=0.0, neginf=0.0)
    return (torch.round(q).clamp(-127, 127) * scale).reshape(x.shape)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros((sum(s["news"]), heads, dim), dtype=torch.float64, device="cuda")
    k, v = s["k"].double(), s["v"].double()
    if case["cache"] == "q8":
        k, v = _exact_q8(k), _exact_q8(v)
    t = at = 0
    for new, length in zip(s["news"], s["lens"]):
        for h in range(heads):
            if new == 0 or length == 0:
                break  # nothing to see: zeros
            kk, vv = (x[at:at + length, h * kv_heads // heads] for x in (k, v))
            w = (s["q"][t:t + new, h].double() @ kk.t().contiguous()) / math.sqrt(dim)
            if case["op"] == "attend":
                behind = torch.arange(length - new, length, device="cuda")[:, None] - torch.arange(length, device="cuda")
                w = torch.where((behind < 0) | (behind >= (case["window"] or length + 1)), -math.inf, w)
            out[t:t + new, h] = torch.softmax(w, 1) @ vv.contiguous()
        t += new
        at += length
    return _exact_q8(out.flatten(1)) if case["out"] == "q8" else out
