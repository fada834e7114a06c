"""Paged caches for tests: the documented tile layout, written out element by element, and attention and rotary positions
in 64 bits."""
import math

import numpy as np
import torch

import oracle

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def row_of(r):
    return (r & ~12) | ((r & 4) << 1) | ((r & 8) >> 1)


def _index(page, dim, which, q8):
    """[slot][channel] -> element (or byte) in a head's tiles of a page."""
    r = np.arange(page)[:, None]
    d = np.arange(dim)[None, :]
    tile, r = r // 32, r % 32
    if q8:
        if which == "k":
            at = d // 32 * 1024 + ((d % 16 // 8) * 32 + row_of(r)) * 16 + d % 32 // 16 * 8 + d % 8
        else:
            at = d // 32 * 1024 + ((r % 16 // 8) * 32 + d % 32) * 16 + r // 16 * 8 + r % 8
        return tile * 34 * dim + at
    if which == "k":
        return tile * 32 * dim + ((d // 16 * 2 + d % 16 // 8) * 32 + row_of(r)) * 8 + d % 8
    return tile * 32 * dim + ((d // 32 * 4 + r // 8) * 32 + d % 32) * 8 + r % 8


def _scale_index(page, dim):
    r = np.arange(page)[:, None]
    b = np.arange(dim // 32)[None, :]
    return r // 32 * 34 * dim + 32 * dim + (b * 32 + r % 32) * 2


def quantized(x):
    """torch numbers [..., dim] -> (codes int8, scales float16) as the library's q8 blocks (its oracle's rounding)."""
    shape = x.shape
    flat = x.reshape(-1, 32).float().contiguous()
    rows = -(-flat.shape[0] // 8) * 8  # the oracle takes rows of 256
    padded = np.zeros((rows, 32), np.float32)
    padded[:flat.shape[0]] = flat.numpy()
    q, dh, _ = oracle.quantize(padded.reshape(-1, 256))
    q, dh = q.reshape(-1, 32)[:flat.shape[0]], dh.reshape(-1)[:flat.shape[0]].view(np.float16)
    return torch.from_numpy(q.copy()).reshape(shape), torch.from_numpy(dh.copy()).reshape(*shape[:-1], shape[-1] // 32)


def held(x, dtype):
    """What a cache holds of numbers x, as the product takes them, in 64 bits."""
    if dtype == "q8":
        q, s = quantized(x)
        return (q.unflatten(-1, (-1, 32)).float() * s.float().unsqueeze(-1)).flatten(-2).half().double()
    return x.to(dtype).double()


def packed(x, dtype, which):
    """[n_pages][heads][page][dim] -> the pool's bytes."""
    n, heads, page, dim = x.shape
    if dtype == "q8":
        q, s = quantized(x)
        out = np.zeros((n, heads, page // 32 * 34 * dim), np.uint8)
        out[:, :, _index(page, dim, which, True)] = (q.numpy().astype(np.int16) + 128).astype(np.uint8)
        at = _scale_index(page, dim)
        bits = s.numpy().view(np.uint16)
        out[:, :, at] = (bits & 255).astype(np.uint8)
        out[:, :, at + 1] = (bits >> 8).astype(np.uint8)
        return torch.from_numpy(out.reshape(-1))
    out = np.zeros((n, heads, page * dim), np.uint16)
    out[:, :, _index(page, dim, which, False)] = x.to(dtype).contiguous().view(torch.int16).numpy().view(np.uint16)
    return torch.from_numpy(out.reshape(-1).view(np.uint8))


def unpacked(pool, dtype, which, n, heads, page, dim):
    """The pool's bytes -> numbers [n_pages][heads][page][dim]."""
    b = pool.cpu().numpy()
    if dtype == "q8":
        b = b.reshape(n, heads, -1)
        q = b[:, :, _index(page, dim, which, True)].astype(np.int16) - 128
        at = _scale_index(page, dim)
        s = (b[:, :, at].astype(np.uint16) | (b[:, :, at + 1].astype(np.uint16) << 8)).view(np.float16)
        return torch.from_numpy(q.astype(np.float32) * np.repeat(s.astype(np.float32), 32, -1))
    b = b.view(np.uint16).reshape(n, heads, -1)[:, :, _index(page, dim, which, False)]
    return torch.from_numpy(b.astype(np.int16)).view(dtype).float()


class Paged:
    """Sequences of `lens` slots with `news` new tokens each, in shuffled pages; junk in every slot that is not in use."""

    def __init__(self, news, lens, heads, kv_heads, dim, dtype, page=32, seed=0, junk=float("nan"), spare=2):
        g = torch.Generator().manual_seed(seed)
        self.news, self.lens, self.heads, self.kv_heads, self.dim, self.page = list(news), list(lens), heads, kv_heads, dim, page
        self.dtype = dtype
        self.type = torch.float16 if dtype == "q8" else dtype
        columns = [-(-n // page) for n in lens]
        self.n_pages = sum(columns) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(1, max(columns))), -1, dtype=torch.int32)
        self.k = [torch.randn(n, kv_heads, dim, generator=g) for n in lens]
        self.v = [torch.randn(n, kv_heads, dim, generator=g) for n in lens]
        self.q = (torch.randn(sum(news), heads, dim, generator=g) * 1.5).to(self.type)
        self.where = []
        at = 0
        for i, c in enumerate(columns):
            self.where.append(order[at:at + c])
            self.table[i, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
        self.junk = junk

    def pools(self):
        """(k, v) as the pools' bytes"""
        out = []
        for which, xs in (("k", self.k), ("v", self.v)):
            shape = (self.n_pages, self.kv_heads, self.page, self.dim)
            x = torch.full(shape, self.junk)
            used = torch.zeros(self.n_pages, self.page, dtype=torch.bool)
            for s, pages in zip(xs, self.where):
                j = torch.arange(s.shape[0])
                at = torch.tensor(pages, dtype=torch.long)[j // self.page] if len(pages) else j
                x[at, :, j % self.page] = s
                used[at, j % self.page] = True
            if self.dtype == "q8":  # blocks of finite numbers; those not in use have junk as their scale
                p = packed(torch.where(used[:, None, :, None], x, 1.0), "q8", which)
                b = p.numpy().reshape(self.n_pages, self.kv_heads, -1)
                at = _scale_index(self.page, self.dim)
                junk = int(np.float16(self.junk).view(np.uint16))
                for page, row in (~used).nonzero().tolist():
                    b[page][:, at[row]], b[page][:, at[row] + 1] = junk & 255, junk >> 8
            else:
                p = packed(x, self.dtype, which)
            out.append(p)
        return out

    def starts(self):
        return torch.tensor(np.concatenate([[0], np.cumsum(self.news)]), dtype=torch.int32)

    def cuda(self, qmm, **hints):
        """(cache, batch, q) on the GPU."""
        k, v = self.pools()
        cache = qmm.Cache(self.n_pages, self.kv_heads, self.dim, page=self.page, dtype=self.dtype, k=k.cuda(), v=v.cuda())
        hints = {"max_new": max(self.news), "max_length": max(self.lens), **hints}
        batch = qmm.Batch(self.starts().cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.table.cuda(), **hints)
        return cache, batch, self.q.cuda()

    def seen(self, i, causal, window):
        """[new][length] of sequence i"""
        new, length = self.news[i], self.lens[i]
        if not causal:
            return torch.ones(new, length, dtype=torch.bool)
        behind = torch.arange(length - new, length)[:, None] - torch.arange(length)[None]
        return (behind >= 0) & (behind < (window or length + 1))

    def reference(self, causal=True, window=0, scale=None):
        """(outputs in 64 bits, how far a kernel's may be off before they are stored): [n_tok][heads][dim].

        With u half a step of the products' type and f = 2^-24: a score is off by at most (dim + 3) f scale sum|q k| and
        its power of two by that, relative, and another 2^-21 for its argument's rounding per unit of |scale s| (a score
        minus the maximum, both in base 2) and 2^-22 of its own; p is rounded by u (below f16's normal range by
        2^-25 at most); a product of n keys and their sum add n + 64 rounded steps each, n/32 + 8 rescalings among them."""
        scale = self.dim ** -0.5 if scale is None else scale
        out = torch.zeros(sum(self.news), self.heads, self.dim, dtype=torch.float64)
        off = torch.zeros_like(out)
        f, u, t = 2.0 ** -24, HALF[self.type], 0
        for i, (new, n) in enumerate(zip(self.news, self.lens)):
            if new and n:
                k, v = (held(x[i], self.dtype).repeat_interleave(self.heads // self.kv_heads, 1).transpose(0, 1)
                        for x in (self.k, self.v))
                q = self.q[t:t + new].double().transpose(0, 1)
                seen = self.seen(i, causal, window)
                s = (q @ k.transpose(1, 2)).masked_fill(~seen, -math.inf) * scale
                top = s.amax(2, keepdim=True)
                p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                total = p.sum(2, keepdim=True)
                p = p / torch.where(total == 0, torch.ones_like(total), total)
                wrong = (self.dim + 3) * f * scale * (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(2, keepdim=True)
                wrong = wrong + s.masked_fill(~seen, 0).abs().amax(2, keepdim=True) * 2.0 ** -21
                far = u + 2 * (wrong + 2.0 ** -22) + (3 * n + 200) * f
                clean = v.nan_to_num(0.0, 0.0, 0.0)
                out[t:t + new] = (p @ clean).transpose(0, 1)
                off[t:t + new] = (far * (p @ clean.abs()) + 2.0 ** -25 * (seen.double() @ clean.abs())).transpose(0, 1)
            t += new
        return out, off


def rotated(x, positions, frequencies, magnitude, layout):
    """x [n_tok][heads][dim] turned, in 64 bits."""
    x = x.double()
    n = 2 * len(frequencies)
    angle = positions.double()[:, None] * torch.as_tensor(frequencies)[None]
    cos, sin = torch.cos(angle)[:, None] * magnitude, torch.sin(angle)[:, None] * magnitude
    a, b = (x[..., :n // 2], x[..., n // 2:n]) if layout == "half" else (x[..., 0:n:2], x[..., 1:n:2])
    c, d = a * cos - b * sin, a * sin + b * cos
    y = x.clone()
    if layout == "half":
        y[..., :n // 2], y[..., n // 2:n] = c, d
    else:
        y[..., 0:n:2], y[..., 1:n:2] = c, d
    return y
