"""A paged key-value cache for the tests, and the attention over it in float64. Everything starts as NaN: what no call
wrote, and what lies behind a sequence's last token, must not reach any result."""
from __future__ import annotations

import math
import random

import torch

E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100


def quantize(x):
    """Codes and scales of float32 x, one scale for the last dimension, step by step as the contract states."""
    a = x.abs().amax(-1).clamp_min(FLOOR)
    return (x * (torch.tensor(448.0) / a)[..., None]).to(E4M3), a * (torch.tensor(1.0) / torch.tensor(448.0))


class Cache:
    """Pages on the CPU with the strides of `layout`; device() copies them, strides and all."""

    def __init__(self, lengths, H, D, page, e4m3=False, layout="heads", seed=0, spare=2, cols_more=1):
        rng = random.Random(seed)
        self.H, self.D, self.S, self.e4m3, self.layout = H, D, page, e4m3, layout
        held = [-(-n // page) for n in lengths]
        self.P = sum(held) + spare
        order = list(range(self.P))
        rng.shuffle(order)
        cols = max(max(held) + cols_more, 1)
        self.table = torch.full((len(lengths), cols), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            self.table[b, n:] = rng.choice([-1, self.P, 2 ** 31 - 1, -2 ** 31])  # no pages either way
            at += n
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.store, self.k, self.v = self._empty(torch.bfloat16 if not e4m3 else torch.uint8, (D,), 0x7F)
        self.scale_store, self.ks, self.vs = self._empty(torch.float32, (), None) if e4m3 else (None, None, None)

    def _empty(self, dtype, tail, code):
        P, H, S = self.P, self.H, self.S
        fill = math.nan if code is None or dtype != torch.uint8 else code
        if self.layout == "tokens":
            store = torch.full((2, P, S, H, *tail), fill, dtype=dtype)
            k, v = (store[i].transpose(1, 2) for i in range(2))
        elif self.layout == "both":
            store = torch.full((P, 2, H, S, *tail), fill, dtype=dtype)
            k, v = store[:, 0], store[:, 1]
        elif self.layout == "gaps":
            store = torch.full((2, P, H + 1, S + 2, *(n + 16 for n in tail)), fill, dtype=dtype)
            k, v = (store[i][:, :H, 1:S + 1, ..., :self.D] if tail else store[i][:, :H, 1:S + 1] for i in range(2))
        else:
            store = torch.full((2, P, H, S, *tail), fill, dtype=dtype)
            k, v = store[0], store[1]
        return store, k, v

    def place(self, b, i):
        return int(self.table[b, i // self.S]), i % self.S

    def fill(self, seed=1, scale=1.0):
        """Values in every place that a sequence holds; the values that they stand for, float64 [n, H, D] of each."""
        g = torch.Generator().manual_seed(seed)
        self.keys, self.values = [], []
        for b, n in enumerate(self.lengths.tolist()):
            pair = []
            for pages, scales in ((self.k, self.ks), (self.v, self.vs)):
                x = (torch.randn(n, self.H, self.D, generator=g) * scale + 0.25).bfloat16()
                i = torch.arange(n)
                p, o = self.table[b].long()[i // self.S], i % self.S
                if self.e4m3:
                    c, s = quantize(x.float())
                    pages[p, :, o] = c.view(torch.uint8)
                    scales[p, :, o] = s
                    pair.append(c.float().double() * s.double()[..., None])
                else:
                    pages[p, :, o] = x
                    pair.append(x.double())
            self.keys.append(pair[0])
            self.values.append(pair[1])
        return self

    def device(self):
        """k_pages, v_pages, table, lengths, and the scales as keywords, on the GPU."""
        def view(like, store, on):
            return on.as_strided(like.shape, like.stride(), like.storage_offset())
        self.on = self.store.cuda()
        k, v = view(self.k, self.store, self.on), view(self.v, self.store, self.on)
        self.more = {}
        if self.e4m3:
            k, v = k.view(E4M3), v.view(E4M3)
            self.scales_on = self.scale_store.cuda()
            self.more = {"k_scales": view(self.ks, self.scale_store, self.scales_on),
                         "v_scales": view(self.vs, self.scale_store, self.scales_on)}
        self.args = (k, v, self.table.cuda(), self.lengths.cuda())
        return self.args


def attention(cache, q, starts, scale, window=0, sinks=0, gone=()):
    """(out, tolerance) in float64 for rows starts[b] .. starts[b + 1]; `gone`: (b, page column) that are no pages.

    Tolerance, element by element: p is rounded to bf16, at most 2^-8 of it, and so is the result; with A = sum p |v| / sum p
    that is 2^-8 A + 2^-8 (|o| + 2^-8 A). A score is a float32 sum of D exact products, off by at most D 2^-23 sum |q k| scale,
    and a few float32 roundings of its value and of exp2: twice that on each p, numerator and denominator."""
    T, Hq, D = q.shape
    G = Hq // cache.H
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, n in enumerate(cache.lengths.tolist()):
        t0, t1 = int(starts[b]), int(starts[b + 1])
        if t1 <= t0:
            continue
        i = torch.arange(t0, t1) + (n - t1)
        j = torch.arange(n)
        seen = (j[None] <= i[:, None])
        if window:
            seen &= (i[:, None] - j[None] < window) | (j[None] < sinks)
        for bb, col in gone:
            if bb == b:
                seen &= (j // cache.S != col)[None]
        for h in range(Hq):
            k, v = cache.keys[b][:, h // G], cache.values[b][:, h // G]
            x = q[t0:t1, h].double()
            z = (x @ k.t()) * scale
            some = seen.any(1)
            zz = z.masked_fill(~seen, -math.inf)
            p = torch.exp(zz - torch.where(some, zz.amax(1) if n else torch.zeros(t1 - t0, dtype=torch.float64), 0.0)[:, None])
            p = torch.where(some[:, None], p / p.sum(1, keepdim=True).clamp_min(1e-300), 0.0) if n else p
            out[t0:t1, h] = p @ v
            A = p @ v.abs()
            dz = D * 2.0 ** -23 * scale * (x.abs() @ k.abs().t()).amax(1, keepdim=True) if n else torch.zeros(t1 - t0, 1)
            dz = dz + 8 * 2.0 ** -23 * (1 + z.abs().amax(1, keepdim=True) if n else 1)
            tol[t0:t1, h] = (2.0 ** -8 + 4 * dz) * A + 2.0 ** -8 * (out[t0:t1, h].abs() + (2.0 ** -8 + 4 * dz) * A)
    return out, tol


def rotate(x, angle, interleaved):
    """(y, tolerance of float32) of float64 x [T, H, D] by angle [T, n / 2]: float32 sine and cosine, two products and a sum."""
    half = angle.shape[1]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    y, tol = x.clone(), torch.zeros_like(x)
    ia, ib = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    # 2^-22 for sine and cosine (a float32 remainder of a turn, and the functions), 2^-24 for each product and the sum
    tol[..., ia] = tol[..., ib] = (a.abs() + b.abs()) * (2.0 ** -21 + 4 * 2.0 ** -24)
    return y, tol
