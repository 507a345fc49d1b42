"""Plain float64 references of the 4-bit cache, written from its definition (CPU),
and the inputs of its tests."""
from __future__ import annotations

import math

import torch

from step_reference import HALF_STEP


def quantise(x, group):
    """Head rows x [.., D] -> (codes [.., D] whole numbers, scale, minimum [.., D / group]) in
    float64; the scale is rounded to x's type, groups that are not finite are NaN."""
    g = x.double().unflatten(-1, (-1, group))
    low, high = g.amin(-1), g.amax(-1)
    bad = ~torch.isfinite(g).all(-1) | ((high - low) > torch.finfo(torch.float32).max)
    scale = ((high - low) / 15).to(x.dtype).double()
    scale = torch.where(bad, math.nan, scale)
    low = torch.where(bad, math.nan, low)
    ratio = (g - low[..., None]) / scale[..., None]
    code = torch.where(scale[..., None] > 0, ratio.round().clamp(0, 15), 0.0)
    return code.flatten(-2), scale, low


def pack(code):
    c = code.to(torch.uint8)
    return c[..., 0::2] + 16 * c[..., 1::2]


def unpack(codes):
    out = torch.empty(codes.shape[:-1] + (codes.shape[-1] * 2,), dtype=torch.uint8)
    out[..., 0::2] = codes % 16
    out[..., 1::2] = codes // 16
    return out


def values(codes, pairs):
    """Values of packed codes [.., D / 2] and pairs [.., D / group, 2], float64."""
    c = unpack(codes).double()
    c = c.unflatten(-1, (pairs.shape[-2], -1))
    return (c * pairs[..., :1].double() + pairs[..., 1:].double()).flatten(-2)


class Pool:
    """A 4-bit cache.  What no test token owns has random codes and NaN scales."""

    def __init__(self, blocks, hkv, bs, d, group, dtype, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.bs, self.dtype, self.group, self.d, self.hkv = bs, dtype, group, d, hkv
        codes, pairs = (blocks, hkv, bs, d // 2), (blocks, hkv, bs, d // group, 2)
        self.k, self.v = (torch.randint(0, 256, codes, generator=self.g, dtype=torch.uint8)
                          for _ in range(2))
        self.ks, self.vs = (torch.full(pairs, math.nan, dtype=dtype) for _ in range(2))
        self.order = torch.randperm(blocks, generator=self.g).tolist()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, dtype=torch.float32).to(self.dtype)

    def put(self, blk, at, k, v):
        for x, codes, pairs in ((k, self.k, self.ks), (v, self.v, self.vs)):
            c, s, m = quantise(x, self.group)
            codes[blk, :, at] = pack(c)
            pairs[blk, :, at] = torch.stack([s, m], -1).to(self.dtype)

    def fill(self, table, n, spread=1.0, offset=0.0):
        """Blocks (into ``table``) and values for a sequence of n tokens."""
        for j in range(-(-n // self.bs)):
            table[j] = self.order.pop()
        t = torch.arange(n)
        if n:
            k = (self.randn(n, self.hkv, self.d).float() * spread + offset).to(self.dtype)
            v = (self.randn(n, self.hkv, self.d).float() + offset).to(self.dtype)
            self.put(table[t // self.bs].long(), t % self.bs, k, v)

    def rows(self, table, n):
        """(k, v, value scales per element), each [n, Hkv, D] in float64."""
        t = torch.arange(n)
        blk, at = table[t // self.bs].long(), t % self.bs
        s = self.vs[blk, :, at][..., 0].double().repeat_interleave(self.group, -1)
        return (values(self.k[blk, :, at], self.ks[blk, :, at]),
                values(self.v[blk, :, at], self.vs[blk, :, at]), s)

    def cuda(self):
        return tuple(x.cuda() for x in (self.k, self.v, self.ks, self.vs))


def decode_problem(lens, hq, hkv, d, bs, group, dtype, seed, spread=1.0, offset=0.0):
    """(q, pool, tables, lens, ref, mag, step): mag is the weighted mean of |v|, step that of
    the values' scales."""
    pool = Pool(sum(-(-n // bs) for n in lens) + 3, hkv, bs, d, group, dtype, seed)
    tables = torch.full((len(lens), max(1, -(-max(lens) // bs))), -1, dtype=torch.int32)
    q = pool.randn(len(lens), hq, d)
    ref, mag, step = (torch.zeros(q.shape, dtype=torch.float64) for _ in range(3))
    G = hq // hkv
    for b, n in enumerate(lens):
        pool.fill(tables[b], n, spread, offset)
        if n == 0:
            continue
        k, v, s = pool.rows(tables[b], n)
        for h in range(hq):
            a = (k[:, h // G] @ q[b, h].double()) * d ** -0.5
            w = torch.softmax(a, 0)
            ref[b, h] = w @ v[:, h // G]
            mag[b, h] = w @ v[:, h // G].abs()
            step[b, h] = w @ s[:, h // G]
    return q, pool, tables, torch.tensor(lens, dtype=torch.int32), ref, mag, step


def assert_decode(got, ref, mag, step, out_dtype, portable, logits=1.0, what=""):
    """|got - ref| against what rounding allows.  Logits are float32 sums of exact products, off
    by a few 2^-24 of sum |q k|, below 1e-5 where the logits are of order 1 (``logits``: how much
    larger they are here): the weights move by twice that, relatively, and a weighted mean with
    them.  The sums of codes and of minima cancel: each is at most 15 steps beyond the values.
    The tensor-core kernel rounds the weight and its product with the scale to float16, half a
    step 2^-11 each, and they multiply c - 8, at most 8.  One rounding to the output type."""
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    bound = 2e-5 * logits * (mag + 15 * step) + 1e-6
    if not portable:
        bound = bound + 2.0 ** -10 * 8 * step
    bound = bound + HALF_STEP[out_dtype] * (ref.abs() + bound)
    bad = (got - ref).abs() > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((got - ref).abs().max()):.3e}")
