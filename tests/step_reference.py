"""Plain float64 references of the serving-step operators, written from their
definitions (CPU, one sequence at a time), and the inputs of their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

# half a step of a 16-bit element type, relative (0: float32 stays float32)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def plan(ctx, new, free, count, tables, max_tokens, bs, num_blocks, base=0):
    """The step plan, request by request.  Returns (tables, query_start,
    seq_lens, positions, slots, left, statuses)."""
    B, width = tables.shape
    tables = tables.copy()
    start, lens, pos, slots, seen = [0], [], [], [], set()
    if not 0 <= count <= len(free):
        count = 0
    left, rows, full = count, 0, False
    for b in range(B):
        C, n = int(ctx[b]), int(new[b])
        if C < 0 or n < 0 or C + n > width * bs:
            seen.add(8)
            C, n = min(max(C, 0), width * bs), 0
        have, need = -(-C // bs), -(-(C + n) // bs)
        if full or need - have > left or rows + n > max_tokens:
            full = True
            seen.add(10)
            n = need = 0
        for j in range(have, need):
            left -= 1
            tables[b, j] = free[left]
        for t in range(C, C + n):
            block = int(tables[b, t // bs])
            ok = 0 <= block < num_blocks
            if not ok:
                seen.add(7)
            slots.append(block * bs + t % bs if ok else -1)
            pos.append(base + t)
        rows += n
        start.append(rows)
        lens.append(C + n)
    pad = max_tokens - rows
    return (tables, np.array(start), np.array(lens), np.array(pos + [0] * pad),
            np.array(slots + [-1] * pad), left, seen)


def norm_rope(x, w, cos_sin, pos, eps, offset, interleaved):
    """x [T, H, D] normed (w not None) and rotated, float64."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (w.double() + offset)
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    out = y.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        c = cos_sin[pos.long(), j].double()[:, None]
        s = cos_sin[pos.long(), rot // 2 + j].double()[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def visible(p, window, sinks):
    """Tokens that the query at position p sees, in order."""
    return [t for t in range(p + 1) if t < sinks or t > p - window]


def attend(q, k, v, scale):
    """One row: q [D], k, v [n, D] -> (output, weighted mean of |v|), float64."""
    if k.shape[0] == 0:
        return torch.zeros_like(v[:0].sum(0)), torch.zeros_like(v[:0].sum(0))
    s = (k @ q) * scale
    w = torch.exp(s - s.max())
    w = w / w.sum()
    return w @ v, w @ v.abs()


def paged_rows(cache, table, tokens, bs):
    t = torch.as_tensor(list(tokens), dtype=torch.long)
    return cache[table[t // bs].long(), :, t % bs].double()


def rows_attend(q, k, v, scale):
    """q [Hq, D] over k, v [n, Hkv, D]: (out [Hq, D], mean |v| [Hq, D])."""
    G = q.shape[0] // k.shape[1]
    outs = [attend(q[h].double(), k[:, h // G], v[:, h // G], scale) for h in range(q.shape[0])]
    return torch.stack([o for o, _ in outs]), torch.stack([m for _, m in outs])


def assert_within(got, ref, mag, dtype, out_dtype, rounded_p, what=""):
    """|got - ref| against what rounding allows.  float32 sums: each logit is
    off by a few 2^-24 of sum |q k| (below 1e-5 here), so the weights by that
    relative amount: 2e-5 of the mean |v|.  ``rounded_p``: the weights enter
    the product with the values in 16 bits, half a step each, against a sum
    of the same or of unrounded ones: at most two half steps of the mean |v|.
    One rounding to the output type."""
    got, ref = got.double().cpu(), ref.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    u = HALF_STEP[dtype] if rounded_p and dtype != torch.float32 else 0.0
    bound = (2e-5 + 2 * u) * mag + 1e-6
    bound = bound + HALF_STEP[out_dtype] * (ref.abs() + bound)
    bad = (got - ref).abs() > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((got - ref).abs().max()):.3e}")


class Paged:
    """Random paged caches; ``ids`` of owned blocks are drawn without repeats,
    and what no test token owns is NaN."""

    def __init__(self, blocks, hkv, bs, d, dtype, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.bs, self.dtype = bs, dtype
        self.k = torch.full((blocks, hkv, bs, d), math.nan, dtype=dtype)
        self.v = torch.full((blocks, hkv, bs, d), math.nan, dtype=dtype)
        self.order = torch.randperm(blocks, generator=self.g).tolist()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, dtype=torch.float32).to(self.dtype)

    def fill(self, table, tokens):
        """Give the tokens of one sequence blocks (into ``table``) and values."""
        for t in tokens:
            if table[t // self.bs] < 0:
                table[t // self.bs] = self.order.pop()
        at = torch.as_tensor(list(tokens), dtype=torch.long)
        if len(at) == 0:
            return
        blk = table[at // self.bs].long()
        hkv, d = self.k.shape[1], self.k.shape[3]
        self.k[blk, :, at % self.bs] = self.randn(len(at), hkv, d)
        self.v[blk, :, at % self.bs] = self.randn(len(at), hkv, d)


def split_x(k, v):
    nb, hkv, bs, d = k.shape
    x = 16 // k.element_size()
    return (k.view(nb, hkv, bs, d // x, x).permute(0, 1, 3, 2, 4).contiguous(),
            v.permute(0, 1, 3, 2).contiguous())


def window_decode_problem(lens, window, sinks, hq, hkv, d, bs, dtype, seed):
    """(q, paged, tables, lens, ref, mag): only visible tokens have values and
    blocks; everything else is NaN, and table entries without a block are -1."""
    need = sum(len({t // bs for t in visible(L - 1, window, sinks)}) for L in lens)
    pg = Paged(need + 3, hkv, bs, d, dtype, seed)
    width = max(1, -(-max(lens) // bs))
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    q = pg.randn(len(lens), hq, d)
    ref, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b, L in enumerate(lens):
        see = visible(L - 1, window, sinks)
        pg.fill(tables[b], see)
        if see:
            ref[b], mag[b] = rows_attend(q[b], paged_rows(pg.k, tables[b], see, bs),
                                         paged_rows(pg.v, tables[b], see, bs), d ** -0.5)
    return q, pg, tables, torch.tensor(lens, dtype=torch.int32), ref, mag


def window_prefill_problem(ctx, new, window, sinks, hq, hkv, d, bs, dtype, seed):
    """Context tokens that no row sees are NaN and may have no block."""
    need, seen = 0, []
    for C, n in zip(ctx, new):
        s = sorted({t for p in range(C, C + n) for t in (list(range(min(sinks, C))) +
                    list(range(max(0, p - window + 1), C)))}) if n else []
        seen.append(s)
        need += len({t // bs for t in s})
    pg = Paged(need + 3, hkv, bs, d, dtype, seed)
    tables = torch.full((len(ctx), max(1, -(-max(ctx) // bs))), -1, dtype=torch.int32)
    T = sum(new)
    q, k, v = pg.randn(T, hq, d), pg.randn(T, hkv, d), pg.randn(T, hkv, d)
    ref, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    start = [0]
    for b, (C, n) in enumerate(zip(ctx, new)):
        pg.fill(tables[b], seen[b])
        s0 = start[-1]
        start.append(s0 + n)
        kk = torch.zeros(C + n, hkv, d, dtype=torch.float64)
        vv = torch.zeros(C + n, hkv, d, dtype=torch.float64)
        if seen[b]:
            kk[seen[b]] = paged_rows(pg.k, tables[b], seen[b], bs)
            vv[seen[b]] = paged_rows(pg.v, tables[b], seen[b], bs)
        kk[C:], vv[C:] = k[s0:s0 + n].double(), v[s0:s0 + n].double()
        for i in range(n):
            see = visible(C + i, window, sinks)
            ref[s0 + i], mag[s0 + i] = rows_attend(q[s0 + i], kk[see], vv[see], d ** -0.5)
    return (q, k, v, pg, tables, torch.tensor(start, dtype=torch.int32),
            torch.tensor(ctx, dtype=torch.int32), ref, mag)


def prefix_problem(prefix, lens, hq, hkv, d, bs, dtype, seed):
    blocks = -(-prefix // bs) + sum(-(-L // bs) for L in lens)
    pg = Paged(blocks + 3, hkv, bs, d, dtype, seed)
    shared = torch.full((max(1, -(-prefix // bs)),), -1, dtype=torch.int32)
    pg.fill(shared, range(prefix))
    tables = torch.full((len(lens), max(1, -(-max(lens) // bs))), -1, dtype=torch.int32)
    q = pg.randn(len(lens), hq, d)
    ref, mag = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    kp = paged_rows(pg.k, shared, range(prefix), bs)
    vp = paged_rows(pg.v, shared, range(prefix), bs)
    for b, L in enumerate(lens):
        pg.fill(tables[b], range(L))
        k = torch.cat([kp, paged_rows(pg.k, tables[b], range(L), bs)])
        v = torch.cat([vp, paged_rows(pg.v, tables[b], range(L), bs)])
        if k.shape[0]:
            ref[b], mag[b] = rows_attend(q[b], k, v, d ** -0.5)
    return q, pg, shared, tables, torch.tensor(lens, dtype=torch.int32), ref, mag
