"""Measured cases of the 4-bit paged cache and of the rotation with several axes.

Four operators: norm + rotation + cache write where each pair of the rotation
has one of several positions (time, height, width); the write of keys and
values into a paged cache of 4-bit codes with a scale and a minimum for each
group; the widening of such pages into 16-bit pages, for the prefill calls; and
decode attention over the 4-bit cache.

A group of elements of a head row holds codes c in 0..15 that stand for
c * scale + minimum; element 2i is the low half of byte i, 2i + 1 the high half.

``run`` with ``own`` false computes each in elementary torch operations in
32 bits; with ``own`` true it makes the library's calls.  ``exact`` computes
them in 64 bits, row by row or sequence by sequence, from the definitions.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # decode step of a model that takes images: 32 new rows, GQA 32/8, three axes one after
        # another
        dict(name="axes_decode_32", op="axes", tokens=32, heads=32, kv_heads=8, dim=128, rot=128,
             block=32, dtype="bf16", interleaved=False, split_x=False, sections="16/24/24",
             alternate=False),
        # a chunk of a video prompt, 24/4 heads of 256, three axes dealt out in turn
        dict(name="axes_video_8192", op="axes", tokens=8192, heads=24, kv_heads=4, dim=256,
             rot=256, block=16, dtype="bf16", interleaved=False, split_x=False,
             sections="48/40/40", alternate=True),
        # an image's odd number of rows in f16: two axes, partial rotation of neighbouring pairs,
        # into the split-x cache layout
        dict(name="axes_image_1001", op="axes", tokens=1001, heads=16, kv_heads=2, dim=128, rot=64,
             block=16, dtype="f16", interleaved=True, split_x=True, sections="16/16",
             alternate=False),
        # decode step: 32 new rows of 8 heads into the 4-bit cache
        dict(name="store_decode_32", op="store", tokens=32, heads=32, kv_heads=8, dim=128,
             group=64, block=32, dtype="bf16"),
        # a prefill chunk, with the values that the cache now stands for
        dict(name="store_chunk_8192", op="store", tokens=8192, heads=24, kv_heads=4, dim=256,
             group=64, block=16, dtype="bf16"),
        # an odd chunk in f16, as many KV heads as query heads, small groups
        dict(name="store_f16_1001", op="store", tokens=1001, heads=16, kv_heads=16, dim=128,
             group=32, block=16, dtype="f16"),
        # the cached context of a long prompt, widened before its next chunk
        dict(name="load_context_24576", op="load", seqs=1, len_lo=24576, len_hi=24576, kv_heads=4,
             dim=256, group=64, block=16, dtype="bf16"),
        # contexts of a ragged batch of chunks
        dict(name="load_ragged_33", op="load", seqs=33, len_lo=1, len_hi=6000, kv_heads=16,
             dim=128, group=32, block=16, dtype="f16"),
        # a few short requests: the latency of a call
        dict(name="decode_short_8", op="decode", seqs=8, len_lo=1, len_hi=200, heads=32,
             kv_heads=8, dim=128, group=64, block=32, dtype="bf16"),
        # one long conversation
        dict(name="decode_one_100k", op="decode", seqs=1, len_lo=100000, len_hi=100000, heads=24,
             kv_heads=4, dim=256, group=64, block=16, dtype="bf16"),
        # f16, as many query as KV heads, small groups
        dict(name="decode_f16_33", op="decode", seqs=33, len_lo=1000, len_hi=30000, heads=16,
             kv_heads=16, dim=128, group=32, block=16, dtype="f16"),
        # a serving batch, lengths from a few tokens to 100K, one group a head row
        dict(name="decode_serving_256", op="decode", seqs=256, len_lo=16, len_hi=100000, heads=32,
             kv_heads=8, dim=128, group=128, block=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "store", "load", "decode"])
    heads, kv_heads, dim, block = rng.choice(
        [(24, 4, 256, 16), (24, 4, 256, 32), (32, 8, 128, 32), (16, 16, 128, 16),
         (16, 2, 128, 64), (6, 1, 256, 16), (40, 8, 128, 16), (12, 4, 64, 16), (32, 2, 128, 16)])
    dtype = rng.choice(["bf16", "f16"])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    if op == "axes":
        rot = rng.choice([dim, dim // 2])
        axes, left, sections = rng.choice([2, 3, 3, 4]), rot // 2, []
        for a in range(axes - 1):
            sections.append(rng.randint(1, left // (axes - a)))
            left -= sections[-1]
        sections.insert(0, left)  # the first axis has the most pairs
        return dict(op=op, tokens=_log_int(rng, 1, 8000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rot, block=block, dtype=dtype, interleaved=rng.random() < 0.5,
                    split_x=rng.random() < 0.25, sections="/".join(map(str, sections)),
                    alternate=max(a + axes * (s - 1) for a, s in enumerate(sections) if a)
                    < rot // 2 and rng.random() < 0.5)
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 8000), heads=heads, kv_heads=kv_heads, dim=dim,
                    group=group, block=rng.choice([block, 8, 20]), dtype=dtype)
    if op == "load":
        return dict(op=op, seqs=_log_int(rng, 1, 40), len_lo=1, len_hi=_log_int(rng, 100, 20000),
                    kv_heads=kv_heads, dim=dim, group=group, block=block, dtype=dtype)
    return dict(op=op, seqs=_log_int(rng, 1, 100), len_lo=1, len_hi=_log_int(rng, 100, 100000),
                heads=heads, kv_heads=kv_heads, dim=dim, group=group, block=block, dtype=dtype)


def _lens(case):
    """Lengths of a case's requests, spread over the logarithm of their range: part of the case,
    not of the seed, so that ``work`` can count them."""
    n, lo, hi = case["seqs"], case["len_lo"], case["len_hi"]
    if lo >= hi:
        return np.full(n, lo, dtype=np.int64)
    r = np.random.RandomState([n, lo, hi])
    x = np.exp(r.uniform(np.log(lo), np.log(hi + 1), size=n)).astype(np.int64)
    return np.clip(x, lo, hi)


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _cover(a, b):
    return -(-a // b)


def _axis_of(c):
    """The axis of each pair of the rotation: sections one after another, or dealt out in turn
    (axis a > 0 has pairs a, a + axes, a + 2 axes, ..., the first axis what is left)."""
    sections = [int(x) for x in c["sections"].split("/")]
    if not c["alternate"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    of = [0] * sum(sections)
    for a, n in enumerate(sections):
        for i in range(n if a else 0):
            of[a + i * len(sections)] = a
    return of


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _prepare_axes(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, hq, hkv, d, bs = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    qkv = _normal((T, hq + 2 * hkv, d), dt, g)  # one projection's output; q, k, v are its slices
    blocks = _cover(T, bs) + 5
    if c["split_x"]:
        kc, vc = _normal((blocks, hkv, d // 8, bs, 8), dt, g), _normal((blocks, hkv, d, bs), dt, g)
    else:
        kc, vc = _normal((blocks, hkv, bs, d), dt, g), _normal((blocks, hkv, bs, d), dt, g)
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:T]
    if T >= 256:  # a chunk: whole blocks in any order
        slots = (torch.randperm(blocks, generator=g, device="cuda")[:, None] * bs
                 + torch.arange(bs, device="cuda")[None, :]).reshape(-1)[:T]
    far = 40000
    inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
    axis_of = _axis_of(c)
    axes = max(axis_of) + 1
    t = torch.arange(T, device="cuda")
    if T >= 256:  # frames of 16 x 28 patches after some text: frame, row, column (and one more)
        grid = [t // 448, t // 28 % 16, t % 28, t % 7]
        pos = torch.stack([17001 + x for x in grid[4 - axes - (axes < 4):][:axes]])
    else:         # decoded text: the axes move together, or lag after an image
        pos = torch.randint(0, far - 100, (1, T), generator=g, device="cuda") + torch.randint(
            0, 100, (axes, 1), generator=g, device="cuda")
    return dict(op="axes", heads=hq, kv_heads=hkv, dim=d, rot=c["rot"], block=bs,
                interleaved=c["interleaved"], split_x=c["split_x"], qkv=qkv, axis_of=axis_of,
                axis_at=torch.tensor(axis_of, device="cuda"),
                wq=1 + 0.1 * _normal((d,), torch.float32, g).to(dt),
                wk=1 + 0.1 * _normal((d,), torch.float32, g).to(dt), eps=1e-6,
                pos=pos.to(torch.int32).contiguous(), slots=slots.to(torch.int64).contiguous(),
                cos_sin=cos_sin, q_out=torch.empty((T, hq, d), dtype=dt, device="cuda"), kc=kc,
                vc=vc)


def _quantise(x, group):
    """Codes (uint8, two to a byte) and (scale, minimum) pairs of the head rows x [.., D]."""
    f = x.float().unflatten(-1, (-1, group))
    low = f.amin(-1, keepdim=True)
    scale = ((f.amax(-1, keepdim=True) - low) / 15).to(x.dtype).float()
    code = torch.where(scale > 0, torch.round((f - low) / scale).clamp(max=15), 0.0)
    code = code.flatten(-2).to(torch.uint8)
    pairs = torch.cat([scale, low], dim=-1).to(x.dtype)
    return code[..., 0::2] | (code[..., 1::2] << 4), pairs


def _widen(codes, pairs, dtype):
    """The values that codes [.., D / 2] and pairs [.., D / group, 2] stand for, in ``dtype``."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).to(dtype)
    c = c.unflatten(-1, (pairs.shape[-2], -1))
    return (c * pairs[..., :1].to(dtype) + pairs[..., 1:].to(dtype)).flatten(-2)


def _pool4(blocks, hkv, bs, d, group, dt, g, hot):
    """A pool of 4-bit pages: rows of N(0, 1), a thousandth of them ``hot`` times as large."""
    codes = torch.empty((blocks, hkv, bs, d // 2), dtype=torch.uint8, device="cuda")
    pairs = torch.empty((blocks, hkv, bs, d // group, 2), dtype=dt, device="cuda")
    step = max(1, (1 << 28) // (hkv * bs * d))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, hkv, bs, d), generator=g, device="cuda")
        large = torch.rand((n, 1, bs, 1), generator=g, device="cuda") < 0.001
        codes[i:i + n], pairs[i:i + n] = _quantise(torch.where(large, hot * x, x).to(dt), group)
    return codes, pairs


def _prepare_store(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, hq, hkv, d, bs = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    blocks = _cover(T, bs) + 5
    kc, ks = _pool4(blocks, hkv, bs, d, c["group"], dt, g, 1.0)
    vc, vs = _pool4(blocks, hkv, bs, d, c["group"], dt, g, 1.0)
    slots = (torch.randperm(blocks, generator=g, device="cuda")[:, None] * bs
             + torch.arange(bs, device="cuda")[None, :]).reshape(-1)[:T]
    out = dict(dtype=dt, device="cuda")
    return dict(op="store", kv_heads=hkv, group=c["group"], block=bs,
                k=_normal((T, hkv, d), dt, g),  # normed and rotated
                qkv=_normal((T, hq + 2 * hkv, d), dt, g),  # the values are its last heads
                slots=slots.contiguous(), kc=kc, ks=ks, vc=vc, vs=vs,
                k_out=torch.empty((T, hkv, d), **out), v_out=torch.empty((T, hkv, d), **out))


def _tables(counts, pool, seed):
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pool)[: int(counts.sum())]
    t = np.full((len(counts), int(counts.max())), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(counts):
        t[r, :n] = ids[at:at + n]
        at += n
    return t


def _prepare_load(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    hkv, d, bs = c["kv_heads"], c["dim"], c["block"]
    lens = _lens(c)
    counts = _cover(lens, bs)
    pool, wide = int(counts.sum()) + 9, int(counts.sum()) + 3
    kc, ks = _pool4(pool, hkv, bs, d, c["group"], dt, g, 1.0)
    vc, vs = _pool4(pool, hkv, bs, d, c["group"], dt, g, 1.0)
    out = dict(dtype=dt, device="cuda")
    return dict(op="load", block=bs, kc=kc, ks=ks, vc=vc, vs=vs,
                tables=_i32(_tables(counts, pool, seed)),
                to=_i32(_tables(counts, wide, seed + 1)), counts=counts.tolist(), lens=_i32(lens),
                max_len=int(lens.max()), k_wide=torch.zeros((wide, hkv, bs, d), **out),
                v_wide=torch.zeros((wide, hkv, bs, d), **out))


def _prepare_decode(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    B, hq, hkv, d, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    lens = _lens(c)
    counts = _cover(lens, bs)
    pool = int(counts.sum()) + 3
    kc, ks = _pool4(pool, hkv, bs, d, c["group"], dt, g, 6.0)
    vc, vs = _pool4(pool, hkv, bs, d, c["group"], dt, g, 1.0)
    return dict(op="decode", block=bs, q=_normal((B, hq, d), dt, g), kc=kc, ks=ks, vc=vc, vs=vs,
                tables=_i32(_tables(counts, pool, seed)), lens=_i32(lens),
                host_lens=lens.tolist(), max_len=int(lens.max()), scale=1.0 / math.sqrt(d),
                out=torch.empty((B, hq, d), dtype=dt, device="cuda"))


_PREPARE = dict(axes=_prepare_axes, store=_prepare_store, load=_prepare_load,
                decode=_prepare_decode)


# ----------------------------------------------------------------------- run

def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _qkv(s):
    hq, hkv = s["heads"], s["kv_heads"]
    return s["qkv"][:, :hq], s["qkv"][:, hq:hq + hkv], s["qkv"][:, hq + hkv:]


def _plain_norm_rope(x, w, cos, sin, s):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    rot = s["rot"]
    y = x[..., :rot]
    if s["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_axes(s):
    q, k, v = _qkv(s)
    half = s["rot"] // 2
    at = s["pos"].long()[s["axis_at"]].T  # [T, pairs]: each pair's position
    j = torch.arange(half, device=at.device)
    cos, sin = s["cos_sin"][at, j][:, None], s["cos_sin"][at, half + j][:, None]
    dt = q.dtype
    s["q_out"].copy_(_plain_norm_rope(q, s["wq"], cos, sin, s).to(dt))
    kr = _plain_norm_rope(k, s["wk"], cos, sin, s).to(dt)
    blk, at = s["slots"] // s["block"], s["slots"] % s["block"]
    if s["split_x"]:
        s["kc"][blk, :, :, at] = kr.view(kr.shape[0], kr.shape[1], -1, s["kc"].shape[-1])
        s["vc"][blk, :, :, at] = v
    else:
        s["kc"][blk, :, at] = kr
        s["vc"][blk, :, at] = v
    return dict(q=s["q_out"], kc=s["kc"], vc=s["vc"])


def _own_axes(s):
    import paged_attention_decode_v2_gb300 as pa
    q, k, v = _qkv(s)
    pa.qk_norm_rope_axes(q, k, v, s["pos"], s["slots"], s["cos_sin"], s["q_out"], s["kc"], s["vc"],
                         axis_of=s["axis_of"], q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                         interleaved=s["interleaved"], split_x=s["split_x"])
    return dict(q=s["q_out"], kc=s["kc"], vc=s["vc"])


def _stored(s):
    """The pools after the write, codes as whole numbers, and the values of the new rows."""
    return dict(k_codes=s["kc"], v_codes=s["vc"], k_scales=s["ks"], v_scales=s["vs"],
                k=s["k_out"], v=s["v_out"])


def _plain_store(s):
    blk, at = s["slots"] // s["block"], s["slots"] % s["block"]
    v = s["qkv"][:, -s["kv_heads"]:]
    for x, codes, pairs, out in ((s["k"], s["kc"], s["ks"], s["k_out"]),
                                 (v, s["vc"], s["vs"], s["v_out"])):
        c, p = _quantise(x, s["group"])
        codes[blk, :, at] = c
        pairs[blk, :, at] = p
        out.copy_(_widen(c, p, torch.float32).to(out.dtype))
    return _stored(s)


def _own_store(s):
    import paged_attention_decode_v2_gb300 as pa
    pa.store_kv4(s["k"], s["qkv"][:, -s["kv_heads"]:], s["slots"], s["kc"], s["vc"], s["ks"],
                 s["vs"], k_out=s["k_out"], v_out=s["v_out"])
    return _stored(s)


def _plain_load(s):
    for b, n in enumerate(s["counts"]):
        of, to = s["tables"][b, :n].long(), s["to"][b, :n].long()
        s["k_wide"][to] = _widen(s["kc"][of], s["ks"][of], torch.float32).to(s["k_wide"].dtype)
        s["v_wide"][to] = _widen(s["vc"][of], s["vs"][of], torch.float32).to(s["v_wide"].dtype)
    return dict(k=s["k_wide"], v=s["v_wide"])


def _own_load(s):
    import paged_attention_decode_v2_gb300 as pa
    pa.load_kv4(s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["to"], s["k_wide"],
                s["v_wide"], max_seq_len=s["max_len"])
    return dict(k=s["k_wide"], v=s["v_wide"])


def _plain_decode(s):
    bs = s["block"]
    hkv, d = s["kc"].shape[1], s["q"].shape[2]
    for b, L in enumerate(s["host_lens"]):
        blk = s["tables"][b, :_cover(L, bs)].long()
        k = _widen(s["kc"][blk], s["ks"][blk], torch.float32).transpose(0, 1).flatten(1, 2)[:, :L]
        v = _widen(s["vc"][blk], s["vs"][blk], torch.float32).transpose(0, 1).flatten(1, 2)[:, :L]
        q = s["q"][b].float().view(hkv, -1, d)
        a = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
        p = torch.exp(a - a.amax(-1, keepdim=True))
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        s["out"][b].copy_(o.reshape(-1, d).to(s["out"].dtype))
    return s["out"]


def _own_decode(s):
    import paged_attention_decode_v2_gb300 as pa
    if "ws" not in s:
        s["ws"] = pa.alloc_kv4_workspace(s["q"], s["kc"], s["ks"], s["tables"],
                                         max_seq_len=s["max_len"])
    return pa.decode_kv4(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"],
                         s["out"], s["ws"], max_seq_len=s["max_len"], scale=s["scale"])


_PLAIN = dict(axes=_plain_axes, store=_plain_store, load=_plain_load, decode=_plain_decode)
_OWN = dict(axes=_own_axes, store=_own_store, load=_own_load, decode=_own_decode)


# ---------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    d = c["dim"]
    if op == "axes":
        rows = c["tokens"] * (c["heads"] + 2 * c["kv_heads"])
        axes = c["sections"].count("/") + 1
        return {"bytes": 2 * rows * d * 2 + c["tokens"] * (4 * c["rot"] + 4 * axes + 8) + 2 * d * 2,
                "flops": 8 * rows * d}
    row = d // 2 + d // c["group"] * 4  # a head row's codes, scales and minima
    if op == "store":
        rows = 2 * c["tokens"] * c["kv_heads"]
        return {"bytes": rows * (2 * d * 2 + row) + 8 * c["tokens"], "flops": 5 * rows * d}
    lens = _lens(c)
    if op == "load":  # whole pages
        pages = int(_cover(lens, c["block"]).sum())
        rows = 2 * pages * c["block"] * c["kv_heads"]
        return {"bytes": rows * (row + 2 * d) + 8 * pages, "flops": 2 * rows * d}
    tokens = int(lens.sum())
    return {"bytes": 2 * tokens * c["kv_heads"] * row + 2 * c["seqs"] * c["heads"] * d * 2,
            "flops": 4 * d * c["heads"] * tokens}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of ``run`` in 64 bits."""
    return _EXACT[case["op"]](prepare(case, seed))


def _exact_axes(s):
    hq, hkv, rot = s["heads"], s["kv_heads"], s["rot"]
    x = s["qkv"].double()
    w = torch.cat([s["wq"].double().expand(hq, -1), s["wk"].double().expand(hkv, -1)])
    y = x[:, :hq + hkv]
    y = y / torch.sqrt(torch.mean(y ** 2, dim=-1, keepdim=True) + s["eps"]) * w
    turn = []
    for j, axis in enumerate(s["axis_of"]):  # a pair's factor, row by row
        at = s["cos_sin"][s["pos"][axis].long()].double()
        turn.append(torch.complex(at[:, j], at[:, rot // 2 + j]))
    turn = torch.stack(turn, dim=1)[:, None]
    z = y[..., :rot].unflatten(-1, (rot // 2, 2) if s["interleaved"] else (2, rot // 2))
    pair = -1 if s["interleaved"] else -2
    z = torch.complex(z.select(pair, 0), z.select(pair, 1)) * turn
    y = torch.cat([torch.stack([z.real, z.imag], dim=pair).flatten(-2), y[..., rot:]], dim=-1)
    kc, vc = s["kc"].double(), s["vc"].double()
    k, v = y[:, hq:], x[:, hq + hkv:]
    for t, slot in enumerate(s["slots"].tolist()):
        b, at = divmod(slot, s["block"])
        if s["split_x"]:
            kc[b, :, :, at] = k[t].view(hkv, -1, kc.shape[-1])
            vc[b, :, :, at] = v[t]
        else:
            kc[b, :, at] = k[t]
            vc[b, :, at] = v[t]
    return dict(q=y[:, :hq], kc=kc, vc=vc)


def _exact_store(s):
    out = dict(k_codes=None, v_codes=None)
    place = s["slots"].tolist()
    bs, group = s["block"], s["group"]
    for name, x, pairs in (("k", s["k"], s["ks"]), ("v", s["qkv"][:, -s["kv_heads"]:], s["vs"])):
        x = x.double()
        n = x.shape[-1] // group
        parts, values = [], []
        for i in range(n):  # a group's step, smallest value, and the values on that grid
            part = x[..., i * group:(i + 1) * group]
            low = part.min(dim=-1).values
            step = ((part.max(dim=-1).values - low) / 15.0).to(pairs.dtype).double()
            grid = torch.div(part - low[..., None], step[..., None]).round().clamp(0, 15)
            grid = torch.where(step[..., None] > 0, grid, 0.0)
            values.append(low[..., None] + step[..., None] * grid)
            parts.append(torch.stack([step, low], dim=-1))
        out[name] = torch.cat(values, dim=-1)
        new = torch.stack(parts, dim=2)
        pool = pairs.double()
        for t, slot in enumerate(place):
            pool[slot // bs, :, slot % bs] = new[t]
        out[name + "_scales"] = pool
    return out


def _values64(codes, pairs):
    """Values of head rows in 64 bits: the even and the odd elements, then woven together."""
    d = codes.shape[-1] * 2
    x = torch.empty(codes.shape[:-1] + (d,), dtype=torch.float64, device=codes.device)
    x[..., 0::2] = torch.remainder(codes, 16).double()
    x[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    each = d // pairs.shape[-2]
    return x.mul_(pairs[..., 0].double().repeat_interleave(each, dim=-1)).add_(
        pairs[..., 1].double().repeat_interleave(each, dim=-1))


def _exact_load(s):
    k, v = s["k_wide"].double(), s["v_wide"].double()
    for b, n in enumerate(s["counts"]):
        for of, to in zip(s["tables"][b, :n].split(512), s["to"][b, :n].split(512)):
            k[to.long()] = _values64(s["kc"][of.long()], s["ks"][of.long()])
            v[to.long()] = _values64(s["vc"][of.long()], s["vs"][of.long()])
    return dict(k=k, v=v)


def _exact_decode(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    bs, hkv, d = s["block"], s["kc"].shape[1], s["q"].shape[2]
    for b, L in enumerate(s["host_lens"]):
        t = torch.arange(L, device="cuda")
        blk = s["tables"][b].long()[t // bs]
        q = s["q"][b].double().view(hkv, -1, d)
        for h in range(hkv):
            k = _values64(s["kc"][blk, h, t % bs], s["ks"][blk, h, t % bs])
            w = torch.softmax(torch.mm(q[h], k.T) * s["scale"], dim=-1)
            v = _values64(s["vc"][blk, h, t % bs], s["vs"][blk, h, t % bs])
            out[b].view(hkv, -1, d)[h] = torch.mm(w, v)
    return out


_EXACT = dict(axes=_exact_axes, store=_exact_store, load=_exact_load, decode=_exact_decode)
