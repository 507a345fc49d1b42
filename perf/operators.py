"""Measured cases of the serving operators around paged attention.

Five operators, in the order a serving step calls them: the step plan (block
tables, slots and positions from request lengths), the per-head norm +
rotation + cache write, decode attention with a sliding window and sinks, its
prefill form, and decode attention of a batch that shares a prefix.

``run`` with ``own`` false computes each in elementary torch operations in
32 bits; with ``own`` true it makes the library's calls.  ``exact`` computes
them in 64 bits, sequence by sequence, from the definitions.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's bookkeeping of a full serving batch: every request appends a token
        dict(name="plan_decode_256", op="plan", seqs=256, ctx_lo=16, ctx_hi=32768, new_lo=1,
             new_hi=1, block=16),
        # many requests, decodes and long prefill chunks side by side
        dict(name="plan_mixed_1000", op="plan", seqs=1000, ctx_lo=1, ctx_hi=20000, new_lo=1,
             new_hi=500, block=32),
        # decode step: 32 new rows, GQA 32/8 (the serving batch's heads)
        dict(name="norm_rope_decode_32", op="rope", tokens=32, heads=32, kv_heads=8, dim=128,
             rot=128, block=32, dtype="bf16", interleaved=False, split_x=False),
        # one prefill chunk of 8192 rows, 24/4 heads of 256 (the long-context batch's heads)
        dict(name="norm_rope_chunk_8192", op="rope", tokens=8192, heads=24, kv_heads=4, dim=256,
             rot=256, block=16, dtype="bf16", interleaved=False, split_x=False),
        # an odd chunk in f16 with partial, interleaved rotation, into the split-x cache layout
        dict(name="norm_rope_splitx_1001", op="rope", tokens=1001, heads=16, kv_heads=2, dim=128,
             rot=64, block=16, dtype="f16", interleaved=True, split_x=True),
        # one long conversation on a windowed layer: the latency of a lone request
        dict(name="window_one_100k", op="window", seqs=1, len_lo=100000, len_hi=100000,
             window=4096, sinks=4, heads=24, kv_heads=4, dim=256, block=16, dtype="bf16"),
        # a serving batch on a windowed layer, lengths from a few tokens to 100K
        dict(name="window_serving_256", op="window", seqs=256, len_lo=16, len_hi=100000,
             window=1024, sinks=16, heads=32, kv_heads=8, dim=128, block=32, dtype="bf16"),
        # f16, a window that ends inside blocks, as many query as KV heads
        dict(name="window_f16_33", op="window", seqs=33, len_lo=1000, len_hi=30000,
             window=2000, sinks=3, heads=16, kv_heads=16, dim=128, block=16, dtype="f16"),
        # one chunk of a long prompt on a windowed layer
        dict(name="window_prefill_4096", op="window_prefill", seqs=1, ctx_lo=12288, ctx_hi=12288,
             new_lo=4096, new_hi=4096, window=2048, sinks=64, heads=24, kv_heads=4, dim=256,
             block=16, dtype="bf16"),
        # ragged chunks of five prompts, a short window
        dict(name="window_prefill_mixed", op="window_prefill", seqs=5, ctx_lo=1, ctx_hi=6000,
             new_lo=17, new_hi=1500, window=512, sinks=4, heads=32, kv_heads=8, dim=128,
             block=32, dtype="f16"),
        # a few requests on one document
        dict(name="prefix_8x8192", op="prefix", seqs=8, prefix=8192, own_lo=1, own_hi=256,
             heads=24, kv_heads=4, dim=256, block=16, dtype="bf16"),
        # a full serving batch behind one long shared prompt
        dict(name="prefix_256x32000", op="prefix", seqs=256, prefix=32000, own_lo=1, own_hi=500,
             heads=32, kv_heads=8, dim=128, block=32, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "window", "window_prefill", "prefix"])
    shape = rng.choice([(24, 4, 256, 16), (24, 4, 256, 32), (32, 8, 128, 32), (16, 16, 128, 16),
                        (16, 2, 128, 64), (6, 1, 256, 16), (40, 8, 128, 16)])
    heads, kv_heads, dim, block = shape
    dtype = rng.choice(["bf16", "f16"])
    if op == "plan":
        lo = _log_int(rng, 1, 50)
        return dict(op=op, seqs=_log_int(rng, 1, 1000), ctx_lo=1, ctx_hi=_log_int(rng, 100, 20000),
                    new_lo=1, new_hi=lo + _log_int(rng, 1, 450),
                    block=rng.choice([8, 16, 32, 64]))
    if op == "rope":
        split_x = rng.random() < 0.25
        return dict(op=op, tokens=_log_int(rng, 1, 8000), heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), block=block, dtype=dtype,
                    interleaved=rng.random() < 0.5, split_x=split_x)
    if op == "window":
        return dict(op=op, seqs=_log_int(rng, 1, 200), len_lo=1, len_hi=_log_int(rng, 1000, 100000),
                    window=_log_int(rng, 64, 1100), sinks=rng.choice([0, 1, 4, 17, 64]),
                    heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype)
    if op == "window_prefill":
        return dict(op=op, seqs=_log_int(rng, 1, 5), ctx_lo=1, ctx_hi=_log_int(rng, 100, 6000),
                    new_lo=1, new_hi=_log_int(rng, 50, 1500), window=_log_int(rng, 64, 2000),
                    sinks=rng.choice([0, 1, 4, 17, 64]), heads=heads, kv_heads=kv_heads, dim=dim,
                    block=block, dtype=dtype)
    return dict(op=op, seqs=_log_int(rng, 1, 200), prefix=_log_int(rng, 100, 20000), own_lo=1,
                own_hi=_log_int(rng, 2, 400), heads=heads, kv_heads=kv_heads, dim=dim,
                block=block, dtype=dtype)


def _lens(case, lo, hi, salt):
    """Lengths of a case's requests, spread over the logarithm of lo..hi: part of the case,
    not of the seed, so that ``work`` can count them."""
    n = case["seqs"]
    if lo >= hi:
        return np.full(n, lo, dtype=np.int64)
    r = np.random.RandomState([n, lo, hi, salt])
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


def _tables(counts, first, width, pool, seed):
    """Rows of block ids: row r holds counts[r] ids from column first[r], -1 elsewhere."""
    ids = np.random.RandomState(seed % (1 << 31)).permutation(pool)[: int(counts.sum())]
    t = np.full((len(counts), width), -1, dtype=np.int32)
    at = 0
    for r, (n, f) in enumerate(zip(counts, first)):
        t[r, f:f + n] = ids[at:at + n]
        at += n
    return t


def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _prepare_plan(c, seed):
    ctx, new = _lens(c, c["ctx_lo"], c["ctx_hi"], 1), _lens(c, c["new_lo"], c["new_hi"], 2)
    bs = c["block"]
    have, need = _cover(ctx, bs), _cover(ctx + new, bs)
    width = int(need.max()) + 3
    pool = int(need.sum()) + 100
    r = np.random.RandomState(seed % (1 << 31))
    ids = r.permutation(pool).astype(np.int32)
    tables = np.full((c["seqs"], width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(have):
        tables[b, :n] = ids[at:at + n]
        at += n
    free = ids[at:]
    total = int(new.sum()) + 64  # rows of a padded batch behind the last request
    z = dict(dtype=torch.int32, device="cuda")
    return dict(op="plan", block=bs, pool=pool, ctx=_i32(ctx), new=_i32(new), free=_i32(free),
                count=_i32([len(free)]), tables=_i32(tables),
                query_start=torch.zeros(c["seqs"] + 1, **z), seq_lens=torch.zeros(c["seqs"], **z),
                positions=torch.zeros(total, **z),
                slots=torch.zeros(total, dtype=torch.int64, device="cuda"),
                left=torch.zeros(1, **z))


def _prepare_rope(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, hq, hkv, d, bs = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    qkv = _normal((T, hq + 2 * hkv, d), dt, g)  # one projection's output; q, k, v are its slices
    blocks = _cover(T, bs) + 5
    x = 8
    if c["split_x"]:
        kc = _normal((blocks, hkv, d // x, bs, x), dt, g)
        vc = _normal((blocks, hkv, d, bs), dt, g)
    else:
        kc, vc = _normal((blocks, hkv, bs, d), dt, g), _normal((blocks, hkv, bs, d), dt, g)
    slots = torch.randperm(blocks * bs, generator=g, device="cuda")[:T] if T < 256 else (
        torch.randperm(blocks, generator=g, device="cuda")[:, None] * bs
        + torch.arange(bs, device="cuda")[None, :]).reshape(-1)[:T]
    far = 40000
    inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1).float().contiguous()
    pos = (torch.arange(T, device="cuda") + 17001 if T >= 256 else
           torch.randint(0, far, (T,), generator=g, device="cuda")).to(torch.int32)
    return dict(op="rope", heads=hq, kv_heads=hkv, dim=d, rot=c["rot"], block=bs,
                interleaved=c["interleaved"], split_x=c["split_x"], qkv=qkv,
                wq=1 + 0.1 * _normal((d,), torch.float32, g).to(dt),
                wk=1 + 0.1 * _normal((d,), torch.float32, g).to(dt), eps=1e-6, pos=pos,
                slots=slots.to(torch.int64).contiguous(), cos_sin=cos_sin,
                q_out=torch.empty((T, hq, d), dtype=dt, device="cuda"), kc=kc, vc=vc)


def _window_blocks(lens, window, sinks, bs):
    """First block column of the window part, the blocks from it on, and the sink blocks."""
    first = np.maximum(lens - window, 0) // bs
    return first, _cover(lens, bs) - first, np.minimum(_cover(min(sinks, 1 << 30), bs), first)


def _prepare_window(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    B, hq, hkv, d, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    lens = _lens(c, c["len_lo"], c["len_hi"], 3)
    first, n_win, n_sink = _window_blocks(lens, c["window"], c["sinks"], bs)
    pool = int(n_win.sum() + n_sink.sum()) + 3
    width = int(_cover(lens.max(), bs))
    # blocks between the sinks and the window have been given back: their entries say -1
    both = _tables(np.concatenate([n_win, n_sink]), np.concatenate([first, 0 * first]), width,
                   pool, seed)
    tables = np.maximum(both[:B], both[B:])
    return dict(op="window", window=c["window"], sinks=c["sinks"], block=bs,
                q=_normal((B, hq, d), dt, g), kc=_normal((pool, hkv, bs, d), dt, g),
                vc=_normal((pool, hkv, bs, d), dt, g), tables=_i32(tables), lens=_i32(lens),
                max_len=int(lens.max()), scale=1.0 / math.sqrt(d),
                out=torch.empty((B, hq, d), dtype=dt, device="cuda"))


def _prepare_window_prefill(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    B, hq, hkv, d, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    ctx, new = _lens(c, c["ctx_lo"], c["ctx_hi"], 4), _lens(c, c["new_lo"], c["new_hi"], 5)
    counts = _cover(ctx, bs)
    pool = int(counts.sum()) + 3
    tables = _tables(counts, 0 * counts, int(counts.max()), pool, seed)
    T = int(new.sum())
    start = np.concatenate([[0], np.cumsum(new)])
    return dict(op="window_prefill", window=c["window"], sinks=c["sinks"], block=bs,
                q=_normal((T, hq, d), dt, g), k=_normal((T, hkv, d), dt, g),
                v=_normal((T, hkv, d), dt, g), kc=_normal((pool, hkv, bs, d), dt, g),
                vc=_normal((pool, hkv, bs, d), dt, g), tables=_i32(tables), start=_i32(start),
                ctx=_i32(ctx), max_ctx=int(ctx.max()), max_new=int(new.max()),
                scale=1.0 / math.sqrt(d), out=torch.empty((T, hq, d), dtype=dt, device="cuda"))


def _prepare_prefix(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    B, hq, hkv, d, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    lens = _lens(c, c["own_lo"], c["own_hi"], 6)
    counts = np.concatenate([_cover(lens, bs), [_cover(c["prefix"], bs)]])
    pool = int(counts.sum()) + 3
    tables = _tables(counts, 0 * counts, int(counts.max()), pool, seed)
    return dict(op="prefix", block=bs, q=_normal((B, hq, d), dt, g),
                kc=_normal((pool, hkv, bs, d), dt, g), vc=_normal((pool, hkv, bs, d), dt, g),
                prefix_blocks=_i32(tables[B, :counts[B]]), prefix_len=_i32([c["prefix"]]),
                max_prefix=c["prefix"], tables=_i32(tables[:B, :int(counts[:B].max())]),
                lens=_i32(lens), max_len=int(lens.max()), scale=1.0 / math.sqrt(d),
                out=torch.empty((B, hq, d), dtype=dt, device="cuda"))


_PREPARE = dict(plan=_prepare_plan, rope=_prepare_rope, window=_prepare_window,
                window_prefill=_prepare_window_prefill, prefix=_prepare_prefix)


# ----------------------------------------------------------------------- run

def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _outputs(s):
    """The step plan's outputs, all buffers of the caller's."""
    return dict(tables=s["tables"], query_start=s["query_start"], seq_lens=s["seq_lens"],
                positions=s["positions"], slots=s["slots"], left=s["left"])


def _plain_plan(s):
    bs, ctx, new = s["block"], s["ctx"].long(), s["new"].long()
    have, need = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    off = torch.cumsum(need - have, 0) - (need - have)
    ends = torch.cumsum(new, 0)
    count, width = s["count"].long(), s["tables"].shape[1]
    col = torch.arange(width, device=ctx.device)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    pick = (count - 1 - (off[:, None] + col - have[:, None])).clamp(0, s["free"].numel() - 1)
    s["tables"].copy_(torch.where(fresh, s["free"][pick], s["tables"]))
    s["query_start"][:1] = 0
    s["query_start"][1:] = ends
    s["seq_lens"].copy_(ctx + new)
    t = torch.arange(s["slots"].numel(), device=ctx.device)
    b = torch.searchsorted(ends, t, right=True).clamp(max=ctx.numel() - 1)
    pos = ctx[b] + t - (ends - new)[b]
    live = t < ends[-1]
    pos = torch.where(live, pos, 0)
    s["positions"].copy_(pos)
    block = s["tables"][b, (pos // bs).clamp(max=width - 1)].long()
    s["slots"].copy_(torch.where(live, block * bs + pos % bs, -1))
    s["left"].copy_(count - (need - have).sum())
    return _outputs(s)


def _own_plan(s):
    import paged_attention_decode_v2_gb300 as pa
    pa.plan_step(s["ctx"], s["new"], s["free"], s["count"], s["tables"], s["query_start"],
                 s["seq_lens"], s["positions"], s["slots"], s["left"], block_size=s["block"],
                 num_blocks=s["pool"])
    return _outputs(s)


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


def _plain_rope(s):
    q, k, v = _qkv(s)
    row = s["cos_sin"][s["pos"].long()]
    cos, sin = row[:, None, :s["rot"] // 2], row[:, None, s["rot"] // 2:]
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


def _own_rope(s):
    import paged_attention_decode_v2_gb300 as pa
    q, k, v = _qkv(s)
    pa.qk_norm_rope(q, k, v, s["pos"], s["slots"], s["cos_sin"], s["q_out"], s["kc"], s["vc"],
                    q_weight=s["wq"], k_weight=s["wk"], eps=s["eps"],
                    interleaved=s["interleaved"], split_x=s["split_x"])
    return dict(q=s["q_out"], kc=s["kc"], vc=s["vc"])


def _attend(q, k, v, seen, scale):
    """Softmax attention of q [B, Hkv, G, D] over k, v [B, N, Hkv, D], keys where ``seen``."""
    logit = torch.einsum("bhgd,bnhd->bhgn", q, k) * scale
    logit = logit.masked_fill(~seen[:, None, None, :], -math.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True))
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    return torch.einsum("bhgn,bnhd->bhgd", p, v) / p.sum(-1, keepdim=True)


def _plain_window(s):
    q, lens, bs = s["q"], s["lens"].long()[:, None], s["block"]
    hkv = s["kc"].shape[1]
    n = min(s["window"] + s["sinks"], s["max_len"])
    j = torch.arange(n, device=q.device)[None, :]
    lo = (lens - s["window"]).clamp(min=0)  # the window's first token
    sinks = torch.minimum(lo, torch.full_like(lo, s["sinks"]))  # sinks that lie before it
    t = torch.where(j < sinks, j, lo + j - sinks)
    seen = t < lens
    t = torch.where(seen, t, lens - 1)
    blk = torch.gather(s["tables"].long(), 1, t // bs)
    k, v = s["kc"][blk, :, t % bs].float(), s["vc"][blk, :, t % bs].float()
    o = _attend(q.float().view(q.shape[0], hkv, -1, q.shape[2]), k, v, seen, s["scale"])
    s["out"].copy_(o.reshape(q.shape).to(q.dtype))
    return s["out"]


def _own_window(s):
    import paged_attention_decode_v2_gb300 as pa
    if "ws" not in s:
        s["ws"] = pa.alloc_window_workspace(s["q"], s["kc"], s["tables"], window=s["window"],
                                            num_sinks=s["sinks"], max_seq_len=s["max_len"])
    return pa.decode_window(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["out"], s["ws"],
                            window=s["window"], num_sinks=s["sinks"], max_seq_len=s["max_len"],
                            scale=s["scale"])


def _plain_window_prefill(s):
    q, bs, ctx = s["q"], s["block"], s["ctx"].long()[:, None]
    start = s["start"].long()
    new = (start[1:] - start[:-1])[:, None]
    hkv, d = s["k"].shape[1:]
    dev = q.device
    # keys of every sequence side by side: its context, then its chunk
    j = torch.arange(s["max_ctx"] + s["max_new"], device=dev)[None, :]
    cached, real = j < ctx, j < ctx + new
    col = torch.where(cached, j // bs, 0)
    blk = torch.gather(s["tables"].long(), 1, col)
    row = torch.where(real & ~cached, start[:-1, None] + j - ctx, 0)
    pick = (cached & real)[:, :, None, None]
    k = torch.where(pick, s["kc"][blk, :, j % bs], s["k"][row]).float()
    v = torch.where(pick, s["vc"][blk, :, j % bs], s["v"][row]).float()
    i = torch.arange(s["max_new"], device=dev)[None, :]
    live = i < new
    qrow = torch.where(live, start[:-1, None] + i, 0)
    qb = q[qrow].float().view(qrow.shape[0], -1, hkv, q.shape[1] // hkv, d)
    p = (ctx + i)[:, :, None]  # positions
    t = j[:, None, :]
    seen = (t <= p) & ((t < s["sinks"]) | (t > p - s["window"])) & real[:, None, :]
    logit = torch.einsum("bihgd,bnhd->bhgin", qb, k) * s["scale"]
    logit = logit.masked_fill_(~seen[:, None, None], -math.inf)
    w = torch.exp_(logit.sub_(logit.amax(-1, keepdim=True)))
    v = v.masked_fill(~real[:, :, None, None], 0.0)
    o = torch.einsum("bhgin,bnhd->bihgd", w, v) / w.sum(-1).permute(0, 3, 1, 2)[..., None]
    o = o.reshape(o.shape[0], o.shape[1], q.shape[1], d)
    t = torch.arange(q.shape[0], device=dev)
    b = torch.searchsorted(start[1:], t, right=True)
    s["out"].copy_(o[b, t - start[b]].to(q.dtype))
    return s["out"]


def _own_window_prefill(s):
    import paged_attention_decode_v2_gb300 as pa
    pa.prefill_window(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["tables"], s["start"], s["ctx"],
                      s["out"], window=s["window"], num_sinks=s["sinks"],
                      max_query_len=s["max_new"], max_ctx_len=s["max_ctx"], scale=s["scale"])
    return s["out"]


def _plain_prefix(s):
    q, bs, n = s["q"], s["block"], s["max_prefix"]
    hkv, d = s["kc"].shape[1], q.shape[2]
    qf = q.float().view(q.shape[0], hkv, -1, d)
    dev = q.device
    t = torch.arange(n, device=dev)
    blk = s["prefix_blocks"].long()[t // bs]
    kp, vp = s["kc"][blk, :, t % bs].float(), s["vc"][blk, :, t % bs].float()
    a = torch.einsum("bhgd,nhd->bhgn", qf, kp) * s["scale"]
    a = a.masked_fill(t >= s["prefix_len"], -math.inf)
    j = torch.arange(s["max_len"], device=dev)[None, :].expand(q.shape[0], -1)
    seen = j < s["lens"][:, None]
    blk = torch.gather(s["tables"].long(), 1, j // bs).clamp(min=0)
    ko, vo = s["kc"][blk, :, j % bs].float(), s["vc"][blk, :, j % bs].float()
    b = torch.einsum("bhgd,bnhd->bhgn", qf, ko) * s["scale"]
    b = b.masked_fill(~seen[:, None, None, :], -math.inf)
    top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a, b = torch.exp(a - top), torch.exp(b - top)
    vo = vo.masked_fill(~seen[:, :, None, None], 0.0)
    o = torch.einsum("bhgn,nhd->bhgd", a, vp) + torch.einsum("bhgn,bnhd->bhgd", b, vo)
    o = o / (a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True))
    s["out"].copy_(o.reshape(q.shape).to(q.dtype))
    return s["out"]


def _own_prefix(s):
    import paged_attention_decode_v2_gb300 as pa
    if "ws" not in s:
        s["ws"] = pa.alloc_prefix_workspace(s["q"], s["kc"], s["tables"],
                                            max_seq_len=s["max_len"],
                                            max_prefix_len=s["max_prefix"])
    return pa.decode_prefix(s["q"], s["kc"], s["vc"], s["prefix_blocks"], s["prefix_len"],
                            s["tables"], s["lens"], s["out"], s["ws"], max_seq_len=s["max_len"],
                            max_prefix_len=s["max_prefix"], scale=s["scale"])


_PLAIN = dict(plan=_plain_plan, rope=_plain_rope, window=_plain_window,
              window_prefill=_plain_window_prefill, prefix=_plain_prefix)
_OWN = dict(plan=_own_plan, rope=_own_rope, window=_own_window,
            window_prefill=_own_window_prefill, prefix=_own_prefix)


# ---------------------------------------------------------------------- work

def _elem(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    c, op = case, case["op"]
    if op == "plan":
        ctx, new = _lens(c, c["ctx_lo"], c["ctx_hi"], 1), _lens(c, c["new_lo"], c["new_hi"], 2)
        bs = c["block"]
        fresh = int((_cover(ctx + new, bs) - _cover(ctx, bs)).sum())
        tokens = int(new.sum()) + 64
        # both lengths, the last filled block's id, the free ids taken; the lengths and starts,
        # the new table entries, a position and a slot for each row
        return {"bytes": 12 * c["seqs"] + 4 * fresh + 8 * c["seqs"] + 4 * fresh + 12 * tokens,
                "flops": 0}
    if op == "rope":
        rows = c["tokens"] * (c["heads"] + 2 * c["kv_heads"])
        return {"bytes": 2 * rows * c["dim"] * _elem(c) + c["tokens"] * (4 * c["rot"] + 12)
                + 2 * c["dim"] * _elem(c), "flops": 8 * rows * c["dim"]}
    e, hq, hkv, d = _elem(c), c["heads"], c["kv_heads"], c["dim"]
    if op == "window":
        lens = _lens(c, c["len_lo"], c["len_hi"], 3)
        lo = np.maximum(lens - c["window"], 0)
        keys = int((lens - lo + np.minimum(lo, c["sinks"])).sum())
        return {"bytes": keys * hkv * d * 2 * e + 2 * c["seqs"] * hq * d * e,
                "flops": 4 * d * hq * keys}
    if op == "window_prefill":
        ctx, new = _lens(c, c["ctx_lo"], c["ctx_hi"], 4), _lens(c, c["new_lo"], c["new_hi"], 5)
        triples, keys = 0, 0
        for C, n in zip(ctx, new):
            p = C + np.arange(n)
            lo = np.maximum(p - c["window"] + 1, 0)
            triples += int((p + 1 - lo + np.minimum(lo, c["sinks"])).sum())
            keys += int(min(C, C - max(C - c["window"] + 1, 0) + min(max(C - c["window"] + 1, 0),
                                                                     c["sinks"])))
        T = int(new.sum())
        return {"bytes": (keys + T) * hkv * d * 2 * e + 2 * T * hq * d * e,
                "flops": 4 * d * hq * triples}
    lens = _lens(c, c["own_lo"], c["own_hi"], 6)
    return {"bytes": (int(lens.sum()) + c["prefix"]) * hkv * d * 2 * e + 2 * c["seqs"] * hq * d * e,
            "flops": 4 * d * hq * (int(lens.sum()) + c["seqs"] * c["prefix"])}


# --------------------------------------------------------------------- exact

def _softmax64(q, k, v, scale, mask=None):
    """Rows of q [H, n, D] over k, v [m, D] in 64 bits."""
    s = torch.matmul(q, k.T) * scale
    if mask is not None:
        s = torch.where(mask, s, -math.inf)
    return torch.matmul(torch.softmax(s, dim=-1), v)


def _rows64(cache, table, tokens, bs):
    at = torch.as_tensor(tokens, device=cache.device, dtype=torch.long)
    return cache[table[at // bs].long(), :, at % bs].double()


def exact(case, seed):
    """The outputs of ``run`` in 64 bits, one sequence and KV head at a time."""
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _EXACT[case["op"]](s).reshape(s["out"].shape)


def _exact_rope(s):
    hq, hkv, rot = s["heads"], s["kv_heads"], s["rot"]
    x = s["qkv"].double()
    w = torch.cat([s["wq"].double().expand(hq, -1), s["wk"].double().expand(hkv, -1)])
    y = x[:, :hq + hkv]
    y = y / torch.sqrt(torch.mean(y ** 2, dim=-1, keepdim=True) + s["eps"]) * w
    turn = torch.complex(s["cos_sin"][:, :rot // 2].double(),
                         s["cos_sin"][:, rot // 2:].double())[s["pos"].long()][:, None]
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


def _exact_window(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    hkv = s["kc"].shape[1]
    for b, L in enumerate(s["lens"].tolist()):
        seen = [t for t in range(min(s["sinks"], L))] + list(
            range(max(L - s["window"], min(s["sinks"], L)), L))
        k = _rows64(s["kc"], s["tables"][b], seen, s["block"])
        v = _rows64(s["vc"], s["tables"][b], seen, s["block"])
        q = s["q"][b].double().view(hkv, -1, 1, s["q"].shape[2])
        out[b] = torch.stack([_softmax64(q[h], k[:, h], v[:, h], s["scale"])
                              for h in range(hkv)]).view(out[b].shape)
    return out


def _exact_window_prefill(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    hkv = s["kc"].shape[1]
    G = s["q"].shape[1] // hkv
    start = s["start"].tolist()
    for b, C in enumerate(s["ctx"].tolist()):
        a, z = start[b], start[b + 1]
        k = torch.cat([_rows64(s["kc"], s["tables"][b], range(C), s["block"]),
                       s["k"][a:z].double()])
        v = torch.cat([_rows64(s["vc"], s["tables"][b], range(C), s["block"]),
                       s["v"][a:z].double()])
        t = torch.arange(C + z - a, device="cuda")
        age = (C + torch.arange(z - a, device="cuda"))[:, None] - t[None, :]
        mask = (age >= 0) & ((age < s["window"]) | (t < s["sinks"])[None, :])
        for h in range(hkv * G):
            out[a:z, h] = _softmax64(s["q"][a:z, h].double()[None], k[:, h // G], v[:, h // G],
                                     s["scale"], mask)[0]
    return out


def _exact_prefix(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    hkv = s["kc"].shape[1]
    n = int(s["prefix_len"])
    kp = _rows64(s["kc"], s["prefix_blocks"], range(n), s["block"])
    vp = _rows64(s["vc"], s["prefix_blocks"], range(n), s["block"])
    for b, L in enumerate(s["lens"].tolist()):
        k = torch.cat([kp, _rows64(s["kc"], s["tables"][b], range(L), s["block"])])
        v = torch.cat([vp, _rows64(s["vc"], s["tables"][b], range(L), s["block"])])
        q = s["q"][b].double().view(hkv, -1, s["q"].shape[2])
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * s["scale"], dim=-1)
        out[b] = torch.einsum("hgn,nhd->hgd", w, v).reshape(out[b].shape)
    return out


_EXACT = dict(window=_exact_window, window_prefill=_exact_window_prefill, prefix=_exact_prefix)
