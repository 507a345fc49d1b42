"""The 4-bit cache on the GPU against plain float64 references: store, load, decode,
and a serving step on it."""
import math

import numpy as np
import pytest
import torch

import kv4_reference as kr
import paged_attention_decode_v2_gb300 as pa
import step_reference as sr
from gpu_helpers import GUARD_B, GUARD_F, _guarded, _guards_intact

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


# ---------------------------------------------------------------- store

def check_codes(x, codes, scale, low, group, dtype):
    """The written codes and pairs of head rows x (float64): the minimum exactly, the scale within
    half a step of the type (and float32's quotient), each code the nearest whole number of
    (x - m) / s -- halves and float32's quotient, 2^-20 of at most 15, aside."""
    g = x.unflatten(-1, (-1, group))
    assert torch.equal(low, g.amin(-1))
    want = (g.amax(-1) - low) / 15
    tiny = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}[dtype]  # half the least subnormal
    assert ((scale - want).abs() <= (sr.HALF_STEP[dtype] + 2.0 ** -23) * want + tiny).all()
    c = codes.unflatten(-1, (-1, group))
    zero = (scale == 0)[..., None].expand_as(c)
    assert (c[zero] == 0).all()
    ratio = (g - low[..., None]) / scale[..., None]
    off = (c - ratio.clamp(max=15)).abs()
    assert (off[~zero] <= 0.5 + 2.0 ** -16).all(), float(off[~zero].max())


def run_store(x, hkv, d, group, bs, dtype, slots, blocks, dense=True, seed=0):
    """x [T, 2 Hkv, D] on the CPU; returns (pool before, pool after, k_out, v_out, status)."""
    pool = kr.Pool(blocks, hkv, bs, d, group, dtype, seed)
    pool.ks.fill_(3.0), pool.vs.fill_(3.0)
    g = pool.cuda()
    xg = x.cuda()
    T = x.shape[0]
    outs = [_guarded(T * hkv * d, dtype, GUARD_F, "cuda") for _ in range(2)] if dense else None
    ko, vo = (o[1].view(T, hkv, d).fill_(7) for o in outs) if dense else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.store_kv4(xg[:, :hkv], xg[:, hkv:], slots.cuda(), *g, k_out=ko, v_out=vo, status=status)
    torch.cuda.synchronize()
    if dense:
        assert all(_guards_intact(o[0], T * hkv * d, GUARD_F) for o in outs)
    after = [t.cpu() for t in g]
    return (pool.k, pool.v, pool.ks, pool.vs), after, ko, vo, int(status)


def check_store(x, hkv, d, group, bs, dtype, slots, blocks, dense=True, exact=True):
    before, after, ko, vo, status = run_store(x, hkv, d, group, bs, dtype, slots, blocks, dense)
    assert status == 0
    live = slots >= 0
    at = slots[live]
    for i, (rows, out) in enumerate(((x[live, :hkv], ko), (x[live, hkv:], vo))):
        codes, pairs = after[i], after[i + 2]
        c = kr.unpack(codes[at // bs, :, at % bs]).double()
        p = pairs[at // bs, :, at % bs].double()
        check_codes(rows.double(), c, p[..., 0], p[..., 1], group, dtype)
        if exact:
            # of 16-bit rows the differences are exact and no quotient is near a border that it
            # does not meet, so float32 and float64 agree
            want, s, m = kr.quantise(rows, group)
            assert torch.equal(c, want) and torch.equal(p[..., 0], s) and torch.equal(p[..., 1], m)
        v = kr.values(codes[at // bs, :, at % bs], pairs[at // bs, :, at % bs])
        if dense:
            got = out.cpu()[live].double()
            # one float32 operation, one rounding
            slack = (sr.HALF_STEP[dtype] + 2.0 ** -23) * v.abs() + 2.0 ** -24 * v.abs().max()
            assert ((got - v).abs() <= slack).all()
            assert (out.cpu()[~live] == 7).all()
        # nothing else has changed
        codes[at // bs, :, at % bs] = before[i][at // bs, :, at % bs]
        pairs[at // bs, :, at % bs] = before[i + 2][at // bs, :, at % bs]
        assert torch.equal(codes, before[i]) and torch.equal(pairs, before[i + 2])


@pytest.mark.parametrize("T,hkv,d,group,bs", [
    (1, 1, 64, 32, 1), (1, 8, 128, 128, 16), (3, 2, 64, 64, 7), (33, 8, 128, 64, 32),
    (257, 4, 256, 64, 16), (100, 5, 128, 32, 20), (64, 3, 256, 128, 16), (70, 16, 256, 32, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_store(T, hkv, d, group, bs, dtype):
    g = torch.Generator().manual_seed(T * d + group)
    x = (torch.randn(T, 2 * hkv, d, generator=g) * 2 + 0.5).to(dtype)
    blocks = -(-T // bs) + 2
    slots = torch.randperm(blocks * bs, generator=g)[:T]
    if T > 9:
        slots[[2, T - 1]] = -1
    check_store(x, hkv, d, group, bs, dtype, slots, blocks, exact=dtype != F32)
    check_store(x, hkv, d, group, bs, dtype, slots, blocks, dense=False, exact=dtype != F32)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_store_ranges(dtype):
    """Groups without a range, with a tiny one, of one sign, at the ends of the type."""
    big = torch.finfo(dtype).max / 2.5
    rows = torch.zeros(8, 2, 128)
    rows[1] = 3.25
    rows[2] = 1 + torch.linspace(0, 2 ** -7, 128)
    rows[3] = -torch.linspace(1, 2, 128)
    rows[4] = torch.linspace(-big, big, 128)
    rows[5] = torch.linspace(0, 1, 128) * torch.finfo(dtype).tiny
    rows[6, :, 5] = 1e-3
    rows[7] = torch.linspace(-1, 1, 128)
    rows[7, :, 64] = 30000.0
    x = rows.to(dtype)
    # below the least normal scale the quotient is not near its float64 value: the properties only
    check_store(x, 1, 128, 64, 16, dtype, torch.arange(8), 2, exact=False)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_store_of_what_is_not_finite(dtype):
    g = torch.Generator().manual_seed(8)
    x = torch.randn(6, 4, 128, generator=g).to(dtype)
    x[1, 0, 3] = math.nan
    x[2, 1, 70] = math.inf
    x[3, 2, 127] = -math.inf
    x[4, 3, 0], x[4, 3, 1] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    before, after, ko, vo, status = run_store(x, 2, 128, 64, 16, dtype, torch.arange(6), 1)
    ref = kr.quantise(x, 64)
    bad = torch.isnan(ref[1])
    assert int(bad.sum()) == (3 if dtype == F16 else 4)    # float32 holds float16's whole range
    pairs = torch.cat([after[2][0], after[3][0]]).transpose(0, 1)[:6]
    assert torch.equal(torch.isnan(pairs[..., 0].double()), bad)
    assert torch.equal(torch.isnan(pairs[..., 1].double()), bad)
    out = torch.cat([ko, vo], 1).cpu()
    assert torch.equal(torch.isnan(out), bad.repeat_interleave(64, -1))
    if dtype != F32:
        assert torch.equal(pairs[..., 0].double()[~bad], ref[1][~bad])


def test_store_bad_slots():
    g = torch.Generator().manual_seed(9)
    x = torch.randn(5, 4, 64, generator=g).to(BF16)
    for slot in (-2, 32, 1 << 40):
        slots = torch.tensor([0, slot, 2, -1, 31])
        before, after, ko, vo, status = run_store(x, 2, 64, 64, 16, BF16, slots, 2)
        assert status == pa.PA_ERR_BAD_SLOT
        assert (ko[3] == 7).all() and not (ko[1] == 7).any()   # padding; the bad row's values
        for a, b in zip(after, before):
            changed = (a != b).flatten(3).any(-1).any(1).flatten()
            assert set(torch.nonzero(changed).flatten().tolist()) <= {0, 2, 31}


def test_store_strided_and_in_place():
    """k and v as slices of a fused projection, and k_out, v_out over contiguous k and v."""
    g = torch.Generator().manual_seed(10)
    x = torch.randn(40, 12, 128, generator=g).to(F16)
    slots = torch.arange(40)
    pools = [kr.Pool(3, 2, 16, 128, 32, F16, 1).cuda() for _ in range(2)]
    xg = x.cuda()
    ko = torch.empty(40, 2, 128, dtype=F16, device="cuda")
    vo = torch.empty_like(ko)
    pa.store_kv4(xg[:, 8:10], xg[:, 10:], slots.cuda(), *pools[0], k_out=ko, v_out=vo)
    assert torch.equal(xg.cpu(), x)
    k, v = xg[:, 8:10].contiguous(), xg[:, 10:].contiguous()
    pa.store_kv4(k, v, slots.cuda(), *pools[1], k_out=k, v_out=v)
    assert torch.equal(k, ko) and torch.equal(v, vo)
    for a, b in zip(*pools):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())
    # what the cache holds now is a fixed point: the values store as themselves to within the
    # rounding of the scale
    assert ((k.double() - x[:, 8:10].cuda().double()).abs().max() < 0.3)


def test_store_rows_without_a_grid_and_empty():
    pool = kr.Pool(1, 2, 16, 64, 32, BF16, 1).cuda()
    x = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    pa.store_kv4(x, x, torch.zeros(0, dtype=torch.int64, device="cuda"), *pool)
    x = torch.zeros(3, 2, 64, dtype=BF16, device="cuda")
    before = [t.clone() for t in pool]
    pa.store_kv4(x, x.clone(), torch.full((3,), -1, device="cuda"), *pool)
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(pool, before))


# ---------------------------------------------------------------- load

@pytest.mark.parametrize("lens,hkv,d,group,bs", [
    ((1,), 1, 64, 32, 1), ((0, 5, 16, 17, 300), 2, 128, 64, 16), ((100, 0, 33), 5, 256, 128, 20),
    (tuple(range(70)), 3, 64, 64, 8), ((2000,), 4, 256, 64, 16), ((63, 64, 65), 8, 128, 32, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_load(lens, hkv, d, group, bs, dtype):
    pages = [-(-n // bs) for n in lens]
    pool = kr.Pool(sum(pages) + 2, hkv, bs, d, group, dtype, seed=sum(lens))
    tables = torch.full((len(lens), max(1, max(pages)) + 1), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        pool.fill(tables[b], n)
    wide = sum(pages) + 3
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(wide, generator=g).tolist()
    to = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32)
    for b, n in enumerate(pages):
        to[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    n_out = wide * hkv * bs * d
    outs = [_guarded(n_out, dtype, GUARD_F, "cuda") for _ in range(2)]
    ko, vo = (o[1].view(wide, hkv, bs, d).fill_(7) for o in outs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.load_kv4(*pool.cuda(), i32(tables), i32(lens), i32(to), ko, vo, max_seq_len=max(max(lens), 1),
                status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert all(_guards_intact(o[0], n_out, GUARD_F) for o in outs)
    for got, codes, pairs in ((ko.cpu(), pool.k, pool.ks), (vo.cpu(), pool.v, pool.vs)):
        left = torch.ones(wide, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(pages[b]):
                left[to[b, j]] = False
                m = min(bs, n - j * bs)                     # places past the end: anything
                want = kr.values(codes[tables[b, j]], pairs[tables[b, j]])[:, :m]
                err = (got[to[b, j]][:, :m].double() - want).abs()
                slack = (sr.HALF_STEP[dtype] + 2.0 ** -23) * want.abs() + 2.0 ** -22
                assert (err <= slack).all()
        assert (got[left] == 7).all()


def test_load_bad_lengths_and_pages():
    pool = kr.Pool(8, 2, 16, 128, 64, BF16, seed=3)
    tables = torch.full((4, 3), -1, dtype=torch.int32)
    for b in range(4):
        pool.fill(tables[b], 32)
    to = torch.arange(12, dtype=torch.int32).view(4, 3)

    def run(lens=(32, 32, 32, 32), tables=tables, to=to, most=48):
        ko = torch.full((12, 2, 16, 128), 7.0, dtype=BF16, device="cuda")
        vo = ko.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.load_kv4(*pool.cuda(), i32(tables), i32(lens), i32(to), ko, vo, max_seq_len=most,
                    status=status)
        return ko.cpu(), vo.cpu(), int(status)

    good = run()
    assert good[2] == 0
    for bad in (-1, 49, 1 << 30):
        ko, vo, st = run(lens=(32, bad, 32, 32))
        assert st == pa.PA_ERR_BAD_SEQ_LEN
        assert (ko[3:6] == 7).all() and torch.equal(ko[:3], good[0][:3])
        assert torch.equal(vo[6:], good[1][6:])
    for bad in (-1, 8, 1 << 30):
        t = tables.clone()
        t[2, 1] = bad
        ko, vo, st = run(tables=t)
        assert st == pa.PA_ERR_BAD_BLOCK_ID
        assert torch.isnan(ko[7]).all() and torch.isnan(vo[7]).all()
        keep = torch.arange(12) != 7
        assert torch.equal(ko[keep], good[0][keep])
    for bad in (-1, 12):
        t = to.clone()
        t[2, 1] = bad
        ko, vo, st = run(to=t)
        assert st == pa.PA_ERR_BAD_BLOCK_ID
        assert (ko[7] == 7).all() and torch.equal(ko[6], good[0][6])
    # bounds of zero: lengths are still looked at
    assert run(lens=(0, 0, 0, 0), most=0)[2] == 0
    assert run(lens=(0, 1, 0, 0), most=0)[2] == pa.PA_ERR_BAD_SEQ_LEN


# ---------------------------------------------------------------- decode

def run_decode(q, pool, tables, lens, scale=None, max_len=None, out_dtype=None, portable=False,
               partition_size=1024, status=0, workspace=None):
    d = q.shape[2]
    out_dtype = out_dtype or q.dtype
    whole, flat = _guarded(q.numel(), out_dtype, GUARD_F, "cuda")
    out = flat.fill_(math.nan).view(q.shape)
    max_len = int(max(lens)) if max_len is None else max_len
    qg, (kc, vc, ks, vs), bt = q.cuda(), pool.cuda(), i32(tables)
    ws = workspace
    if ws is None:
        p = pa.Params(q.shape[0], q.shape[1], pool.hkv, d, pool.bs, kc.shape[0], bt.shape[1],
                      max_len, partition_size, 0, pa._dtype_code(q.dtype),
                      pa._dtype_code(out_dtype), 1.0, 0)
        n = pa.kv4_workspace_size(p, pool.group)
        ws_whole, ws = _guarded(n, torch.uint8, GUARD_B, "cuda")
        ws.fill_(0xFF)                                      # NaN everywhere
        pa.workspace_init(ws)
    pa.decode_kv4(qg, kc, vc, ks, vs, bt, i32(lens), out, ws, max_seq_len=max_len,
                  scale=d ** -0.5 if scale is None else scale, partition_size=partition_size, portable=portable)
    torch.cuda.synchronize()
    assert _guards_intact(whole, q.numel(), GUARD_F), "write outside out"
    if workspace is None:
        assert _guards_intact(ws_whole, ws.numel(), GUARD_B), "write outside the workspace"
    assert pa.read_device_status(ws) == status
    return out


SHAPES = [
    # hq, hkv, d, bs, group
    (24, 4, 256, 16, 64), (32, 8, 128, 32, 128), (16, 16, 128, 16, 32), (6, 1, 256, 32, 32),
    (8, 1, 128, 16, 64), (12, 4, 64, 16, 64), (5, 1, 64, 7, 32), (32, 2, 128, 64, 64),
    (20, 2, 256, 1, 128), (34, 2, 64, 20, 32), (4, 4, 256, 8, 64)]
LENS = [(1,), (16, 15, 17, 0, 64), (100, 1, 333), (700, 1200)]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("hq,hkv,d,bs,group", SHAPES)
@pytest.mark.parametrize("dtype,portable", [(BF16, False), (F16, False), (BF16, True),
                                            (F32, False)])
def test_decode(hq, hkv, d, bs, group, lens, dtype, portable):
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, hq, hkv, d, bs, group, dtype,
                                                           seed=hq + d + len(lens))
    for out_dtype in {dtype, F32}:
        got = run_decode(q, pool, tables, n, out_dtype=out_dtype, portable=portable)
        kr.assert_decode(got, ref, mag, step, out_dtype, portable or dtype == F32)


@pytest.mark.parametrize("hq,hkv,d,bs,group", [
    (8, 2, 256, 16, 32), (8, 2, 256, 32, 64), (8, 2, 256, 16, 128), (8, 2, 128, 16, 32),
    (8, 2, 128, 32, 64), (8, 2, 128, 20, 128), (8, 2, 64, 16, 32), (8, 2, 64, 48, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decode_batch(hq, hkv, d, bs, group, dtype):
    """More pairs than half the SMs (80): narrow CTAs, sequences in one part and in several, rows
    without a token among them."""
    r = np.random.RandomState(d + group)
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(1000), size=36))] + [0, 2600, 1, 2176]
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, hq, hkv, d, bs, group, dtype, 3)
    got = run_decode(q, pool, tables, n, out_dtype=F32)
    kr.assert_decode(got, ref, mag, step, F32, False)


@pytest.mark.parametrize("hq,d,bs,group", [
    (4, 256, 16, 32), (10, 256, 32, 64), (6, 256, 16, 128), (8, 128, 16, 32), (4, 128, 32, 64),
    (12, 128, 20, 128), (6, 64, 16, 32), (16, 64, 48, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("seqs", [1, 2, 24])
def test_decode_few_pairs(hq, d, bs, group, dtype, seqs):
    """Two KV heads of a sequence or two past 6000 tokens (wide CTAs, in parts), and of 24 of up to
    131072 / head_dim (wide CTAs, one part each)."""
    lens = [6007, 450][:seqs] if seqs < 24 else [131072 // d, 321, 0, 1] + [
        64 * i + i % 3 - 1 for i in range(1, 7)] * 3 + [500, 130]
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, hq, 2, d, bs, group, dtype,
                                                           d + group + seqs)
    got = run_decode(q, pool, tables, n, out_dtype=F32)
    kr.assert_decode(got, ref, mag, step, F32, False)


@pytest.mark.parametrize("d,group,low,high,seqs", [
    (64, 32, 2050, 2400, 200), (128, 128, 1025, 1280, 160), (256, 64, 513, 640, 160),
    (256, 128, 900, 1000, 40), (64, 64, 2100, 2100, 160)])
def test_decode_even_batch(d, group, low, high, seqs):
    """Many sequences of about one length: even parts of the longest, or all of it; among them one
    without a token and one that is short."""
    r = np.random.RandomState(d + seqs)
    lens = [int(x) for x in r.randint(low, high + 1, size=seqs - 2)] + [0, 77]
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, 6, 2, d, 16, group, BF16, 9)
    got = run_decode(q, pool, tables, n, out_dtype=F32)
    kr.assert_decode(got, ref, mag, step, F32, False)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("portable", [False, True])
def test_decode_long(dtype, portable):
    """One sequence over the whole GPU, and parts that end inside tiles and pages."""
    q, pool, tables, n, ref, mag, step = kr.decode_problem((20011,), 8, 2, 128, 16, 64, dtype, 5)
    got = run_decode(q, pool, tables, n, portable=portable, max_len=20016)
    kr.assert_decode(got, ref, mag, step, dtype, portable)


def test_decode_many_sequences():
    """More sequences than the list's spans of 32 and more items than CTAs, so that they come from
    the queue; most short, some without a token, some in several parts; the same workspace again
    and again, in a graph, and one that has not been initialised (its items go by number)."""
    r = np.random.RandomState(1)
    lens = [int(x) for x in np.exp(r.uniform(0, np.log(600), size=301))]
    lens[7] = lens[64] = lens[300] = 0
    lens[33], lens[200] = 2900, 5000
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, 8, 4, 64, 16, 32, BF16, 6)
    first = None
    for size in (64, 100, 1024):
        got = run_decode(q, pool, tables, n, partition_size=size)
        kr.assert_decode(got, ref, mag, step, BF16, False)
        first = got if first is None else first
    qg, caches, bt, ng = q.cuda(), pool.cuda(), i32(tables), i32(n)
    kc, vc, ks, vs = caches
    for init in (True, False):
        ws = pa.alloc_kv4_workspace(qg, kc, ks, bt, max_seq_len=5000, partition_size=64)
        if not init:
            ws.fill_(0x77)
        out = torch.empty_like(qg)
        call = lambda: pa.decode_kv4(qg, kc, vc, ks, vs, bt, ng, out, ws, max_seq_len=5000,
                                     scale=64 ** -0.5, partition_size=64)
        for _ in range(3):
            out.fill_(math.nan)
            call()
            assert torch.equal(out, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
            call()
        for _ in range(2):
            out.fill_(math.nan)
            graph.replay()
            assert torch.equal(out, first)
        if init:
            assert pa.read_device_status(ws) == pa.PA_OK
    # bad lengths and pages among them
    m, t = n.clone(), tables.clone()
    m[40], m[290] = -3, 5001
    t[33, 100], t[250, 0] = -1, pool.k.shape[0]
    bad = [33, 40, 290] + ([250] if lens[250] else [])
    whole = run_decode(q, pool, tables, m, max_len=5000, status=pa.PA_ERR_BAD_SEQ_LEN)
    assert torch.isnan(whole[[40, 290]]).all()
    whole = run_decode(q, pool, t, n, status=pa.PA_ERR_BAD_BLOCK_ID)
    assert torch.isnan(whole[[33] + ([250] if lens[250] else [])]).all()
    keep = [b for b in range(301) if b not in bad]
    kr.assert_decode(whole[keep], ref[keep], mag[keep], step[keep], BF16, False)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("spread,offset", [(12.0, 0.0), (1.0, 20.0), (1e-3, 0.0)])
def test_decode_peaked_offset_and_small_keys(dtype, portable, spread, offset):
    """Logits of size 12 to 60; groups far from zero; steps of 10^-4."""
    q, pool, tables, n, ref, mag, step = kr.decode_problem(
        (513, 90), 6, 2, 128, 16, 64, dtype, 7, spread, offset)
    got = run_decode(q, pool, tables, n, portable=portable, out_dtype=F32)
    kr.assert_decode(got, ref, mag, step, F32, portable, logits=max(spread, offset, 1.0) * 4)


def grow(lens, factor):
    """A problem whose later tokens have much larger (or smaller) steps."""
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, 4, 2, 128, 16, 64, BF16, 11)
    for b, L in enumerate(lens):
        for t in range(L):
            blk, at = int(tables[b, t // 16]), t % 16
            f = 2.0 ** (factor * (t // 37))
            pool.vs[blk, :, at] = (pool.vs[blk, :, at].float() * f).to(BF16)
        k, v, s = pool.rows(tables[b], L)
        for h in range(4):
            w = torch.softmax((k[:, h // 2] @ q[b, h].double()) * 128 ** -0.5, 0)
            ref[b, h], mag[b, h] = w @ v[:, h // 2], w @ v[:, h // 2].abs()
            step[b, h] = w @ s[:, h // 2]
    return q, pool, tables, n, ref, mag, step


@pytest.mark.parametrize("factor", [2, -2, 4])
@pytest.mark.parametrize("portable", [False, True])
def test_decode_steps_that_grow_and_shrink(factor, portable):
    q, pool, tables, n, ref, mag, step = grow((400, 60), factor)
    got = run_decode(q, pool, tables, n, portable=portable, out_dtype=F32)
    kr.assert_decode(got, ref, mag, step, F32, portable)


def test_decode_queries_of_any_size():
    """Queries up to 2^100 and down to 2^-60 (bf16): logits as with queries of order 1."""
    for e in (100, 40, 14, -20, -60):
        q, pool, tables, n, ref, mag, step = kr.decode_problem((200,), 4, 2, 128, 16, 64, BF16, 12)
        got = run_decode((q.float() * 2.0 ** e).to(BF16), pool, tables, n, out_dtype=F32,
                         scale=128 ** -0.5 * 2.0 ** -e)
        kr.assert_decode(got, ref, mag, step, F32, False)


def test_decode_queries_past_the_operands():
    """From 2^116 on a head's row is NaN; the other rows are as they were."""
    q, pool, tables, n, *_ = kr.decode_problem((200, 90), 8, 2, 128, 16, 64, BF16, 12)
    want = run_decode(q, pool, tables, n, out_dtype=F32)
    q[0, 3] *= 2.0 ** 120
    got = run_decode(q, pool, tables, n, out_dtype=F32)
    assert bool(got[0, 3].isnan().all())
    want[0, 3] = got[0, 3] = 0.
    assert torch.equal(got, want)


@pytest.mark.parametrize("portable", [False, True])
def test_decode_scales_of_any_sign(portable):
    q, pool, tables, n, ref, mag, step = kr.decode_problem((150, 9), 4, 2, 128, 16, 64, BF16, 12)
    scale = 128 ** -0.5
    got = run_decode(-q, pool, tables, n, scale=-scale, out_dtype=F32, portable=portable)
    kr.assert_decode(got, ref, mag, step, F32, portable)
    got = run_decode(q, pool, tables, n, scale=1e-40, out_dtype=F32, portable=portable)
    zero = run_decode(0 * q, pool, tables, n, out_dtype=F32, portable=portable)
    for b in range(2):                                      # equal weights: the mean
        v = pool.rows(tables[b], int(n[b]))[1].mean(0).repeat_interleave(2, 0)
        s = pool.rows(tables[b], int(n[b]))[2].mean(0).repeat_interleave(2, 0)
        for x in (got, zero):
            kr.assert_decode(x[b], v, v.abs() + 2, s, F32, portable)


@pytest.mark.parametrize("portable", [False, True])
def test_decode_what_is_not_finite(portable):
    """A NaN scale of a visible token makes the heads that see it NaN (keys) or their group
    (values); NaN queries their row; other sequences are as they were."""
    q, pool, tables, n, ref, mag, step = kr.decode_problem((80, 90, 100, 64), 4, 2, 128, 16, 64,
                                                           BF16, 13)
    blk = int(tables[0, 3])
    pool.ks[blk, 1, 2, 0] = math.nan
    pool.vs[int(tables[1, 0]), 0, 5, 1, 0] = math.nan
    q[2, 3, 7] = math.nan
    out = run_decode(q, pool, tables, n, portable=portable).cpu()
    nan = torch.isnan(out)
    assert nan[0, 2:].all() and not nan[0, :2].any()
    assert nan[1, :2, 64:].all() and not nan[1, 2:].any()
    assert nan[2, 3].all() and not nan[2, :3].any()
    assert not nan[3].any()
    kr.assert_decode(out[3], ref[3], mag[3], step[3], BF16, portable)
    kr.assert_decode(out[0, :2], ref[0, :2], mag[0, :2], step[0, :2], BF16, portable)


@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("long", [False, True])
def test_decode_bad_lengths_and_pages(portable, long):
    lens = (900, 2500, 40) if long else (40, 60, 17)
    q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, 4, 2, 128, 16, 64, BF16, 14)
    for bad in (-1, max(lens) + 1, 1 << 30):
        m = n.clone()
        m[1] = bad
        out = run_decode(q, pool, tables, m, max_len=max(lens), portable=portable,
                         status=pa.PA_ERR_BAD_SEQ_LEN).cpu()
        assert torch.isnan(out[1]).all()
        kr.assert_decode(out[::2], ref[::2], mag[::2], step[::2], BF16, portable)
    for bad in (-1, pool.k.shape[0], 1 << 30):
        t = tables.clone()
        t[1, (lens[1] - 1) // 16] = bad
        out = run_decode(q, pool, t, n, portable=portable, status=pa.PA_ERR_BAD_BLOCK_ID).cpu()
        assert torch.isnan(out[1]).all()
        kr.assert_decode(out[::2], ref[::2], mag[::2], step[::2], BF16, portable)


def test_decode_empty_and_bound_zero():
    q, pool, tables, n, *_ = kr.decode_problem((0, 0), 4, 2, 128, 16, 64, BF16, 15)
    for portable in (False, True):
        assert (run_decode(q, pool, tables, n, max_len=0, portable=portable) == 0).all()
        assert (run_decode(q, pool, tables, n, max_len=16, portable=portable) == 0).all()
        out = run_decode(q, pool, tables, torch.tensor([0, 1]), max_len=0, portable=portable,
                         status=pa.PA_ERR_BAD_SEQ_LEN)
        assert (out[0] == 0).all() and torch.isnan(out[1]).all()


def test_decode_is_the_same_for_any_place_of_the_pages_and_any_run():
    q, pool, tables, n, ref, mag, step = kr.decode_problem((3000, 900), 8, 2, 128, 16, 64, BF16, 16)
    a = run_decode(q, pool, tables, n)
    assert torch.equal(a, run_decode(q, pool, tables, n))
    perm = torch.randperm(pool.k.shape[0], generator=torch.Generator().manual_seed(1))
    moved = tables.clone()
    moved[tables >= 0] = torch.argsort(perm)[tables[tables >= 0].long()].int()
    pool.k, pool.v, pool.ks, pool.vs = (x[perm] for x in (pool.k, pool.v, pool.ks, pool.vs))
    assert torch.equal(a, run_decode(q, pool, moved, n))


def test_one_workspace_for_smaller_steps():
    big = kr.decode_problem((2000,) * 40, 8, 2, 64, 16, 64, BF16, 17)
    ws = pa.alloc_kv4_workspace(big[0].cuda(), big[1].k, big[1].ks, big[2], max_seq_len=2000)
    for lens in ((2000,), (1, 700), (5,) * 40, (1500, 0, 3)):
        q, pool, tables, n, ref, mag, step = kr.decode_problem(lens, 8, 2, 64, 16, 64, BF16, 18)
        got = run_decode(q, pool, tables, n, workspace=ws)
        kr.assert_decode(got, ref, mag, step, BF16, False)


def test_two_graphs_that_share_a_workspace():
    a = kr.decode_problem((3000, 40), 8, 2, 64, 16, 64, BF16, 30)
    b = kr.decode_problem([int(x) for x in range(1, 400, 2)] + [2600], 8, 4, 64, 16, 64, BF16, 31)
    runs = []
    big = b[0].cuda()
    ws = pa.alloc_kv4_workspace(big, b[1].k, b[1].ks, torch.zeros(201, 188), max_seq_len=3000)
    for q, pool, tables, n, ref, mag, step in (a, b):
        qg, caches, bt, ng = q.cuda(), pool.cuda(), i32(tables), i32(n)
        bt = torch.nn.functional.pad(bt, (0, 188 - bt.shape[1]), value=-1).contiguous()
        out = torch.empty_like(qg)

        def call(qg=qg, caches=caches, bt=bt, ng=ng, out=out):
            pa.decode_kv4(qg, *caches, bt, ng, out, ws, max_seq_len=3000, scale=64 ** -0.5)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, out, ref, mag, step, (qg, caches, bt, ng)))
    for _ in range(3):
        for graph, out, ref, mag, step, _ in runs:
            out.fill_(math.nan)
            graph.replay()
            kr.assert_decode(out, ref, mag, step, BF16, False)
    assert pa.read_device_status(ws) == pa.PA_OK


def random_pool(blocks, hkv, bs, d, group, seed):
    """Codes at random, steps of 0.2 to 0.4, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc, ks, vs = pa.alloc_kv4_cache(blocks, hkv, bs, d, group_size=group)
    for codes, pairs in ((kc, ks), (vc, vs)):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda"))
        pairs[..., 0] = 0.2 + 0.2 * torch.rand(pairs.shape[:-1], generator=g, device="cuda")
        pairs[..., 1] = -8 * pairs[..., 0]
    return (kc, vc, ks, vs), g


@pytest.mark.parametrize("seqs,longest,hq,hkv", [(5000, 40, 2, 1), (1, 600000, 8, 1),
                                                 (3, 250000, 10, 1), (700, 3000, 4, 2),
                                                 (1000, 2500, 4, 2)])
def test_many_sequences_and_long_ones_beside_the_portable_kernel(seqs, longest, hq, hkv):
    d, bs, group = 64, 16, 32
    lens = torch.randint(0, longest + 1, (seqs,), generator=torch.Generator().manual_seed(seqs))
    lens[0] = longest
    pages = (lens + bs - 1) // bs
    total = int(pages.sum())
    caches, g = random_pool(total + 1, hkv, bs, d, group, 1)
    tables = torch.full((seqs, int(pages.max())), -1, dtype=torch.int32)
    order = torch.randperm(total, generator=torch.Generator().manual_seed(2)).int()
    at = torch.cumsum(pages, 0) - pages
    col = torch.arange(tables.shape[1])[None, :]
    live = col < pages[:, None]
    tables[live] = order[(at[:, None] + col)[live]]
    q = torch.randn(seqs, hq, d, generator=g, device="cuda").to(BF16)
    bt, n = tables.cuda(), lens.int().cuda()
    outs = []
    ws = pa.alloc_kv4_workspace(q, caches[0], caches[2], bt, max_seq_len=longest)
    for portable in (False, True):
        out = torch.full(q.shape, math.nan, device="cuda")
        pa.decode_kv4(q, *caches, bt, n, out, ws, max_seq_len=longest, scale=d ** -0.5,
                      portable=portable)
        assert pa.read_device_status(ws) == pa.PA_OK
        outs.append(out.double())
    # both within assert_decode's bounds of the same values: |v| below 8 steps, steps of 0.4
    bound = 2 * 2e-5 * (3.2 + 15 * 0.4) + 2.0 ** -10 * 8 * 0.4 + 1e-5
    assert torch.isfinite(outs[0]).all()
    assert float((outs[0] - outs[1]).abs().max()) <= bound
    assert (outs[0][(lens == 0).cuda()] == 0).all()


@pytest.mark.parametrize("portable", [False, True])
def test_the_longest_sequence(portable):
    """2^31 - 4097 tokens, in 4 pages taken over and over: positions, parts and their count stay
    in their bits.  The reference counts each of the pages' tokens as often as the row has it."""
    d, bs, blocks, n = 64, 65536, 4, 2 ** 31 - 4097
    pool = kr.Pool(blocks, 1, bs, d, 32, BF16, seed=41)
    pages = torch.empty(blocks, dtype=torch.int32)
    pool.fill(pages, blocks * bs)
    q = pool.randn(1, 2, d)
    k, v, s = pool.rows(pages, blocks * bs)
    table = pages[torch.arange(-(-n // bs)) % blocks]
    times = torch.full((blocks * bs,), n // (blocks * bs), dtype=torch.float64)
    times[:n % (blocks * bs)] += 1
    ref, mag, step = (torch.empty(1, 2, d, dtype=torch.float64) for _ in range(3))
    for h in range(2):
        a = (k[:, 0] @ q[0, h].double()) * d ** -0.5
        w = torch.softmax(a + times.log(), 0)
        ref[0, h], mag[0, h], step[0, h] = w @ v[:, 0], w @ v[:, 0].abs(), w @ s[:, 0]
    got = run_decode(q, pool, table[None], torch.tensor([n], dtype=torch.int32), out_dtype=F32,
                     portable=portable, partition_size=1 << 18)
    kr.assert_decode(got, ref, mag, step, F32, portable)


def test_pools_past_32_bits():
    """Codes past 2^31 bytes and pages whose elements pass 2^32: store, load and decode there."""
    hkv, d, bs, group = 8, 256, 64, 128
    blocks = (1 << 31) // (hkv * bs * d // 2) + 40
    kc, vc, ks, vs = pa.alloc_kv4_cache(blocks, hkv, bs, d, group_size=group)
    g = torch.Generator().manual_seed(3)
    n = 150
    k, v = (torch.randn(n, hkv, d, generator=g).to(BF16) for _ in range(2))
    table = torch.tensor([[blocks - 1, blocks - 30, blocks - 7]], dtype=torch.int32)
    t = torch.arange(n)
    slots = table[0, t // bs].long() * bs + t % bs
    pa.store_kv4(k.cuda(), v.cuda(), slots.cuda(), kc, vc, ks, vs)
    q = torch.randn(1, 16, d, generator=g).to(BF16)
    out = torch.empty_like(q, device="cuda")
    ws = pa.alloc_kv4_workspace(out, kc, ks, table, max_seq_len=n)
    pa.decode_kv4(q.cuda(), kc, vc, ks, vs, table.cuda(), i32([n]), out, ws, max_seq_len=n,
                  scale=d ** -0.5)
    wide = [torch.zeros(4, hkv, bs, d, dtype=BF16, device="cuda") for _ in range(2)]
    pa.load_kv4(kc, vc, ks, vs, table.cuda(), i32([n]), i32([[2, 0, 3]]), *wide, max_seq_len=n)
    (ck, sk, mk), (cv, sv, mv) = kr.quantise(k, group), kr.quantise(v, group)
    kv, vv = (kr.values(kr.pack(c), torch.stack([s, m], -1)) for c, s, m in ((ck, sk, mk),
                                                                             (cv, sv, mv)))
    place = torch.tensor([2, 0, 3])[t // bs]
    assert torch.equal(wide[0].cpu()[place, :, t % bs], kv.float().to(BF16))
    assert torch.equal(wide[1].cpu()[place, :, t % bs], vv.float().to(BF16))
    for h in range(16):
        w = torch.softmax((kv[:, h // 2] @ q[0, h].double()) * d ** -0.5, 0)
        step = w @ sv[:, h // 2].repeat_interleave(group, -1)
        kr.assert_decode(out[0, h], w @ vv[:, h // 2], w @ vv[:, h // 2].abs(), step, BF16, False)


# ---------------------------------------------------------------- together

def test_a_serving_step_on_the_4_bit_cache():
    """Prompt and decode steps as a server runs them: plan, norm + rotation with three axes,
    store, the context widened for the prefill of the next chunk, decode; the decode step
    captured in a graph and replayed for later tokens."""
    hq, hkv, d, bs, group = 8, 2, 128, 16, 64
    of = pa.rope_axes((24, 20, 20), True)
    B, pool_blocks = 3, 40
    dev = "cuda"
    g = torch.Generator().manual_seed(4)
    cs = torch.randn(400, d, generator=g)
    cs = torch.cat([torch.cos(cs[:, :64]), torch.sin(cs[:, :64])], 1).contiguous().to(dev)
    kc, vc, ks, vs = pa.alloc_kv4_cache(pool_blocks, hkv, bs, d, group_size=group)
    tables = torch.full((B, 12), -1, dtype=torch.int32, device=dev)
    free = torch.arange(pool_blocks, dtype=torch.int32, device=dev)
    count = i32([pool_blocks])
    ctx = np.zeros(B, int)
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]   # what the cache stands for

    def rows(T):
        return torch.randn(T, hq + 2 * hkv, d, generator=g).to(BF16)

    def reference(q, b, upto):
        k, v = torch.cat(keys[b])[:upto], torch.cat(vals[b])[:upto]
        return sr.rows_attend(q, k, v, d ** -0.5)

    def step(new):
        nonlocal ctx, count
        T = int(new.sum()) + 2
        start, lens = i32([0] * (B + 1)), i32([0] * B)
        pos, slots = i32([0] * T), torch.zeros(T, dtype=torch.int64, device=dev)
        left = i32([0])
        pa.plan_step(i32(ctx), i32(new), free, count, tables, start, lens, pos, slots, left,
                     block_size=bs, num_blocks=pool_blocks)
        count = left
        x = rows(T).to(dev)
        axes = torch.stack([pos, pos // 7, pos % 7]).contiguous()
        q = torch.empty(T, hq, d, dtype=BF16, device=dev)
        k, v = (torch.empty(T, hkv, d, dtype=BF16, device=dev) for _ in range(2))
        pa.qk_norm_rope_axes(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], axes, slots, cs, q,
                             axis_of=of, k_out=k, v_out=v)
        pa.store_kv4(k, v, slots, kc, vc, ks, vs, k_out=k, v_out=v)
        live = int(new.sum())
        at = start.cpu().tolist()
        for b in range(B):
            keys[b].append(k[at[b]:at[b + 1]].double().cpu())
            vals[b].append(v[at[b]:at[b + 1]].double().cpu())
        old = ctx.copy()
        ctx = ctx + new
        return q[:live], k[:live], v[:live], start, lens, old, at

    for new in (np.array([40, 7, 0]), np.array([20, 33, 50])):
        q, k, v, start, lens, old, at = step(new)
        # the cached context, widened
        to = torch.arange(B * 12, dtype=torch.int32, device=dev).view(B, 12)
        wide = [torch.full((B * 12, hkv, bs, d), math.nan, dtype=BF16, device=dev)
                for _ in range(2)]
        pa.load_kv4(kc, vc, ks, vs, tables, i32(old), to, *wide, max_seq_len=64)
        out = torch.empty_like(q)
        pa.prefill(q, k, v, *wide, to, start, i32(old), out, max_query_len=64, max_ctx_len=64,
                   scale=d ** -0.5)
        for b in range(B):
            for i in range(0, int(new[b]), 9):
                ref, mag = reference(q[at[b] + i].cpu(), b, old[b] + i + 1)
                sr.assert_within(out[at[b] + i], ref, mag, BF16, BF16, True)
    # decode steps: the attention captured once, then replayed on new queries and lengths
    ws = q_buf = graph = None
    for turn in range(4):
        q, k, v, start, lens, old, at = step(np.ones(B, int))
        if graph is None:
            q_buf, lens_buf = q.clone(), lens.clone()
            out = torch.empty_like(q)
            ws = pa.alloc_kv4_workspace(q, kc, ks, tables, max_seq_len=192)
            call = lambda: pa.decode_kv4(q_buf, kc, vc, ks, vs, tables, lens_buf, out, ws,
                                         max_seq_len=192, scale=d ** -0.5)
            call()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
        q_buf.copy_(q), lens_buf.copy_(lens)
        out.fill_(math.nan)
        graph.replay()
        for b in range(B):
            ref, mag = reference(q[b].cpu(), b, int(ctx[b]))
            # k_out and v_out are the values rounded to bf16, half a step: logits move by up to
            # 2^-8 of sum |q k| * scale, about 8 here, the weights by twice that, the values by
            # 2^-8; scales are below 0.5 (a fifteenth of a range of about 5)
            bound = (3 * 2.0 ** -8 * 8) * mag + 2.0 ** -11 * 8 * 0.5 + 2.0 ** -8 * ref.abs()
            assert ((out[b].double().cpu() - ref).abs() <= bound).all()
    assert pa.read_device_status(ws) == pa.PA_OK


def test_two_streams_each_with_its_workspace():
    problems = [kr.decode_problem((1500, 20), 8, 2, 128, 16, 64, BF16, s) for s in (20, 21)]
    state = []
    for q, pool, tables, n, *_ in problems:
        qg, caches, bt = q.cuda(), pool.cuda(), i32(tables)
        state.append((qg, caches, bt, i32(n), torch.empty_like(qg), torch.cuda.Stream(),
                      pa.alloc_kv4_workspace(qg, caches[0], caches[2], bt, max_seq_len=1500)))
    torch.cuda.synchronize()
    for _ in range(20):
        for q, (kc, vc, ks, vs), bt, n, out, stream, ws in state:
            pa.decode_kv4(q, kc, vc, ks, vs, bt, n, out, ws, max_seq_len=1500, scale=128 ** -0.5,
                          stream=stream)
    torch.cuda.synchronize()
    for (*_, ref, mag, step), (_, _, _, _, out, _, ws) in zip(problems, state):
        kr.assert_decode(out, ref, mag, step, BF16, False)
        assert pa.read_device_status(ws) == pa.PA_OK


def test_bindings_check_shapes_and_types():
    pool = kr.Pool(4, 2, 16, 128, 64, BF16, 1)
    kc, vc, ks, vs = pool.cuda()
    k = torch.zeros(3, 2, 128, dtype=BF16, device="cuda")
    v, slots = k.clone(), torch.arange(3, device="cuda")
    pa.store_kv4(k, v, slots, kc, vc, ks, vs)
    for args in ((k[:2], v, slots, kc, vc, ks, vs), (k, v, slots.int(), kc, vc, ks, vs),
                 (k.float(), v, slots, kc, vc, ks, vs), (k, v, slots, kc.char(), vc, ks, vs),
                 (k, v, slots, kc, vc[:3], ks, vs), (k, v, slots, kc, vc, ks.half(), vs.half()),
                 (k, v, slots, kc, vc, ks[:, :, :8], vs[:, :, :8]),
                 (k, v, slots[:2], kc, vc, ks, vs), (k[:, :, :64], v, slots, kc, vc, ks, vs)):
        with pytest.raises(pa.PaError):
            pa.store_kv4(*args)
    wide = torch.zeros(4, 2, 16, 128, dtype=BF16, device="cuda")
    bt, n = i32([[0, 1]]), i32([20])
    pa.load_kv4(kc, vc, ks, vs, bt, n, bt, wide, wide.clone(), max_seq_len=20)
    for args in ((bt, n, bt, wide, wide), (bt, n, bt, wide[:, :1].contiguous(), wide.clone()),
                 (bt, n, bt, wide.half(), wide.half()), (bt, n.long(), bt, wide, wide.clone()),
                 (bt, i32([1, 2]), bt, wide, wide.clone())):
        with pytest.raises(pa.PaError):
            pa.load_kv4(kc, vc, ks, vs, *args, max_seq_len=20)
    q = torch.zeros(1, 8, 128, dtype=BF16, device="cuda")
    ws = pa.alloc_kv4_workspace(q, kc, ks, bt, max_seq_len=20)
    out = q.clone()
    pa.decode_kv4(q, kc, vc, ks, vs, bt, n, out, ws, max_seq_len=20, scale=1.0)
    for kw in (dict(q=q.half()), dict(q=q[:, :, :64].contiguous()), dict(out=out[:, :4]),
               dict(n=n.long()), dict(bt=i32([[0], [1]])), dict(ws=ws[:512]),
               dict(out=out.half())):
        a = dict(q=q, bt=bt, n=n, out=out, ws=ws)
        a.update(kw)
        with pytest.raises(pa.PaError):
            pa.decode_kv4(a["q"], kc, vc, ks, vs, a["bt"], a["n"], a["out"], a["ws"],
                          max_seq_len=20, scale=1.0)
