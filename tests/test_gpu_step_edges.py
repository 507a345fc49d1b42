"""The serving-step operators at the edges of their definitions: values that are
not finite, weights far below the largest, bounds of zero, calls captured in
graphs, repeated on one workspace and made by two threads."""
import math
import threading

import numpy as np
import pytest
import torch

import paged_attention_decode_v2_gb300 as pa
import step_reference as sr
from test_gpu_step import _cos_sin, _run_prefix, _run_window, _run_window_prefill, i32

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------- partial results of an earlier grid

@pytest.mark.parametrize("hq,hkv,d,bs,dtype,prefix,lens", [
    (24, 4, 256, 16, BF16, 3000, tuple(range(0, 80, 2))),     # joins as it attends
    (8, 2, 128, 32, F16, 3000, (700, 3, 0, 90)),              # three kernels
])
def test_decode_prefix_again_and_again_on_one_workspace(hq, hkv, d, bs, dtype, prefix, lens):
    """The last kernel starts before the partials of the call are written: what
    it joins are this call's, not the last one's."""
    p = sr.prefix_problem(prefix, lens, hq, hkv, d, bs, dtype, seed=3)
    gq, kc, vc, shared, gt, gl = [x.cuda() for x in (p[0], p[1].k, p[1].v, *p[2:5])]
    qs = [gq, -gq, gq.flip(0).contiguous()]
    ws = pa.alloc_prefix_workspace(gq, kc, gt, max_seq_len=max(lens), max_prefix_len=prefix)
    plen = i32([prefix])

    def call(q, out):
        pa.decode_prefix(q, kc, vc, shared, plen, gt, gl, out, ws, max_seq_len=max(lens),
                         max_prefix_len=prefix, scale=d ** -0.5)

    first = []
    for q in qs:
        first.append(torch.empty(q.shape, device="cuda"))
        call(q, first[-1])
        torch.cuda.synchronize()
    sr.assert_within(first[0], p[5], p[6], dtype, F32, True)
    outs = [torch.full(gq.shape, float("nan"), device="cuda") for _ in range(60)]
    for i, out in enumerate(outs):
        call(qs[i % 3], out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, first[i % 3]), i
    assert pa.read_device_status(ws) == pa.PA_OK


def test_decode_window_again_and_again_on_one_workspace():
    q, pg, tables, gl, ref, mag = sr.window_decode_problem([5000, 3001], 2048, 5, 24, 4, 256, 16,
                                                           BF16, seed=4)
    gq, kc, vc, gt, gl = [x.cuda() for x in (q, pg.k, pg.v, tables, gl)]
    qs = [gq, -gq, 0.5 * gq]
    ws = pa.alloc_window_workspace(gq, kc, gt, window=2048, num_sinks=5, max_seq_len=5000)

    def call(x, out):
        pa.decode_window(x, kc, vc, gt, gl, out, ws, window=2048, num_sinks=5, max_seq_len=5000,
                         scale=1 / 16)

    first = [torch.empty(gq.shape, device="cuda") for _ in qs]
    for x, out in zip(qs, first):
        call(x, out)
        torch.cuda.synchronize()
    sr.assert_within(first[0], ref, mag, BF16, F32, False)
    outs = [torch.full(gq.shape, float("nan"), device="cuda") for _ in range(60)]
    for i, out in enumerate(outs):
        call(qs[i % 3], out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, first[i % 3]), i


# ------------------------------------------------ norm + rotation: copied elements

def _bits(x):
    return x.contiguous().view(torch.int32 if x.dtype == F32 else torch.int16)


def _same_bits(got, want):
    got, want = got.cpu(), want.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(_bits(got)[~nan], _bits(want)[~nan])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d,rot,inter", [(64, 0, False), (128, 0, True), (256, 0, False),
                                         (64, 32, True), (64, 16, False), (128, 64, False),
                                         (256, 112, True), (256, 240, False)])
def test_elements_outside_the_rotation_are_copied(dtype, d, rot, inter):
    """Without weights they are the input's bits: infinities, NaN and -0 among
    them, none of which reaches another element."""
    T, hq, hkv, bs, sx = 21, 5, 2, 16, d == 64
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn(T, hq + 2 * hkv, d, generator=g).to(dtype)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 0.0]).to(dtype)
    pick = torch.randint(0, 12, x.shape, generator=g)
    pick[..., :rot] = 11                                   # the rotated part stays finite
    pick[:, hq + hkv:] = torch.randint(0, 12, pick[:, hq + hkv:].shape, generator=g)  # values: any
    x = torch.where(pick < 5, odd[pick.clamp(max=4)], x)
    nb = 4
    kc = torch.zeros(nb, hkv, bs, d, dtype=dtype)
    vc = torch.zeros_like(kc)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    gx = x.cuda()
    gk, gv = [t.cuda() for t in (sr.split_x(kc, vc) if sx else (kc, vc))]
    q_out = torch.empty(T, hq, d, dtype=dtype, device="cuda")
    k_out, v_out = [torch.empty(T, hkv, d, dtype=dtype, device="cuda") for _ in range(2)]
    status = i32([0])
    pos = torch.arange(T, dtype=torch.int32, device="cuda") if rot else None
    pa.qk_norm_rope(gx[:, :hq], gx[:, hq:hq + hkv], gx[:, hq + hkv:], pos, slots.cuda(),
                    _cos_sin(rot).cuda() if rot else None, q_out, gk, gv, interleaved=inter,
                    k_out=k_out, v_out=v_out, split_x=sx, status=status)
    assert int(status) == 0
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    _same_bits(q_out[..., rot:], q[..., rot:])
    _same_bits(k_out[..., rot:], k[..., rot:])
    _same_bits(v_out, v)
    for got, src in ((q_out, q), (k_out, k)):
        assert torch.isfinite(got[..., :rot]).all()
        if rot:
            want = sr.norm_rope(torch.where(torch.isfinite(src), src, 0), None, _cos_sin(rot),
                                torch.arange(T), 0.0, 0.0, inter)[..., :rot]
            # two products and a sum in float32, one rounding
            size = src[..., :rot].double().abs().amax(-1, keepdim=True)
            bound = sr.HALF_STEP[dtype] * want.abs() + 4 * 2.0 ** -24 * size + 2.0 ** -25
            assert (got[..., :rot].double().cpu() - want).abs().le(bound).all()
    ek, ev = kc.clone(), vc.clone()
    ek[slots // bs, :, slots % bs] = k_out.cpu()
    ev[slots // bs, :, slots % bs] = v
    if sx:
        ek, ev = sr.split_x(ek, ev)
    _same_bits(gk, ek)
    _same_bits(gv, ev)


def test_zeros_outside_the_rotation_keep_their_sign_under_a_norm():
    T, hq, hkv, d, rot = 3, 4, 1, 128, 32
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, hq + 2 * hkv, d, generator=g).to(BF16)
    x[..., rot::3] = -0.0
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF16)
    assert (w > 0).all()
    gx, gw = x.cuda(), w.cuda()
    q_out = torch.empty(T, hq, d, dtype=BF16, device="cuda")
    pa.qk_norm_rope(gx[:, :hq], gx[:, hq:hq + hkv], gx[:, hq + hkv:], i32(range(T)),
                    torch.arange(T, device="cuda"), _cos_sin(rot).cuda(), q_out, q_weight=gw,
                    k_weight=gw)
    assert torch.equal(torch.signbit(q_out).cpu()[..., rot:], torch.signbit(x[:, :hq])[..., rot:])


def test_a_bad_position_makes_whole_rows_nan():
    """The elements outside the rotation too."""
    T, hq, hkv, d, rot = 5, 3, 2, 128, 32
    x = torch.randn(T, hq + 2 * hkv, d, device="cuda").to(BF16)
    q_out = torch.zeros(T, hq, d, dtype=BF16, device="cuda")
    k_out = torch.zeros(T, hkv, d, dtype=BF16, device="cuda")
    pa.qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i32([0, -1, 2, 300, 4]),
                    torch.arange(T, device="cuda"), _cos_sin(rot).cuda(), q_out, k_out=k_out)
    for t in (q_out, k_out):
        assert torch.isnan(t[[1, 3]]).all() and torch.isfinite(t[[0, 2, 4]]).all()


def test_slots_without_caches_only_mark_padding():
    T, hq, hkv, d = 4, 2, 1, 64
    x = torch.randn(T, hq + 2 * hkv, d, device="cuda").to(BF16)
    slots = torch.tensor([2 ** 30, 2 ** 31 + 7, -1, 2 ** 40], device="cuda")
    q_out = torch.full((T, hq, d), 9.0, dtype=BF16, device="cuda")
    status = i32([0])
    pa.qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], None, slots, None, q_out,
                    status=status)
    assert int(status) == 0
    assert torch.equal(q_out[[0, 1, 3]], x[[0, 1, 3], :hq]) and (q_out[2] == 9.0).all()


# --------------------------------------------------- values that are not finite

@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [(8, 2, 128, 16, BF16), (24, 4, 256, 16, F16),
                                               (4, 2, 64, 16, BF16), (4, 2, 128, 8, F32)])
@pytest.mark.parametrize("portable", [False, True])
def test_decode_prefix_with_nan(hq, hkv, d, bs, dtype, portable):
    G = hq // hkv
    fresh = lambda: sr.prefix_problem(900, (30, 0, 45), hq, hkv, d, bs, dtype, seed=7)
    tc = not portable and d > 64 and dtype != F32
    # a key of the prefix: the heads that see it, and no word of a bad block
    p = fresh()
    p[1].k[p[2][3], 1, 2, 5] = math.nan
    out, ws = _run_prefix(p, 900, portable=portable, check=False)
    assert torch.isnan(out[:, G:2 * G]).all()
    rest = [h for h in range(hq) if h // G != 1]
    sr.assert_within(out[:, rest], p[5][:, rest], p[6][:, rest], dtype, F32, tc)
    assert pa.read_device_status(ws) == pa.PA_OK
    # whole query rows, one with tokens of its own and one without
    p = fresh()
    p[0][0] = math.nan
    p[0][1, 0] = math.nan
    out, ws = _run_prefix(p, 900, portable=portable, check=False)
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, 0]).all()
    sr.assert_within(out[1, 1:], p[5][1, 1:], p[6][1, 1:], dtype, F32, tc)
    sr.assert_within(out[2], p[5][2], p[6][2], dtype, F32, tc)
    assert pa.read_device_status(ws) == pa.PA_OK
    # and beside a bad block the status names the block
    p[2][1] = -1
    out, ws = _run_prefix(p, 900, portable=portable, check=False)
    assert torch.isnan(out).all()
    assert pa.read_device_status(ws) == pa.PA_ERR_BAD_BLOCK_ID


@pytest.mark.parametrize("hq,hkv,d,bs,dtype,kw", [
    (8, 2, 128, 16, BF16, {}), (8, 2, 128, 16, BF16, dict(portable=True)),
    (8, 2, 128, 16, F16, dict(sx=True)), (4, 2, 64, 16, BF16, {}), (4, 2, 128, 8, F32, {})])
def test_decode_prefix_with_nan_and_no_prefix(hq, hkv, d, bs, dtype, kw):
    """Own lists alone, of one part and of three: every kernel that takes them."""
    G = hq // hkv
    p = sr.prefix_problem(0, (30, 300, 45), hq, hkv, d, bs, dtype, seed=16)
    p[0][0] = math.nan
    p[0][1, 0] = math.nan
    p[1].k[p[3][2, 1], 1, 3, 7] = math.nan
    out, ws = _run_prefix(p, 0, P=128, check=False, **kw)
    assert torch.isnan(out[0]).all() and torch.isnan(out[1, 0]).all()
    assert torch.isnan(out[2, G:2 * G]).all()
    sr.assert_within(out[1, 1:], p[5][1, 1:], p[6][1, 1:], dtype, F32, False)
    sr.assert_within(out[2, :G], p[5][2, :G], p[6][2, :G], dtype, F32, False)
    assert pa.read_device_status(ws) == pa.PA_OK


@pytest.mark.parametrize("path", ["v1", "v2"])
def test_cuda_core_decode_with_nan(path):
    """The same kernel behind pa_decode: as the tensor-core ones, NaN and not zeros."""
    q, pg, tables, gl, ref, mag = sr.window_decode_problem([300, 77, 60], 10 ** 6, 0, 8, 2, 128, 16,
                                                           BF16, seed=17)
    q[1] = math.nan
    pg.k[tables[2, 1], 0, 3, 7] = math.nan
    g = [x.cuda() for x in (q, pg.k, pg.v, tables, gl)]
    for portable in (False, True):
        out = torch.empty(q.shape, device="cuda")
        kw = dict(max_seq_len=300, scale=128 ** -0.5, portable=portable)
        if path == "v1":
            pa.decode_v1(*g, out, **kw)
        else:
            params = pa.make_params(g[0], g[1], g[3], max_seq_len=300, scale=1.0,
                                    partition_size=128)
            pa.decode_v2(*g, out, pa.alloc_workspace(params), partition_size=128, **kw)
        assert torch.isnan(out[1]).all() and torch.isnan(out[2, :4]).all()
        sr.assert_within(out[0], ref[0], mag[0], BF16, F32, False)
        sr.assert_within(out[2, 4:], ref[2, 4:], mag[2, 4:], BF16, F32, False)


def test_decode_prefix_of_many_short_sequences_with_nan():
    hq, hkv, d, bs = 8, 4, 128, 32
    lens = [int(x) for x in np.random.RandomState(1).randint(0, 90, size=41)]
    p = sr.prefix_problem(700, lens, hq, hkv, d, bs, BF16, seed=8)
    empty = lens.index(0) if 0 in lens else 0
    p[0][5] = math.nan
    p[0][empty, 3] = math.nan
    out, ws = _run_prefix(p, 700, check=False)
    assert torch.isnan(out[5]).all() and torch.isnan(out[empty, 3]).all()
    good = [i for i in range(41) if i not in (5, empty)]
    sr.assert_within(out[good], p[5][good], p[6][good], BF16, F32, True)
    assert pa.read_device_status(ws) == pa.PA_OK


@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [(8, 2, 128, 16, BF16), (24, 4, 256, 16, F16),
                                               (4, 2, 64, 16, F16), (4, 2, 128, 8, F32)])
@pytest.mark.parametrize("portable", [False, True])
@pytest.mark.parametrize("window,P", [(1500, 128), (100, 512)])
def test_decode_window_with_nan(hq, hkv, d, bs, dtype, portable, window, P):
    G = hq // hkv
    q, pg, tables, gl, ref, mag = sr.window_decode_problem([2500, 777, 60], window, 9, hq, hkv, d,
                                                           bs, dtype, seed=9)
    q[1] = math.nan
    pg.k[tables[2, 1], 0, 3, 7] = math.nan
    out, ws = _run_window(q, pg, tables, gl, window, 9, portable=portable, P=P, check=False)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2, :G]).all()
    sr.assert_within(out[0], ref[0], mag[0], dtype, F32, False)
    sr.assert_within(out[2, G:], ref[2, G:], mag[2, G:], dtype, F32, False)
    assert pa.read_device_status(ws) == pa.PA_OK


@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [(8, 2, 128, 16, BF16), (6, 1, 256, 16, F16),
                                               (4, 2, 64, 16, F16), (4, 2, 128, 8, F32)])
@pytest.mark.parametrize("portable", [False, True])
def test_prefill_window_with_nan(hq, hkv, d, bs, dtype, portable):
    """A NaN query row is one row's; a NaN key those rows' that see it."""
    G, C, n, window, sinks = hq // hkv, 300, 150, 40, 3
    p = sr.window_prefill_problem((C,), (n,), window, sinks, hq, hkv, d, bs, dtype, seed=10)
    q, k, v, pg, tables, start, ctx, ref, mag = p
    q[7] = math.nan
    k[50, 0, 3] = math.nan
    pg.k[tables[0, 290 // bs], hkv - 1, 290 % bs, 1] = math.nan
    out = _run_window_prefill(p, window, sinks, portable=portable)
    bad = torch.zeros(n, hq, dtype=torch.bool)
    bad[7] = True
    for i in range(n):
        see = sr.visible(C + i, window, sinks)
        if C + 50 in see:
            bad[i, :G] = True
        if 290 in see:
            bad[i, hq - G:] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), bad)
    rounded = not portable and d > 64 and dtype != F32
    sr.assert_within(out.cpu()[~bad], ref[~bad], mag[~bad], dtype, F32, rounded)


# ------------------------------------------ many weights far below the largest

def _faint(dtype, n, hkv, d, bs, below, seed):
    """One token that outweighs each of the others by exp(below), its value 0 and
    theirs 1: caches, table, the query row and the exact output."""
    g = torch.Generator().manual_seed(seed)
    blocks = -(-n // bs)
    kc = torch.zeros(blocks, hkv, bs, d, dtype=dtype)
    vc = torch.ones_like(kc)
    table = torch.randperm(blocks, generator=g).to(torch.int32)
    kc[table[0], :, 0, 0] = 16
    vc[table[0], :, 0] = 0
    q = torch.zeros(d, dtype=dtype)
    q[0] = below * d ** 0.5 / 16
    l0 = float(q[0].double()) * 16 * d ** -0.5
    return kc, vc, table, q, l0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d,bs,rows", [(4, 1, 128, 32, 3), (8, 1, 128, 16, 70),
                                              (6, 1, 256, 16, 5)])
def test_many_faint_tokens(dtype, hq, hkv, d, bs, rows):
    """20000 tokens of weight exp(-17.5) next to one of weight 1.  Each weight is
    off by half a step of the element type, or, in f16, by half of its smallest
    step 2^-24 at 2^7 below the largest weight's place: n 2^-32 in all."""
    n = 20000
    kc, vc, table, q1, l0 = _faint(dtype, n, hkv, d, bs, 17.5, 1)
    u = sr.HALF_STEP[dtype]
    extra = n * 2.0 ** -32 if dtype == F16 else 0.0

    def check(out, others):
        w = others * math.exp(-l0)
        ref = w / (1 + w)
        bound = (2e-5 + 2 * u) * ref + extra + 1e-6
        assert float((out.double() - ref).abs().max()) <= bound

    q = q1.expand(rows, hq, d).contiguous().cuda()
    gk, gv, gt = kc.cuda(), vc.cuda(), table.cuda()
    out = torch.empty(q.shape, device="cuda")
    tables = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    ws = pa.alloc_prefix_workspace(q, gk, tables, max_seq_len=bs, max_prefix_len=n)
    pa.decode_prefix(q, gk, gv, gt, i32([n]), tables, i32([0] * rows), out, ws, max_seq_len=bs,
                     max_prefix_len=n, scale=d ** -0.5)
    check(out, n - 1)
    # the same tokens as the context of a chunk, whose own are alike
    k = torch.zeros(rows, hkv, d, dtype=dtype, device="cuda")
    v = torch.ones_like(k)
    out.fill_(math.nan)
    pa.prefill_window(q, k, v, gk, gv, gt.view(1, -1), i32([0, rows]), i32([n]), out,
                      window=2 * n, max_query_len=rows, max_ctx_len=n, scale=d ** -0.5)
    for i in range(rows):
        check(out[i], n + i)


# --------------------------------------------------------------- bounds of zero

@pytest.mark.parametrize("B,hkv", [(3, 2), (40, 4)])
def test_lengths_past_bounds_of_zero_are_reported(B, hkv):
    """Nothing promised and something there: NaN rows and the status, whichever
    kernels run."""
    p = sr.prefix_problem(16, [4] * B, 2 * hkv, hkv, 128, 16, BF16, seed=12)
    q, pg, shared, tables, lens = [p[0].cuda(), p[1], p[2].cuda(), p[3].cuda(), p[4].cuda()]
    kc, vc = pg.k.cuda(), pg.v.cuda()
    out = torch.empty(q.shape, device="cuda")

    def call(max_seq, max_prefix, n, sl):
        ws = pa.alloc_prefix_workspace(q, kc, tables, max_seq_len=max_seq,
                                       max_prefix_len=max_prefix)
        out.fill_(3.0)
        pa.decode_prefix(q, kc, vc, shared, i32([n]), tables, sl, out, ws, max_seq_len=max_seq,
                         max_prefix_len=max_prefix, scale=1.0)
        return pa.read_device_status(ws)

    zero = torch.zeros_like(lens)
    assert call(4, 0, 5, lens) == pa.PA_ERR_BAD_SEQ_LEN and torch.isnan(out).all()
    assert call(0, 0, -1, zero) == pa.PA_ERR_BAD_SEQ_LEN and torch.isnan(out).all()
    one = zero.clone()
    one[1] = 2
    for n in (0, 16):
        assert call(0, n, n, one) == pa.PA_ERR_BAD_SEQ_LEN
        assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2]]).all()
    assert call(0, 0, 0, zero) == pa.PA_OK and (out == 0).all()
    assert call(0, 16, 16, zero) == pa.PA_OK and torch.isfinite(out).all()


def test_lengths_written_just_before_a_call_with_bounds_of_zero():
    """The join is the call's only kernel then, and waits for whatever ran before."""
    p = sr.prefix_problem(0, [0] * 5, 4, 2, 128, 16, BF16, seed=15)
    q, kc, vc, shared, tables = [x.cuda() for x in (p[0], p[1].k, p[1].v, p[2], p[3])]
    ws = pa.alloc_prefix_workspace(q, kc, tables, max_seq_len=0, max_prefix_len=0)
    B, plen, free = 5, i32([0]), i32(range(8))
    plan = dict(tables=torch.full((B, 4), -1, dtype=torch.int32, device="cuda"),
                query_start=i32([0] * (B + 1)), seq_lens=i32([0] * B), positions=i32([0] * B),
                slots=torch.zeros(B, dtype=torch.int64, device="cuda"), free_left=i32([0]))
    outs, news = [], [i32([0, 1, 0, 0, 1]), i32([0] * B)]
    for i in range(20):
        pa.plan_step(i32([0] * B), news[i % 2], free, i32([8]), *plan.values(), block_size=16,
                     num_blocks=8)
        out = torch.full(q.shape, 3.0, device="cuda")
        pa.decode_prefix(q, kc, vc, shared, plen, tables, plan["seq_lens"], out, ws, max_seq_len=0,
                         max_prefix_len=0, scale=1.0)
        outs.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        bad = news[i % 2].bool()
        assert torch.isnan(out[bad]).all() and (out[~bad] == 0).all()
    assert pa.read_device_status(ws) == pa.PA_ERR_BAD_SEQ_LEN


# ----------------------------------------------- captured, and from two threads

@pytest.mark.parametrize("hq,hkv,d,bs,lens", [
    (8, 2, 128, 16, (700, 3, 0, 90)), (24, 4, 256, 16, tuple(range(0, 84, 2))), (4, 2, 64, 8, (9, 0))])
def test_prefix_and_windowed_prefill_captured(hq, hkv, d, bs, lens):
    """Captured once, replayed with other queries and lengths: the eager calls'
    bits."""
    p = sr.prefix_problem(600, lens, hq, hkv, d, bs, BF16, seed=13)
    gq, kc, vc, shared, gt, gl = [x.cuda() for x in (p[0], p[1].k, p[1].v, *p[2:5])]
    plen = i32([600])
    ws = pa.alloc_prefix_workspace(gq, kc, gt, max_seq_len=max(lens), max_prefix_len=600)
    w = sr.window_prefill_problem((300, 40), (90, 33), 70, 5, hq, hkv, d, bs, BF16, seed=14)
    wq, wk, wv, wkc, wvc, wt, start, ctx = [x.cuda() for x in (*w[:3], w[3].k, w[3].v, *w[4:7])]
    eager = [torch.empty(gq.shape, device="cuda"), torch.empty(wq.shape, device="cuda")]
    replayed = [torch.empty_like(t) for t in eager]

    def calls(outs):
        pa.decode_prefix(gq, kc, vc, shared, plen, gt, gl, outs[0], ws, max_seq_len=max(lens),
                         max_prefix_len=600, scale=d ** -0.5)
        pa.prefill_window(wq, wk, wv, wkc, wvc, wt, start, ctx, outs[1], window=70, num_sinks=5,
                          max_query_len=90, max_ctx_len=300, scale=d ** -0.5)

    calls(eager)
    sr.assert_within(eager[0], p[5], p[6], BF16, F32, d > 64)
    sr.assert_within(eager[1], w[7], w[8], BF16, F32, d > 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(replayed)
    for step in range(4):
        gq.copy_(gq.roll(1, 0))
        wq.neg_()
        plen.sub_(37)
        gl.copy_((gl - 1).clamp(min=0))
        for t in replayed:
            t.fill_(math.nan)
        graph.replay()
        calls(eager)
        torch.cuda.synchronize()
        for a, b in zip(eager, replayed):
            assert torch.isfinite(a).all() and torch.equal(a, b), step
    assert pa.read_device_status(ws) == pa.PA_OK


def test_two_threads():
    """Each on a stream of its own: the bindings and the library keep nothing
    between calls that another thread's could reach."""
    probs = [sr.window_decode_problem([900 + 100 * i, 50], 300 + i, 3, 8, 2, 128, 16, BF16, 30 + i)
             for i in range(2)]
    errors = []

    def work(i):
        try:
            q, pg, tables, gl, ref, mag = probs[i]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g = [x.cuda() for x in (q, pg.k, pg.v, tables, gl)]
                ws = pa.alloc_window_workspace(g[0], g[1], g[3], window=300 + i, num_sinks=3,
                                               max_seq_len=900 + 100 * i)
                for _ in range(200):
                    out = torch.full(q.shape, math.nan, device="cuda")
                    pa.decode_window(g[0], g[1], g[2], g[3], g[4], out, ws, window=300 + i,
                                     num_sinks=3, max_seq_len=900 + 100 * i, scale=128 ** -0.5)
                    with pytest.raises(pa.PaError):
                        pa.decode_window(g[0], g[1], g[2], g[3], g[4], out, ws, window=-i,
                                         num_sinks=3, max_seq_len=900 + 100 * i, scale=128 ** -0.5)
                s.synchronize()
                sr.assert_within(out, ref, mag, BF16, F32, False)
                assert pa.read_device_status(ws) == pa.PA_OK
        except BaseException as e:  # noqa: BLE001  (handed to the test's thread)
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
