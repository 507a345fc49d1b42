"""The serving-step operators on the GPU against plain float64 references:
the step plan, norm + rotation + cache write, windowed decode and prefill,
shared-prefix decode, and a run of them together."""
import numpy as np
import pytest
import torch

import paged_attention_decode_v2_gb300 as pa
import step_reference as sr
from gpu_helpers import GUARD_F, _guarded, _guards_intact

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


# ---------------------------------------------------------------- step plan

def _plan_buffers(B, T):
    z = dict(device="cuda")
    return dict(query_start=torch.full((B + 1,), -7, dtype=torch.int32, **z),
                seq_lens=torch.full((B,), -7, dtype=torch.int32, **z),
                positions=torch.full((T,), -7, dtype=torch.int32, **z),
                slots=torch.full((T,), -7, dtype=torch.int64, **z),
                free_left=torch.full((1,), -7, dtype=torch.int32, **z))


def _plan_case(B, bs, ctx_hi, new_hi, seed, width=None, zero_new=0.2):
    r = np.random.RandomState(seed)
    ctx = r.randint(0, ctx_hi + 1, size=B)
    new = r.randint(0, new_hi + 1, size=B) * (r.rand(B) >= zero_new)
    width = width or int((ctx + new).max() // bs + 2)
    pool = B * width + 50
    ids = r.permutation(pool)
    tables = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        n = -(-ctx[b] // bs)
        tables[b, :n] = ids[at:at + n]
        at += n
    return ctx, new, ids[at:].astype(np.int32), tables, pool


def _run_plan(ctx, new, free, count, tables, T, bs, pool, base=None):
    B = len(ctx)
    out = _plan_buffers(B, T)
    gt = i32(tables)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.plan_step(i32(ctx), i32(new), i32(free), i32([count]), gt, out["query_start"],
                 out["seq_lens"], out["positions"], out["slots"], out["free_left"],
                 block_size=bs, num_blocks=pool, base_len=None if base is None else i32([base]),
                 status=status)
    want = sr.plan(ctx, new, free, count, tables, T, bs, pool, base or 0)
    got = (gt, out["query_start"], out["seq_lens"], out["positions"], out["slots"])
    for name, g, w in zip(("tables", "query_start", "seq_lens", "positions", "slots"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(out["free_left"]) == want[5]
    st = int(status)
    assert (st in want[6]) if want[6] else st == 0
    return out


@pytest.mark.parametrize("B,bs,ctx_hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 16, 100, 1, 3), (3, 1, 9, 5, 0), (256, 16, 3000, 1, 8),
    (100, 7, 500, 300, 1000), (1024, 32, 300, 9, 5), (1025, 16, 40, 3, 1), (3001, 64, 200, 40, 9)])
def test_plan(B, bs, ctx_hi, new_hi, pad):
    ctx, new, free, tables, pool = _plan_case(B, bs, ctx_hi, new_hi, seed=B + bs)
    T = int(new.sum()) + pad
    if T == 0:
        T = 1
    _run_plan(ctx, new, free, len(free), tables, T, bs, pool)
    # fewer valid free blocks than entries, and a base for the positions
    need = int((-(-(ctx + new) // bs) - -(-ctx // bs)).sum())
    _run_plan(ctx, new, free, need, tables, T, bs, pool, base=1234567)


def test_plan_without_requests_and_all_idle():
    _run_plan(np.zeros(0, int), np.zeros(0, int), np.arange(4), 3, np.zeros((0, 2), np.int32), 5,
              16, 10)
    _run_plan(np.array([5, 0, 16]), np.zeros(3, int), np.arange(4), 4,
              np.array([[8, -1], [-1, -1], [9, -1]], np.int32), 2, 16, 10)


@pytest.mark.parametrize("limit", ["blocks", "rows"])
@pytest.mark.parametrize("B", [9, 1500, 2600])
def test_plan_admits_in_order_until_something_runs_out(B, limit):
    ctx, new, free, tables, pool = _plan_case(B, 16, 200, 60, seed=B)
    T, count = int(new.sum()) + 4, len(free)
    if limit == "blocks":
        count = int((-(-(ctx + new) // 16) - -(-ctx // 16)).sum()) // 2
    else:
        T = int(new.sum()) // 2
    out = _run_plan(ctx, new, free, count, tables, T, 16, pool)
    assert int(out["query_start"][-1]) < int(new.sum())
    # nothing fits at all
    _run_plan(ctx, new + 1, free, 0, tables * 0 + 1, T, 16, pool)


def test_plan_bad_lengths_and_ids():
    ctx, new, free, tables, pool = _plan_case(40, 16, 200, 60, seed=3)
    ctx[3], new[7], new[11] = -5, -1, 10 ** 6
    _run_plan(ctx, new, free, len(free), tables, int(np.abs(new).sum()), 16, pool)
    ctx, new, free, tables, pool = _plan_case(40, 16, 200, 60, seed=3)
    free[-2] = pool
    tables[5] = -3
    _run_plan(ctx, new, free, len(free), tables, int(new.sum()) + 1, 16, pool)
    # a count outside the list counts as none
    for count in (-1, len(free) + 1):
        _run_plan(ctx, new, free, count, tables, int(new.sum()) + 1, 16, pool)


def test_plan_slots_past_32_bits():
    tables = np.array([[2 ** 27 + 5, -1]], dtype=np.int32)
    out = _run_plan(np.array([3]), np.array([61]), np.array([2 ** 27 + 9]), 1, tables, 61, 32,
                    2 ** 28)
    assert int(out["slots"].max()) > 2 ** 31


# ------------------------------------------------- norm, rotation, cache write

def _cos_sin(rot, n=300, far=0):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = (torch.arange(n, dtype=torch.float64) + far)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _rope_check(got, ref, dtype):
    # float32 products and a sum of squares of D terms: relative 16 * 2^-24 of
    # the row's largest value covers norm, weight and rotation; one rounding
    got = got.double().cpu()
    bound = sr.HALF_STEP[dtype] * ref.abs() + (1 + sr.HALF_STEP[dtype]) * 16 * 2.0 ** -24 * \
        ref.abs().amax(-1, keepdim=True)
    if dtype == F16:
        bound = bound + 2.0 ** -25    # half a subnormal step
    assert (got - ref).abs().le(bound).all()


@pytest.mark.parametrize("dtype,T,hq,hkv,d,rot,bs,inter,sx,norm", [
    (BF16, 1, 24, 4, 256, 256, 16, False, False, True),
    (BF16, 33, 32, 8, 128, 128, 32, False, False, True),
    (F16, 70, 6, 1, 64, 32, 16, True, False, True),
    (F16, 19, 16, 2, 128, 64, 16, True, True, True),
    (BF16, 45, 5, 5, 64, 64, 7, False, True, False),
    (F32, 29, 3, 1, 64, 48, 8, False, False, True),
    (F32, 29, 4, 2, 256, 256, 16, True, True, True),
    (F32, 40, 7, 7, 128, 16, 16, False, True, True),
    (BF16, 500, 9, 3, 256, 112, 16, False, False, True),
    (BF16, 12, 8, 2, 128, 0, 16, False, False, True),
])
def test_qk_norm_rope(dtype, T, hq, hkv, d, rot, bs, inter, sx, norm):
    g = torch.Generator().manual_seed(T + d)
    qkv = (3 * torch.randn(T, hq + 2 * hkv, d, generator=g)).to(dtype)
    wq = torch.randn(d, generator=g).to(dtype) if norm else None
    wk = torch.randn(d, generator=g).to(dtype) if norm else None
    nb = -(-T // bs) + 3
    kc = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
    vc = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[T // 2::7] = -1                                  # padding rows in between
    live = slots >= 0
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    cs = _cos_sin(rot, far=100000) if rot else None
    offset = 1.0 if T % 2 else 0.0
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    rq = sr.norm_rope(q, wq, cs, pos, 1e-5, offset, inter)
    rk = sr.norm_rope(k, wk, cs, pos, 1e-5, offset, inter)

    dev = lambda t: None if t is None else t.cuda()
    gkv = qkv.cuda()                                       # strided slices of one projection
    gk5, gv4 = [t.cuda() for t in (sr.split_x(kc, vc) if sx else (kc, vc))]
    fill = -77.0
    q_out, k_out, v_out = [torch.full((T, h, d), fill, dtype=dtype, device="cuda")
                           for h in (hq, hkv, hkv)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.qk_norm_rope(gkv[:, :hq], gkv[:, hq:hq + hkv], gkv[:, hq + hkv:], pos.cuda(), slots.cuda(),
                    dev(cs), q_out, gk5, gv4, q_weight=dev(wq), k_weight=dev(wk), eps=1e-5,
                    weight_offset=offset, interleaved=inter, k_out=k_out, v_out=v_out, split_x=sx,
                    status=status)
    assert int(status) == 0
    assert torch.equal(gkv.cpu(), qkv)
    _rope_check(q_out[live.cuda()], rq[live], dtype)
    _rope_check(k_out[live.cuda()], rk[live], dtype)
    assert torch.equal(v_out.cpu()[live], v[live])
    for t in (q_out, k_out, v_out):
        assert (t[~live.cuda()] == fill).all()             # padding rows are left alone
    # the caches hold the same bits at the slots, and what they held elsewhere
    ek, ev = kc.clone(), vc.clone()
    s = slots[live]
    ek[s // bs, :, s % bs] = k_out.cpu()[live]
    ev[s // bs, :, s % bs] = v[live]
    if sx:
        ek, ev = sr.split_x(ek, ev)
    assert torch.equal(gk5.cpu(), ek) and torch.equal(gv4.cpu(), ev)
    # in place, without caches or dense keys
    qc = gkv[:, :hq].contiguous()
    kk = gkv[:, hq:hq + hkv].contiguous()
    pa.qk_norm_rope(qc, kk, gkv[:, hq + hkv:], pos.cuda(), slots.cuda(), dev(cs), qc,
                    q_weight=dev(wq), k_weight=dev(wk), eps=1e-5, weight_offset=offset,
                    interleaved=inter, k_out=kk)
    assert torch.equal(qc[live.cuda()], q_out[live.cuda()])
    assert torch.equal(kk[live.cuda()], k_out[live.cuda()])


def test_qk_norm_rope_bad_slots_and_positions():
    T, hq, hkv, d, bs, nb = 12, 4, 2, 128, 16, 3
    g = torch.Generator().manual_seed(1)
    q, k, v = [torch.randn(T, h, d, generator=g).to(BF16).cuda() for h in (hq, hkv, hkv)]
    kc = torch.zeros(nb, hkv, bs, d, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    cs = _cos_sin(d).cuda()
    for bad, code in (("slot", pa.PA_ERR_BAD_SLOT), ("position", pa.PA_ERR_BAD_POSITION)):
        slots = torch.arange(T, dtype=torch.int64)
        pos = torch.arange(T, dtype=torch.int32)
        if bad == "slot":
            slots[2], slots[5], slots[7] = nb * bs, -2, 2 ** 40
            rows = [2, 5, 7]
        else:
            pos[3], pos[9] = -1, 300
            rows = [3, 9]
        kc.zero_(), vc.zero_()
        q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.qk_norm_rope(q, k, v, pos.cuda(), slots.cuda(), cs, q_out, kc, vc, k_out=k_out,
                        status=status)
        assert int(status) == code
        ok = torch.ones(T, dtype=torch.bool)
        ok[rows] = False
        assert torch.isfinite(q_out[ok.cuda()]).all()
        assert torch.isnan(q_out[~ok.cuda()]).all().item() == (bad == "position")
        assert torch.isnan(k_out[~ok.cuda()]).all().item() == (bad == "position")
        flat = kc.permute(0, 2, 1, 3).reshape(nb * bs, hkv, d)
        assert torch.equal(flat[:T][ok.cuda()], k_out[ok.cuda()])
        assert (flat[:T][~ok.cuda()] == 0).all() and (flat[T:] == 0).all()


# ---------------------------------------------------------------- window decode

def _edges(window, sinks, bs):
    """Lengths around everything that changes: nothing, one token, the sinks,
    the window, block boundaries, and far beyond."""
    base = [0, 1, 2, sinks, sinks + 1, window - 1, window, window + 1, window + sinks,
            window + sinks + 1, window + bs, window + sinks + 2 * bs + 1, window + 5 * bs - 1,
            window + 997, window + 2048]
    return [max(0, x) for x in base]


def _run_window(q, pg, tables, lens, window, sinks, out_dtype=F32, portable=False, sx=False,
                P=512, flags=0, check=True, max_len=None):
    kc, vc = [t.cuda() for t in (sr.split_x(pg.k, pg.v) if sx else (pg.k, pg.v))]
    gq, gt, gl = q.cuda(), tables.cuda(), lens.cuda()
    n = q.numel()
    whole, flat = _guarded(n, out_dtype, GUARD_F, "cuda")
    out = flat.view(q.shape)
    out.fill_(float("nan"))
    max_len = max_len or max(1, int(lens.max()))
    ws = pa.alloc_window_workspace(gq, kc, gt, window=window, num_sinks=sinks, max_seq_len=max_len,
                                   partition_size=P, split_x=sx)
    ws[1024:] = 255                                         # NaN: nothing stale may be read
    pa.decode_window(gq, kc, vc, gt, gl, out, ws, window=window, num_sinks=sinks,
                     max_seq_len=max_len, scale=q.shape[2] ** -0.5, partition_size=P,
                     portable=portable, split_x=sx, flags=flags)
    torch.cuda.synchronize()
    assert _guards_intact(whole, n, GUARD_F)
    if check:
        assert pa.read_device_status(ws) == pa.PA_OK
        again = torch.empty_like(out)
        pa.decode_window(gq, kc, vc, gt, gl, again, ws, window=window, num_sinks=sinks,
                         max_seq_len=max_len, scale=q.shape[2] ** -0.5, partition_size=P,
                         portable=portable, split_x=sx, flags=flags)
        assert torch.equal(again, out)                      # the same bits again
    return (out, ws) if not check else out


@pytest.mark.parametrize("dtype,hq,hkv,d,bs,window,sinks,P", [
    (BF16, 24, 4, 256, 16, 300, 4, 512),
    (BF16, 8, 1, 128, 32, 64, 16, 32),
    (F16, 6, 2, 128, 64, 1000, 0, 256),
    (F16, 4, 4, 256, 32, 1, 0, 128),
    (BF16, 16, 2, 128, 16, 17, 65, 64),
    (BF16, 18, 2, 128, 16, 130, 3, 512),
    (F16, 8, 8, 64, 16, 200, 5, 64),
    (F32, 4, 2, 64, 8, 77, 9, 40),
    (F32, 6, 3, 256, 16, 260, 1, 512),
    (BF16, 4, 2, 128, 7, 50, 10, 70),
])
def test_decode_window(dtype, hq, hkv, d, bs, window, sinks, P):
    lens = _edges(window, sinks, bs)
    q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, window, sinks, hq, hkv, d, bs,
                                                           dtype, seed=d + window)
    for kw in (dict(), dict(portable=True), dict(sx=True)):
        got = _run_window(q, pg, tables, gl, window, sinks, P=P, **kw)
        sr.assert_within(got, ref, mag, dtype, F32, False, str(kw))
        assert (got[0] == 0).all()                          # length 0: a row of zeros
    if dtype != F32:
        got = _run_window(q, pg, tables, gl, window, sinks, P=P, out_dtype=dtype)
        sr.assert_within(got, ref, mag, dtype, dtype, False, "16-bit out")


@pytest.mark.parametrize("B,L,window,sinks", [(1, 5000, 4096, 4), (1, 900, 700, 0),
                                              (3, 3000, 2048, 100), (40, 700, 512, 1)])
def test_decode_window_batches(B, L, window, sinks):
    r = np.random.RandomState(B)
    lens = [L] + [int(x) for x in r.randint(1, L, size=B - 1)]
    q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, window, sinks, 24, 4, 256, 16,
                                                           BF16, seed=B)
    got = _run_window(q, pg, tables, gl, window, sinks, P=128)
    sr.assert_within(got, ref, mag, BF16, F32, False)
    got = _run_window(q, pg, tables, gl, window, sinks, P=512)
    sr.assert_within(got, ref, mag, BF16, F32, False)


def test_decode_window_wider_than_everything_is_decode():
    """A window or sinks that cover the sequence: pa_decode's result."""
    lens = [1, 200, 513, 1111]
    q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, 2000, 0, 8, 2, 128, 16, BF16, 5)
    for window, sinks in ((2 ** 31 - 1, 2 ** 31 - 1), (1111, 0), (1, 1111), (5000, 3)):
        got = _run_window(q, pg, tables, gl, window, sinks)
        sr.assert_within(got, ref, mag, BF16, F32, False, f"{window} {sinks}")


def test_decode_window_bad_inputs():
    lens = [700, 300, 500, 400]
    for kw in (dict(), dict(portable=True)):
        q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, 200, 20, 8, 2, 128, 16, BF16,
                                                               6)
        tables[0, 0] = 10 ** 6                              # a sink block
        tables[1, 299 // 16] = -1                           # the last window block
        tables[2, 10] = 10 ** 6                             # between: not read
        out, ws = _run_window(q, pg, tables, gl, 200, 20, check=False, **kw)
        assert torch.isnan(out[:2]).all()
        sr.assert_within(out[2:], ref[2:], mag[2:], BF16, F32, False)
        assert pa.read_device_status(ws) == pa.PA_ERR_BAD_BLOCK_ID
        q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, 200, 20, 8, 2, 128, 16, BF16,
                                                               6)
        gl[1], gl[3] = -1, 701
        out, ws = _run_window(q, pg, tables, gl, 200, 20, check=False, max_len=700, **kw)
        assert torch.isnan(out[1]).all() and torch.isnan(out[3]).all()
        sr.assert_within(out[[0, 2]], ref[[0, 2]], mag[[0, 2]], BF16, F32, False)
        assert pa.read_device_status(ws) == pa.PA_ERR_BAD_SEQ_LEN


# ---------------------------------------------------------------- window prefill

def _run_window_prefill(p, window, sinks, out_dtype=F32, portable=False, sx=False, flags=0,
                        max_ctx=None, max_new=None, fill=float("nan")):
    q, k, v, pg, tables, start, ctx = p[:7]
    kc, vc = [t.cuda() for t in (sr.split_x(pg.k, pg.v) if sx else (pg.k, pg.v))]
    n = q.numel()
    whole, flat = _guarded(n, out_dtype, GUARD_F, "cuda")
    out = flat.view(q.shape)
    out.fill_(fill)
    pa.prefill_window(q.cuda(), k.cuda(), v.cuda(), kc, vc, tables.cuda(), start.cuda(),
                      ctx.cuda(), out, window=window, num_sinks=sinks,
                      max_query_len=max_new or int((start[1:] - start[:-1]).max()),
                      max_ctx_len=int(ctx.max()) if max_ctx is None else max_ctx,
                      scale=q.shape[2] ** -0.5, portable=portable, split_x=sx, flags=flags)
    torch.cuda.synchronize()
    assert _guards_intact(whole, n, GUARD_F)
    return out


@pytest.mark.parametrize("dtype,ctx,new,hq,hkv,d,bs,window,sinks", [
    (BF16, (0, 300, 700), (200, 129, 37), 24, 4, 256, 16, 150, 4),
    (F16, (130, 0, 1000), (60, 150, 1), 8, 8, 128, 32, 64, 0),
    (BF16, (64, 777), (1, 129), 16, 2, 128, 64, 200, 70),
    (BF16, (600,), (213,), 5, 1, 256, 32, 1, 1),
    (F16, (17, 247, 5), (27, 0, 185), 6, 2, 256, 16, 31, 130),
    (BF16, (1300, 900), (70, 300), 12, 1, 128, 16, 333, 17),
    (BF16, (50,), (100,), 4, 2, 128, 16, 4000, 0),
    (F32, (40, 0), (30, 20), 4, 2, 64, 8, 33, 5),
    (F16, (90,), (40,), 9, 1, 128, 7, 21, 3),
])
def test_prefill_window(dtype, ctx, new, hq, hkv, d, bs, window, sinks):
    p = sr.window_prefill_problem(ctx, new, window, sinks, hq, hkv, d, bs, dtype, seed=d + window)
    ref, mag = p[7:]
    got = _run_window_prefill(p, window, sinks)
    sr.assert_within(got, ref, mag, dtype, F32, True)
    assert torch.equal(_run_window_prefill(p, window, sinks), got)
    for kw in (dict(portable=True), dict(sx=True)):
        sr.assert_within(_run_window_prefill(p, window, sinks, **kw), ref, mag, dtype, F32, False,
                         str(kw))
    if dtype != F32:
        got = _run_window_prefill(p, window, sinks, out_dtype=dtype)
        sr.assert_within(got, ref, mag, dtype, dtype, True, "16-bit out")


def test_prefill_window_of_one_token_is_decode_window():
    """A chunk of one token, its key and value also in the cache: decode's row."""
    C, hq, hkv, d, bs, window, sinks = 900, 8, 2, 128, 16, 250, 6
    p = sr.window_prefill_problem((C,), (1,), window, sinks, hq, hkv, d, bs, BF16, seed=9)
    q, k, v, pg, tables, start, ctx, ref, mag = p
    got = _run_window_prefill(p, window, sinks)
    wide = torch.full((1, C // bs + 1), -1, dtype=torch.int32)
    wide[:, :tables.shape[1]] = tables
    if wide[0, C // bs] < 0:
        wide[0, C // bs] = pg.order.pop()
    pg.k[wide[0, C // bs], :, C % bs] = k[0]
    pg.v[wide[0, C // bs], :, C % bs] = v[0]
    dec = _run_window(q, pg, wide, torch.tensor([C + 1], dtype=torch.int32), window, sinks)
    sr.assert_within(got, ref, mag, BF16, F32, True)
    sr.assert_within(dec, ref, mag, BF16, F32, False)


def test_prefill_window_bad_inputs():
    ctx, new = (300, 200, 100, 50), (40, 30, 20, 10)
    for kw in (dict(), dict(portable=True)):
        p = list(sr.window_prefill_problem(ctx, new, 120, 8, 4, 2, 128, 16, BF16, seed=21))
        ref, mag = p[7:]
        s = [int(x) for x in p[5]]
        p[4] = p[4].clone()
        p[4][0, 290 // 16] = -3                             # seen by sequence 0
        p[4][2, 2] = p[4][2, 2]
        p[6] = p[6].clone()
        p[6][1] = 301                                       # past the promised bound
        got = _run_window_prefill(p, 120, 8, max_ctx=300, fill=7.0, **kw)
        assert torch.isnan(got[s[0]:s[1]]).all() and torch.isnan(got[s[1]:s[2]]).all()
        sr.assert_within(got[s[2]:], ref[s[2]:], mag[s[2]:], BF16, F32, True)
        # a chunk longer than max_query_len is left alone
        p = sr.window_prefill_problem(ctx, new, 120, 8, 4, 2, 128, 16, BF16, seed=21)
        got = _run_window_prefill(p, 120, 8, max_new=35, fill=7.0, **kw)
        assert (got[:s[1]] == 7.0).all()
        sr.assert_within(got[s[1]:], ref[s[1]:], mag[s[1]:], BF16, F32, True)


# ---------------------------------------------------------------- shared prefix

def _run_prefix(p, prefix, out_dtype=F32, portable=False, sx=False, P=512, flags=0, max_prefix=None,
                max_len=None, check=True):
    q, pg, shared, tables, lens = p[:5]
    kc, vc = [t.cuda() for t in (sr.split_x(pg.k, pg.v) if sx else (pg.k, pg.v))]
    n = q.numel()
    whole, flat = _guarded(n, out_dtype, GUARD_F, "cuda")
    out = flat.view(q.shape)
    out.fill_(float("nan"))
    gq, gt = q.cuda(), tables.cuda()
    max_len = int(lens.max()) if max_len is None else max_len
    max_prefix = prefix if max_prefix is None else max_prefix
    ws = pa.alloc_prefix_workspace(gq, kc, gt, max_seq_len=max_len, max_prefix_len=max_prefix,
                                   partition_size=P, split_x=sx)
    ws[1024:] = 255
    call = lambda o: pa.decode_prefix(
        gq, kc, vc, shared.cuda(), i32([prefix]), gt, lens.cuda(), o, ws, max_seq_len=max_len,
        max_prefix_len=max_prefix, scale=q.shape[2] ** -0.5, partition_size=P, portable=portable,
        split_x=sx, flags=flags)
    call(out)
    torch.cuda.synchronize()
    assert _guards_intact(whole, n, GUARD_F)
    if not check:
        return out, ws
    assert pa.read_device_status(ws) == pa.PA_OK
    again = torch.empty_like(out)
    call(again)
    assert torch.equal(again, out)
    return out


@pytest.mark.parametrize("dtype,prefix,lens,hq,hkv,d,bs,P", [
    (BF16, 1000, (1, 0, 37, 300), 24, 4, 256, 16, 512),
    (BF16, 1, (5, 16, 17), 8, 2, 128, 16, 64),
    (F16, 129, (0, 0), 4, 4, 128, 32, 128),
    (BF16, 128, (700, 3), 16, 2, 128, 64, 512),
    (BF16, 2500, tuple(range(0, 66)), 32, 8, 128, 32, 128),
    (F16, 777, tuple(range(1, 40)), 7, 1, 256, 32, 64),
    (F16, 300, (9,), 40, 1, 128, 16, 64),
    (BF16, 0, (0, 20, 400), 8, 2, 128, 16, 512),
    (BF16, 5000, (2,), 6, 6, 128, 16, 512),
    (F32, 200, (0, 9, 100), 4, 2, 64, 8, 40),
    (F16, 260, (30, 2), 6, 3, 64, 16, 64),
])
def test_decode_prefix(dtype, prefix, lens, hq, hkv, d, bs, P):
    p = sr.prefix_problem(prefix, lens, hq, hkv, d, bs, dtype, seed=prefix + d)
    ref, mag = p[5:]
    got = _run_prefix(p, prefix, P=P)
    sr.assert_within(got, ref, mag, dtype, F32, True)
    # promised bounds that are wider than what is there
    got = _run_prefix(p, prefix, P=P, max_prefix=p[2].shape[0] * bs,
                      max_len=p[3].shape[1] * bs)
    sr.assert_within(got, ref, mag, dtype, F32, True, "wider bounds")
    for kw in (dict(portable=True), dict(sx=True)):
        sr.assert_within(_run_prefix(p, prefix, P=P, **kw), ref, mag, dtype, F32, False, str(kw))
    if dtype != F32:
        got = _run_prefix(p, prefix, P=P, out_dtype=dtype)
        sr.assert_within(got, ref, mag, dtype, dtype, True, "16-bit out")
    for b, L in enumerate(lens):
        if L == 0 and prefix == 0:
            assert (got[b] == 0).all()


def test_decode_prefix_bad_inputs():
    for kw in (dict(), dict(portable=True)):
        p = sr.prefix_problem(400, (30, 5, 60), 8, 2, 128, 16, BF16, seed=2)
        ref, mag = p[5:]
        p[3][1, 0] = -1                                     # one sequence's own block
        out, ws = _run_prefix(p, 400, check=False, **kw)
        assert torch.isnan(out[1]).all()
        sr.assert_within(out[[0, 2]], ref[[0, 2]], mag[[0, 2]], BF16, F32, True)
        assert pa.read_device_status(ws) == pa.PA_ERR_BAD_BLOCK_ID
        p = sr.prefix_problem(400, (30, 5, 60), 8, 2, 128, 16, BF16, seed=2)
        p[2][7] = 10 ** 6                                   # a prefix block: everyone
        out, ws = _run_prefix(p, 400, check=False, **kw)
        assert torch.isnan(out).all()
        assert pa.read_device_status(ws) == pa.PA_ERR_BAD_BLOCK_ID
        p = sr.prefix_problem(400, (30, 5, 60), 8, 2, 128, 16, BF16, seed=2)
        for n in (-1, 401):
            out, ws = _run_prefix(p, n, max_prefix=400, check=False, **kw)
            assert torch.isnan(out).all()
            assert pa.read_device_status(ws) == pa.PA_ERR_BAD_SEQ_LEN
        p[4][2] = 61
        out, ws = _run_prefix(p, 400, max_len=60, check=False, **kw)
        assert torch.isnan(out[2]).all()
        sr.assert_within(out[:2], ref[:2], mag[:2], BF16, F32, True)


def test_decode_prefix_many_short_sequences():
    """Many sequences with short own lists: the kernel that joins as it goes,
    at both head_dims, with and without a prefix, and its bad inputs."""
    for hq, hkv, d, bs, dtype, prefix in ((24, 4, 256, 16, BF16, 500), (7, 4, 128, 64, F16, 131),
                                          (32, 8, 128, 32, BF16, 0)):
        hq = hq if hq % hkv == 0 else hkv * 3
        lens = [int(x) for x in np.random.RandomState(d).randint(0, 100, size=41)]
        p = sr.prefix_problem(prefix, lens, hq, hkv, d, bs, dtype, seed=11)
        ref, mag = p[5:]
        got = _run_prefix(p, prefix)
        sr.assert_within(got, ref, mag, dtype, F32, True)
        got = _run_prefix(p, prefix, out_dtype=dtype)
        sr.assert_within(got, ref, mag, dtype, dtype, True)
        bad = next(i for i, n in enumerate(lens) if n > 20)
        p[3][bad, 0] = 10 ** 6
        p[4][40] = 101
        out, ws = _run_prefix(p, prefix, max_len=100, check=False)
        good = [i for i in range(40) if i != bad]
        assert torch.isnan(out[bad]).all() and torch.isnan(out[40]).all()
        sr.assert_within(out[good], ref[good], mag[good], dtype, F32, True)
        assert pa.read_device_status(ws) in (pa.PA_ERR_BAD_BLOCK_ID, pa.PA_ERR_BAD_SEQ_LEN)


# ------------------------------------------------------- what is easily missed

@pytest.mark.parametrize("hq,hkv,d,bs", [(6, 1, 128, 16), (4, 2, 256, 32)])
def test_prefill_window_wide_is_prefill(hq, hkv, d, bs):
    """A window wider than the sequences: the plain prefill's result."""
    p = sr.window_prefill_problem((200, 0, 33), (70, 150, 1), 10 ** 6, 0, hq, hkv, d, bs, BF16, 3)
    q, k, v, pg, tables, start, ctx, ref, mag = p
    got = _run_window_prefill(p, 10 ** 6, 0)
    out = torch.empty(q.shape, device="cuda")
    pa.prefill(q.cuda(), k.cuda(), v.cuda(), pg.k.cuda(), pg.v.cuda(), tables.cuda(), start.cuda(),
               ctx.cuda(), out, max_query_len=150, max_ctx_len=200, scale=d ** -0.5)
    sr.assert_within(got, ref, mag, BF16, F32, True)
    sr.assert_within(out, ref, mag, BF16, F32, True)


@pytest.mark.parametrize("B,hi", [(70, 40), (2100, 3)])
def test_prefill_window_many_sequences(B, hi):
    r = np.random.RandomState(B)
    ctx = [int(x) for x in r.randint(0, 20, size=B)]
    new = [int(x) for x in r.randint(0, hi, size=B)]
    p = sr.window_prefill_problem(ctx, new, 9, 2, 2, 1, 128, 16, BF16, seed=B)
    sr.assert_within(_run_window_prefill(p, 9, 2), p[7], p[8], BF16, F32, True)


def test_prefill_window_output_on_16_bytes():
    p = sr.window_prefill_problem((100,), (50,), 60, 4, 4, 2, 128, 16, BF16, seed=5)
    q, k, v, pg, tables, start, ctx, ref, mag = p
    flat = torch.zeros(q.numel() + 8, dtype=BF16, device="cuda")
    out = flat[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    pa.prefill_window(q.cuda(), k.cuda(), v.cuda(), pg.k.cuda(), pg.v.cuda(), tables.cuda(),
                      start.cuda(), ctx.cuda(), out, window=60, num_sinks=4, max_query_len=50,
                      max_ctx_len=100, scale=128 ** -0.5)
    sr.assert_within(out, ref, mag, BF16, BF16, True)
    assert (flat[:8] == 0).all()


def test_waits_that_run_out():
    """The diagnostic flag makes a wait of the tensor-core kernels run out: NaN
    and the status, and the next call is right."""
    stall = pa.PA_FLAG_SELFTEST_STALL
    for d in (128, 256):
        p = sr.window_prefill_problem((100,), (50,), 60, 4, 4, 2, d, 16, BF16, seed=5)
        assert torch.isnan(_run_window_prefill(p, 60, 4, flags=stall)).all()
        sr.assert_within(_run_window_prefill(p, 60, 4), p[7], p[8], BF16, F32, True)
        p = sr.prefix_problem(300, (5, 40), 4, 2, d, 16, BF16, seed=6)
        out, ws = _run_prefix(p, 300, flags=stall, check=False)
        assert torch.isnan(out).all()
        assert pa.read_device_status(ws) == pa.PA_ERR_DEVICE_TIMEOUT
        sr.assert_within(_run_prefix(p, 300), p[5], p[6], BF16, F32, True)
        q, pg, tables, gl, ref, mag = sr.window_decode_problem([700, 90], 300, 4, 4, 2, d, 16, BF16,
                                                               seed=7)
        out, ws = _run_window(q, pg, tables, gl, 300, 4, flags=stall, check=False)
        assert torch.isnan(out).all()
        assert pa.read_device_status(ws) == pa.PA_ERR_DEVICE_TIMEOUT
        sr.assert_within(_run_window(q, pg, tables, gl, 300, 4), ref, mag, BF16, F32, False)


def test_caches_past_32_bit_offsets():
    """Blocks whose elements lie past 2^31 in the pool, for every reader and
    for the writer."""
    hq, hkv, d, bs = 4, 4, 256, 16
    blocks = 2 ** 31 // (hkv * bs * d) + 64
    big_k = torch.empty(blocks, hkv, bs, d, dtype=BF16, device="cuda")
    big_v = torch.empty_like(big_k)
    far = blocks - 60                                       # small problems' blocks go here

    def place(pg, *tables):
        n = pg.k.shape[0]
        assert n < 60
        big_k[far:far + n], big_v[far:far + n] = pg.k.cuda(), pg.v.cuda()
        return [torch.where(t >= 0, t + far, t).cuda() for t in tables]

    q, pg, tables, gl, ref, mag = sr.window_decode_problem([300, 77], 100, 20, hq, hkv, d, bs, BF16,
                                                           1)
    gt, = place(pg, tables)
    out = torch.empty(q.shape, device="cuda")
    for portable in (False, True):
        ws = pa.alloc_window_workspace(q.cuda(), big_k, gt, window=100, num_sinks=20,
                                       max_seq_len=300)
        pa.decode_window(q.cuda(), big_k, big_v, gt, gl.cuda(), out, ws, window=100, num_sinks=20,
                         max_seq_len=300, scale=d ** -0.5, portable=portable)
        sr.assert_within(out, ref, mag, BF16, F32, False)
    p = sr.window_prefill_problem((150,), (40,), 70, 3, hq, hkv, d, bs, BF16, 2)
    gt, = place(p[3], p[4])
    out = torch.empty(p[0].shape, device="cuda")
    for portable in (False, True):
        pa.prefill_window(p[0].cuda(), p[1].cuda(), p[2].cuda(), big_k, big_v, gt, p[5].cuda(),
                          p[6].cuda(), out, window=70, num_sinks=3, max_query_len=40,
                          max_ctx_len=150, scale=d ** -0.5, portable=portable)
        sr.assert_within(out, p[7], p[8], BF16, F32, not portable)
    p = sr.prefix_problem(120, [3] * 40, hq, hkv, d, bs, BF16, 3)
    gs, gt = place(p[1], p[2], p[3])
    out = torch.empty(p[0].shape, device="cuda")
    for portable in (False, True):
        ws = pa.alloc_prefix_workspace(p[0].cuda(), big_k, gt, max_seq_len=3, max_prefix_len=120)
        pa.decode_prefix(p[0].cuda(), big_k, big_v, gs, i32([120]), gt, p[4].cuda(), out, ws,
                         max_seq_len=3, max_prefix_len=120, scale=d ** -0.5, portable=portable)
        sr.assert_within(out, p[5], p[6], BF16, F32, not portable)
    T = 20
    x = torch.randn(T, 3 * hq, d, device="cuda").to(BF16)
    slots = far * bs + torch.arange(T, device="cuda") * 3
    q_out = torch.empty(T, hq, d, dtype=BF16, device="cuda")
    pa.qk_norm_rope(x[:, :hq], x[:, hq:2 * hq], x[:, 2 * hq:], None, slots, None, q_out, big_k,
                    big_v)
    assert torch.equal(big_k[slots // bs, :, slots % bs], x[:, hq:2 * hq])
    assert torch.equal(big_v[slots // bs, :, slots % bs], x[:, 2 * hq:])


def test_nothing_to_do():
    """Empty batches, lists and chunks."""
    q, pg, tables, gl, ref, mag = sr.window_decode_problem([0, 0], 5, 2, 4, 2, 128, 16, BF16, 1)
    out = _run_window(q, pg, tables, gl, 5, 2)
    assert (out == 0).all()
    e = torch.empty(0, 4, 128, dtype=BF16, device="cuda")
    kc, vc = pg.k.cuda(), pg.v.cuda()
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    bt, sl = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([])
    pa.decode_window(e, kc, vc, bt, sl, e.clone(), ws, window=5, max_seq_len=9, scale=1.0)
    pa.decode_prefix(e, kc, vc, i32([0]), i32([3]), bt, sl, e.clone(), ws, max_seq_len=9,
                     max_prefix_len=16, scale=1.0)
    z = torch.empty(0, 2, 128, dtype=BF16, device="cuda")
    pa.prefill_window(e, z, z, kc, vc, torch.zeros(1, 3, dtype=torch.int32, device="cuda"),
                      i32([0, 0]), i32([0]), e.clone(), window=5, max_query_len=4, max_ctx_len=0,
                      scale=1.0)
    pa.qk_norm_rope(e, z, z, None, torch.zeros(0, dtype=torch.int64, device="cuda"), None,
                    e.clone())


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    probs = [sr.prefix_problem(700 + 100 * i, (30, 5, 60), 8, 2, 128, 16, BF16, seed=20 + i)
             for i in range(2)]
    streams = [torch.cuda.Stream() for _ in probs]
    state = []
    for p in probs:
        q, pg, shared, tables, lens = p[:5]
        g = [t.cuda() for t in (q, pg.k, pg.v, shared, tables, lens)]
        ws = pa.alloc_prefix_workspace(g[0], g[1], g[4], max_seq_len=60,
                                       max_prefix_len=shared.shape[0] * 16)
        state.append((g, ws, torch.empty(q.shape, device="cuda")))
    torch.cuda.synchronize()
    plen = [i32([700]), i32([800])]
    for _ in range(20):
        for (g, ws, out), s, n in zip(state, streams, plen):
            pa.decode_prefix(g[0], g[1], g[2], g[3], n, g[4], g[5], out, ws, max_seq_len=60,
                             max_prefix_len=g[3].shape[0] * 16, scale=128 ** -0.5, stream=s)
    torch.cuda.synchronize()
    for (g, ws, out), p in zip(state, probs):
        sr.assert_within(out, p[5], p[6], BF16, F32, True)


# ---------------------------------------------------------------- a run together

@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 128, 16), (6, 1, 256, 16)])
def test_serving_steps_together(hq, hkv, d, bs):
    """Plan, norm + rotation + write, attention: a prefill chunk and then
    decode steps over a windowed layer, the decode captured and replayed,
    against the whole sequence computed at once."""
    g = torch.Generator().manual_seed(d)
    prompt, steps, window, sinks = [300, 41, 7], 5, 120, 4
    B, eps, scale = len(prompt), 1e-6, d ** -0.5
    total = [n + steps for n in prompt]
    x = [torch.randn(n, hq + 2 * hkv, d, generator=g).to(BF16) for n in total]
    wq, wk = [(1 + 0.1 * torch.randn(d, generator=g)).to(BF16).cuda() for _ in range(2)]
    cs = _cos_sin(d, n=400).cuda()
    width = -(-max(total) // bs) + 1
    pool = B * width + 5
    kc = torch.full((pool, hkv, bs, d), float("nan"), dtype=BF16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = i32(np.random.RandomState(1).permutation(pool))
    counts = [i32([pool]), i32([0])]
    lens = [i32([0] * B), i32([0] * B)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(T):
        return dict(start=i32([0] * (B + 1)), pos=i32([0] * T),
                    slots=torch.zeros(T, dtype=torch.int64, device="cuda"),
                    q=torch.zeros(T, hq, d, dtype=BF16, device="cuda"),
                    k=torch.zeros(T, hkv, d, dtype=BF16, device="cuda"),
                    v=torch.zeros(T, hkv, d, dtype=BF16, device="cuda"),
                    out=torch.zeros(T, hq, d, dtype=BF16, device="cuda"),
                    x=torch.zeros(T, hq + 2 * hkv, d, dtype=BF16, device="cuda"))

    def front(f, new, at):
        pa.plan_step(lens[at], new, free, counts[at], tables, f["start"], lens[1 - at], f["pos"],
                     f["slots"], counts[1 - at], block_size=bs, num_blocks=pool, status=status)
        pa.qk_norm_rope(f["x"][:, :hq], f["x"][:, hq:hq + hkv], f["x"][:, hq + hkv:], f["pos"],
                        f["slots"], cs, f["q"], kc, vc, q_weight=wq, k_weight=wk, eps=eps,
                        k_out=f["k"], v_out=f["v"], status=status)

    # prefill: all prompts in one padded step
    T = sum(prompt) + 9
    f = buffers(T)
    f["x"][:sum(prompt)] = torch.cat([x[b][:n] for b, n in enumerate(prompt)]).cuda()
    front(f, i32(prompt), 0)
    f["out"].fill_(7.0)
    pa.prefill_window(f["q"], f["k"], f["v"], kc, vc, tables, f["start"], lens[0], f["out"],
                      window=window, num_sinks=sinks, max_query_len=max(prompt), max_ctx_len=0,
                      scale=scale)
    assert (f["out"][sum(prompt):] == 7.0).all()
    got = [[o] for o in torch.split(f["out"][:sum(prompt)].cpu(), prompt)]

    # decode: two captured steps (the two sets of buffers), replayed in turn
    one = i32([1] * B)
    d0, d1 = buffers(B), buffers(B)
    ws = pa.alloc_window_workspace(d0["q"], kc, tables, window=window, num_sinks=sinks,
                                   max_seq_len=width * bs)

    def decode(f, at):
        front(f, one, at)
        pa.decode_window(f["q"], kc, vc, tables, lens[1 - at], f["out"], ws, window=window,
                         num_sinks=sinks, max_seq_len=width * bs, scale=scale)

    def feed(f, s):
        f["x"].copy_(torch.stack([x[b][n + s] for b, n in enumerate(prompt)]))

    feed(d1, 0)
    decode(d1, 1)                                           # step 0, eager
    torch.cuda.synchronize()
    for b in range(B):
        got[b].append(d1["out"][b:b + 1].cpu())
    graphs = []
    for f, at in ((d0, 0), (d1, 1)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            decode(f, at)
        graphs.append(gr)
    for s in range(1, steps):
        f = (d0, d1)[(s + 1) % 2]
        feed(f, s)
        graphs[(s + 1) % 2].replay()
        torch.cuda.synchronize()
        for b in range(B):
            got[b].append(f["out"][b:b + 1].cpu())
    assert int(status) == 0 and pa.read_device_status(ws) == pa.PA_OK

    for b, n in enumerate(total):
        pos = torch.arange(n, dtype=torch.int32)
        q = sr.norm_rope(x[b][:, :hq], wq.cpu(), cs.cpu(), pos, eps, 0.0, False).to(BF16)
        k = sr.norm_rope(x[b][:, hq:hq + hkv], wk.cpu(), cs.cpu(), pos, eps, 0.0, False).to(BF16)
        v = x[b][:, hq + hkv:]
        o = torch.cat(got[b]).double()
        for p in range(n):
            see = sr.visible(p, window, sinks)
            ref, mag = sr.rows_attend(q[p], k[see].double(), v[see].double(), scale)
            # q and k may round the other way where the float32 value sits next
            # to a border: one step of bf16 in an element moves a logit by at most
            # 2^-7 |q k| of that element; over D of them sqrt(D) 2^-7 scale is
            # a generous share, well below 0.05
            assert (o[p] - ref).abs().le(0.05 * mag + 2.0 ** -7 * ref.abs() + 1e-3).all()


def test_side_stream_and_shared_prefix_after_plan():
    """decode_prefix on a side stream, tables from plan_step with a base."""
    hq, hkv, d, bs, prefix = 8, 2, 128, 16, 200
    p = sr.prefix_problem(prefix, (17, 1, 33), hq, hkv, d, bs, BF16, seed=4)
    ref, mag = p[5:]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _run_prefix(p, prefix)
    s.synchronize()
    sr.assert_within(got, ref, mag, BF16, F32, True)
    out = _plan_buffers(3, 8)
    gt = p[3].cuda()
    pa.plan_step(p[4].cuda(), i32([1, 1, 1]), i32([0, 1, 2]), i32([3]), torch.cat(
        [gt, torch.full((3, 2), -1, dtype=torch.int32, device="cuda")], 1).contiguous(),
        out["query_start"], out["seq_lens"], out["positions"], out["slots"], out["free_left"],
        block_size=bs, num_blocks=p[1].k.shape[0], base_len=i32([prefix]))
    assert out["positions"].tolist()[:3] == [217, 201, 233]


@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 128, 32), (24, 4, 256, 16), (8, 1, 128, 16)])
def test_one_workspace_for_shrinking_batches(hq, hkv, d, bs):
    """Sequences end and lengths are bounded tighter: the workspace stays."""
    B, window, sinks, prefix = 40, 300, 3, 3000
    r = np.random.RandomState(d)
    lens = [int(x) for x in r.randint(1, 700, size=B)]
    scale = d ** -0.5
    q, pg, tables, gl, ref, mag = sr.window_decode_problem(lens, window, sinks, hq, hkv, d, bs,
                                                           BF16, seed=1)
    dev = [x.cuda() for x in (q, pg.k, pg.v, tables, gl)]
    ws = pa.alloc_window_workspace(dev[0], dev[1], dev[3], window=window, num_sinks=sinks,
                                   max_seq_len=700)
    for n in (40, 33, 32, 16, 15, 4, 3, 1):
        out = torch.empty((n, hq, d), device="cuda")
        pa.decode_window(dev[0][:n], dev[1], dev[2], dev[3][:n], dev[4][:n], out, ws,
                         window=window, num_sinks=sinks, max_seq_len=max(lens[:n]), scale=scale)
        sr.assert_within(out, ref[:n], mag[:n], BF16, F32, False, f"window {n}")
    p = sr.prefix_problem(prefix, lens, hq, hkv, d, bs, BF16, seed=2)
    ref, mag = p[5:]
    gq, kc, vc, shared, tab, gl = [x.cuda() for x in (p[0], p[1].k, p[1].v, *p[2:5])]
    ws = pa.alloc_prefix_workspace(gq, kc, tab, max_seq_len=700, max_prefix_len=prefix)
    for n in (40, 33, 32, 16, 15, 4, 3, 1):
        out = torch.empty((n, hq, d), device="cuda")
        pa.decode_prefix(gq[:n], kc, vc, shared, i32([prefix]), tab[:n], gl[:n], out, ws,
                         max_seq_len=max(lens[:n]), max_prefix_len=prefix, scale=scale)
        sr.assert_within(out, ref[:n], mag[:n], BF16, F32, True, f"prefix {n}")
    assert pa.read_device_status(ws) == pa.PA_OK
