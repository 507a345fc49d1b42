"""Decode over the 4-bit cache where a group's scales differ widely from token to token: the
bounds that the header gives, against the float64 reference."""
import math

import pytest
import torch

import kv4_reference as kr
import paged_attention_decode_v2_gb300 as pa
import step_reference as sr
from test_gpu_kv4 import run_decode

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def large_but_unseen(tokens, large, ratio, d, group, dtype, seed):
    """Token ``large`` has values and steps ``ratio`` times the others', and a key against the
    queries: a weight around 2^-45 of the largest.  Four query heads on one KV head."""
    pool = kr.Pool(-(-tokens // 16) + 2, 1, 16, d, group, dtype, seed)
    base = pool.randn(d).float()
    q = (base + 0.1 * pool.randn(1, 4, d).float()).to(dtype)
    k, v = pool.randn(tokens, 1, d).float(), pool.randn(tokens, 1, d).float()
    k[large, 0] = -32 * math.sqrt(d) * base / (base @ base)
    v[large] *= ratio
    if dtype == F16:
        v *= 2.0 ** -9
    table = torch.tensor([pool.order.pop() for _ in range(-(-tokens // 16))], dtype=torch.int32)
    t = torch.arange(tokens)
    pool.put(table[t // 16].long(), t % 16, k.to(dtype), v.to(dtype))
    return q, pool, table[None]


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128),
                                     (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("dtype,power", [(BF16, 10), (BF16, 16), (BF16, 20), (BF16, 24),
                                         (F16, 10), (F16, 16), (F16, 20)])
@pytest.mark.parametrize("tokens,large", [(20, 0), (20, 19), (300, 40)])
@pytest.mark.parametrize("portable", [False, True])
def test_a_large_token_that_no_query_sees(d, group, dtype, power, tokens, large, portable):
    """The row is the other tokens' mean, to their own steps.  A weight times a scale is rounded
    to float16, half a step 2^-11 of it, or 2^-35 of the largest scale where that is more (the
    weight being at most 1), and multiplies c - 8, at most 8.  The minima meet the weights in two
    parts: bf16 2^-17 of them; f16 2^-22, or 2^-33 of the largest weight.  Logits as in
    assert_decode."""
    q, pool, tables = large_but_unseen(tokens, large, 2.0 ** power, d, group, dtype, d + power)
    k, v, s = pool.rows(tables[0], tokens)
    got = run_decode(q, pool, tables, torch.tensor([tokens]), portable=portable,
                     out_dtype=F32).double().cpu()
    for h in range(4):
        a = (k[:, 0] @ q[0, h].double()) * d ** -0.5
        w = torch.softmax(a, 0)
        assert float(w[large] / w.max()) < 2.0 ** -36
        ref, mag, step = w @ v[:, 0], w @ v[:, 0].abs(), w @ s[:, 0]
        bound = 2e-5 * (mag + 15 * step) + 1e-9
        if not portable:
            bound = bound + 2.0 ** -11 * 8 * step + 2.0 ** -17 * (mag + 15 * step)
            few = tokens * w.max()         # tokens, each with an error beside a weight of 1
            bound = bound + few * 2.0 ** -35 * 8 * s[:, 0].amax(0)
            if dtype == F16:
                bound = bound + few * 2.0 ** -33 * (v[:, 0].abs() + 15 * s[:, 0]).amax(0)
        bound = bound + sr.HALF_STEP[F32] * (ref.abs() + bound)
        bad = (got[0, h] - ref).abs() > bound
        assert not bad.any(), (int(bad.sum()), float(((got[0, h] - ref).abs() / bound).max()))


def test_parts_of_many_pairs_stay_below_the_longest():
    """One row of 2^19 tokens among 4900 short ones and a partition size as large: its parts, whose
    length the kernel leaves in the control block, are at most 2^17 tokens.  The pages are taken
    over and over; a token counts as often as the row has it."""
    d, bs, blocks, n, B = 64, 4096, 4, 1 << 19, 4900
    pool = kr.Pool(blocks, 1, bs, d, 32, BF16, seed=3)
    pages = torch.empty(blocks, dtype=torch.int32)
    pool.fill(pages, blocks * bs)
    q = pool.randn(B, 2, d)
    k, v, s = pool.rows(pages, blocks * bs)
    tables = torch.full((B, n // bs), -1, dtype=torch.int32)
    tables[:, 0] = pages[0]
    tables[5] = pages[torch.arange(n // bs) % blocks]
    lens = torch.ones(B, dtype=torch.int32)
    lens[5] = n
    p = pa.Params(B, 2, 1, d, bs, blocks, n // bs, n, n, 0, pa.PA_BF16, pa.PA_F32, 1.0, 0)
    ws = torch.empty(pa.kv4_workspace_size(p, 32), dtype=torch.uint8, device="cuda")
    pa.workspace_init(ws)
    got = run_decode(q, pool, tables, lens, out_dtype=F32, partition_size=n, workspace=ws)
    assert 0 < int(ws[512:516].view(torch.int32)) <= 1 << 17
    for b in (5, 6, B - 1):
        m = blocks * bs if b == 5 else 1
        for h in range(2):
            w = torch.softmax((k[:m, 0] @ q[b, h].double()) * d ** -0.5, 0)
            kr.assert_decode(got[b, h], w @ v[:m, 0], w @ v[:m, 0].abs(), w @ s[:m, 0], F32, False)


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128),
                                     (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_repeated_runs_are_bit_for_bit_the_same(d, group, dtype):
    """The lanes of a warp hand scales and weights to one another in shared memory, many tiles a
    row, with new references and powers on the way."""
    lens = (1500, 37, 700) * 12
    q, pool, tables, n, *_ = kr.decode_problem(lens, 4, 2, d, 16, group, dtype, 5, spread=3.0)
    first = run_decode(q, pool, tables, n)
    for _ in range(20):
        assert torch.equal(run_decode(q, pool, tables, n), first)


def test_a_range_that_rounds_past_the_type():
    """-65504 to 65504 of f16: s = 8733.9 rounds to 8736, and code 15 stands for 65536."""
    x = torch.zeros(1, 1, 64, dtype=F16)
    x[0, 0, 0], x[0, 0, 1] = 65504.0, -65504.0
    pool = [t.cuda() for t in kr.Pool(1, 1, 16, 64, 64, F16, 1).cuda()]
    k, v = x.cuda(), (x / 2).cuda()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    pa.store_kv4(k, v, torch.zeros(1, dtype=torch.int64, device="cuda"), *pool, k_out=ko, v_out=vo)
    assert pool[2][0, 0, 0, 0].tolist() == [8736.0, -65504.0]
    assert ko[0, 0, 0] == math.inf and ko[0, 0, 1] == -65504.0
    assert torch.isfinite(ko[0, 0, 1:]).all() and torch.isfinite(vo).all()


def test_one_workspace_for_the_16_bit_and_the_4_bit_decode():
    """Both keep their counters in the control block: calls in turn, on one workspace, each as if
    it were alone; items from the queue, and a row reduced in one launch."""
    lens = [1200, 40, 700] * 50
    q, pool, tables, n, *_ = kr.decode_problem(lens, 8, 4, 64, 16, 32, BF16, 8)
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.randn(1300, 4, 16, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    q16 = torch.randn(1, 24, 128, generator=g, device="cuda").to(BF16)
    table = torch.randperm(1300, generator=g, device="cuda")[None, :1250].int()
    n16 = torch.tensor([20000], dtype=torch.int32, device="cuda")
    out16 = torch.empty_like(q16)
    p = pa.make_params(q16, kc, table, max_seq_len=20000, scale=128 ** -0.5, partition_size=512)
    p4 = pa.Params(150, 8, 4, 64, 16, pool.k.shape[0], tables.shape[1], 1200, 1024, 0, pa.PA_BF16,
                   pa.PA_BF16, 1.0, 0)
    ws = torch.empty(max(pa.workspace_size(p), pa.kv4_workspace_size(p4, 32)), dtype=torch.uint8,
                     device="cuda")
    pa.workspace_init(ws)

    def decode16():
        out16.fill_(math.nan)
        pa.decode_v2(q16, kc, vc, table, n16, out16, ws, max_seq_len=20000, scale=128 ** -0.5,
                     partition_size=512)
        return out16.clone()

    alone = run_decode(q, pool, tables, n), decode16()
    assert torch.isfinite(alone[0]).all() and torch.isfinite(alone[1]).all()
    for _ in range(5):
        assert torch.equal(run_decode(q, pool, tables, n, workspace=ws), alone[0])
        assert torch.equal(decode16(), alone[1])
    assert pa.read_device_status(ws) == pa.PA_OK
