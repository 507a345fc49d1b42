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
