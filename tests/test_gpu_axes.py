"""Rotation with several axes on the GPU against a plain float64 reference."""
import math

import pytest
import torch

import paged_attention_decode_v2_gb300 as pa
import step_reference as sr

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def table(rot, n=500):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def reference(x, w, cos_sin, pos, axis_of, eps, offset, interleaved):
    """Pair by pair: each with the position of its axis."""
    y = sr.norm_rope(x, w, None, None, eps, offset, interleaved)
    rot = cos_sin.shape[1]
    out = y.clone()
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
        at = pos[axis_of[j]].long()
        c, s = cos_sin[at, j].double()[:, None], cos_sin[at, rot // 2 + j].double()[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def close(got, ref, dtype):
    """Norm, products and sums in float32 (a few 2^-24 of |a| + |b|, both below 8 here), one
    rounding to the type."""
    err = (got.double().cpu() - ref).abs()
    assert (err <= sr.HALF_STEP[dtype] * ref.abs() + 1e-5).all(), float(err.max())


def problem(T, hq, hkv, d, rot, axes, dtype, seed, blocks=None, bs=16):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(dtype)
    blocks = blocks or -(-max(T, 1) // bs) + 2
    return dict(qkv=rand(T, hq + 2 * hkv, d), wq=1 + 0.1 * rand(d), wk=1 + 0.1 * rand(d),
                pos=torch.randint(0, 500, (axes, T), generator=g, dtype=torch.int32),
                slots=torch.randperm(blocks * bs, generator=g)[:T], cs=table(rot),
                kc=rand(blocks, hkv, bs, d), vc=rand(blocks, hkv, bs, d))


CASES = [
    # T, hq, hkv, d, rot, axis_of, interleaved, split_x, dtype
    (1, 8, 2, 128, 128, pa.rope_axes((16, 24, 24)), False, False, BF16),
    (33, 32, 8, 128, 128, pa.rope_axes((24, 20, 20), True), False, False, BF16),
    (300, 24, 4, 256, 256, pa.rope_axes((128,)), False, False, BF16),
    (77, 24, 4, 256, 128, pa.rope_axes((1, 30, 2, 31)), True, False, F16),
    (65, 16, 2, 128, 64, pa.rope_axes((11, 21)), True, True, F16),
    (40, 3, 3, 64, 64, bytes(j * 7 % 4 for j in range(32)), False, True, BF16),
    (19, 12, 4, 64, 48, bytes(j % 3 for j in range(24)), False, False, F32),
    (513, 6, 1, 256, 256, bytes(j * j % 4 for j in range(128)), True, False, F32),
]


@pytest.mark.parametrize("T,hq,hkv,d,rot,of,inter,sx,dtype", CASES,
                         ids=[f"{c[0]}-{c[3]}-{c[4]}-{max(c[5]) + 1}" for c in CASES])
def test_axes(T, hq, hkv, d, rot, of, inter, sx, dtype):
    axes = max(of) + 1
    p = problem(T, hq, hkv, d, rot, axes, dtype, seed=T)
    if T > 4:
        p["slots"][3] = -1                                   # a padding row
    g = {k: v.cuda() for k, v in p.items()}
    kc, vc = sr.split_x(g["kc"], g["vc"]) if sx else (g["kc"].clone(), g["vc"].clone())
    q_out = torch.full((T, hq, d), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((T, hkv, d), 7.0, dtype=dtype, device="cuda")
    v_out = k_out.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = g["qkv"][:, :hq], g["qkv"][:, hq:hq + hkv], g["qkv"][:, hq + hkv:]
    pa.qk_norm_rope_axes(q, k, v, g["pos"], g["slots"], g["cs"], q_out, kc, vc, axis_of=of,
                         q_weight=g["wq"], k_weight=g["wk"], interleaved=inter, split_x=sx,
                         k_out=k_out, v_out=v_out, status=status)
    assert int(status) == 0
    live = p["slots"] >= 0
    x = p["qkv"]
    want_q = reference(x[:, :hq], p["wq"], p["cs"], p["pos"], of, 1e-6, 0.0, inter)
    want_k = reference(x[:, hq:hq + hkv], p["wk"], p["cs"], p["pos"], of, 1e-6, 0.0, inter)
    close(q_out[live.cuda()], want_q[live], dtype)
    close(k_out[live.cuda()], want_k[live], dtype)
    assert (q_out[~live.cuda()] == 7).all() and (k_out[~live.cuda()] == 7).all()
    assert torch.equal(v_out[live.cuda()].cpu(), x[live, hq + hkv:])
    # the caches hold k_out and v_out at their slots, and what they held elsewhere
    kp, vp = p["kc"].clone(), p["vc"].clone()
    at = p["slots"][live]
    kp[at // 16, :, at % 16] = k_out.cpu()[live]
    vp[at // 16, :, at % 16] = v_out.cpu()[live]
    if sx:
        kp, vp = sr.split_x(kp, vp)
    assert torch.equal(kc.cpu(), kp) and torch.equal(vc.cpu(), vp)


@pytest.mark.parametrize("inter", [False, True])
def test_equal_positions_and_one_axis_are_the_plain_rotation(inter):
    """Text: the same position on every axis gives what qk_norm_rope gives, bit by bit."""
    p = {k: v.cuda() for k, v in problem(50, 8, 2, 128, 128, 3, BF16, seed=1).items()}
    q, k, v = p["qkv"][:, :8], p["qkv"][:, 8:10], p["qkv"][:, 10:]
    kw = dict(q_weight=p["wq"], k_weight=p["wk"], interleaved=inter)
    want = torch.empty(50, 8, 128, dtype=BF16, device="cuda")
    pa.qk_norm_rope(q, k, v, p["pos"][1].contiguous(), p["slots"], p["cs"], want, p["kc"],
                    p["vc"], **kw)
    for pos, of in ((p["pos"][1:2], bytes(64)),
                    (p["pos"][1:2].expand(3, -1).contiguous(), pa.rope_axes((20, 22, 22)))):
        kc, vc, got = p["kc"].clone().zero_(), p["vc"].clone().zero_(), want * 0
        pa.qk_norm_rope_axes(q, k, v, pos.contiguous(), p["slots"], p["cs"], got, kc, vc,
                             axis_of=of, **kw)
        assert torch.equal(got, want)
        at = p["slots"]
        assert torch.equal(kc[at // 16, :, at % 16], p["kc"][at // 16, :, at % 16])


@pytest.mark.parametrize("axis", [0, 1, 2, 3])
def test_a_bad_position_on_any_axis(axis):
    p = {k: v.cuda() for k, v in problem(9, 4, 2, 64, 64, 4, BF16, seed=2).items()}
    p["pos"][axis, 5] = 500 if axis % 2 else -1
    q, k, v = p["qkv"][:, :4], p["qkv"][:, 4:6], p["qkv"][:, 6:]
    out = torch.zeros(9, 4, 64, dtype=BF16, device="cuda")
    kc, vc = p["kc"].clone(), p["vc"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.qk_norm_rope_axes(q, k, v, p["pos"], p["slots"], p["cs"], out, kc, vc,
                         axis_of=bytes(32), status=status)   # no pair on axes 1 to 3
    assert int(status) == pa.PA_ERR_BAD_POSITION
    assert torch.isnan(out[5]).all()
    assert torch.isfinite(out[torch.arange(9) != 5]).all()
    at = int(p["slots"][5])
    assert torch.equal(kc[at // 16, :, at % 16], p["kc"][at // 16, :, at % 16])
    assert torch.equal(vc[at // 16, :, at % 16], p["vc"][at // 16, :, at % 16])


def test_without_rotation_and_empty():
    p = {k: v.cuda() for k, v in problem(5, 4, 2, 64, 64, 2, BF16, seed=3).items()}
    q, k, v = p["qkv"][:, :4], p["qkv"][:, 4:6], p["qkv"][:, 6:]
    out = torch.zeros(5, 4, 64, dtype=BF16, device="cuda")
    pa.qk_norm_rope_axes(q, k, v, None, p["slots"], None, out, p["kc"], p["vc"], axis_of=b"")
    assert torch.equal(out, q)
    # no rows: addresses may be null
    pa.qk_norm_rope(q[:0], k[:0], v[:0], p["pos"][0, :0], p["slots"][:0], p["cs"], out[:0],
                    p["kc"], p["vc"])
    pa.qk_norm_rope_axes(q[:0], k[:0], v[:0], p["pos"][:, :0].contiguous(), p["slots"][:0],
                         p["cs"], out[:0], p["kc"], p["vc"], axis_of=pa.rope_axes((16, 16)))


def test_bindings_check_positions_and_axes():
    p = {k: v.cuda() for k, v in problem(5, 4, 2, 64, 64, 2, BF16, seed=3).items()}
    q, k, v = p["qkv"][:, :4], p["qkv"][:, 4:6], p["qkv"][:, 6:]
    out = torch.zeros(5, 4, 64, dtype=BF16, device="cuda")

    def call(pos=p["pos"], of=pa.rope_axes((16, 16)), cs=p["cs"]):
        pa.qk_norm_rope_axes(q, k, v, pos, p["slots"], cs, out, p["kc"], p["vc"], axis_of=of)

    call()
    for kw in (dict(pos=p["pos"][0]), dict(pos=p["pos"][:, :4].contiguous()),
               dict(pos=p["pos"].long()), dict(pos=p["pos"].expand(2, 5).t().contiguous().t()),
               dict(pos=torch.zeros(5, 5, dtype=torch.int32, device="cuda")),
               dict(of=bytes(31)), dict(of=bytes(33)), dict(of=bytes([2] * 32)),
               dict(of=bytes(200)), dict(pos=None), dict(pos=p["pos"][:0])):
        with pytest.raises(pa.PaError):
            call(**kw)


def test_captured_and_replayed():
    """Positions, slots and rows change in place between replays."""
    a, b = (problem(21, 8, 2, 128, 128, 3, BF16, seed=s) for s in (5, 6))
    of = pa.rope_axes((24, 20, 20), True)
    g = {k: v.cuda() for k, v in a.items()}
    q, k, v = g["qkv"][:, :8], g["qkv"][:, 8:10], g["qkv"][:, 10:]
    out = torch.zeros(21, 8, 128, dtype=BF16, device="cuda")
    call = lambda: pa.qk_norm_rope_axes(q, k, v, g["pos"], g["slots"], g["cs"], out, g["kc"],
                                        g["vc"], axis_of=of, q_weight=g["wq"], k_weight=g["wk"])
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for p in (b, a):
        for name in ("qkv", "pos", "slots", "wq", "wk"):
            g[name].copy_(p[name])
        out.fill_(math.nan)
        graph.replay()
        want = reference(p["qkv"][:, :8], p["wq"], p["cs"], p["pos"], of, 1e-6, 0.0, False)
        close(out, want, BF16)
