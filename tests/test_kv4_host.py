"""Refusals of the calls on the 4-bit cache and of the rotation with several axes,
and what of them needs no GPU (every call fails a host check, or is an empty batch,
before anything is enqueued; the fake addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import kv4_reference as kr
import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build
from test_abi_host import params

A = [0x10000000 * (i + 1) for i in range(20)]   # distinct, far apart, never dereferenced
BAD, NO, ALIGN = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    pa_build.build()
    return pa.lib()


# ---------------------------------------------------------------- the reference

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_reference_values_are_within_half_a_step(dtype, group):
    """|value - x| <= s / 2, and s was rounded from range / 15: half a step of the type more
    (relative), over 15 steps."""
    g = torch.Generator().manual_seed(group)
    x = (torch.randn(40, 3, 256, generator=g) * 3 + 1).to(dtype)
    c, s, m = kr.quantise(x, group)
    v = kr.values(kr.pack(c), torch.stack([s, m], -1).to(dtype))
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[dtype]
    slack = (s * (0.5 + 15 * u)).repeat_interleave(group, -1)
    assert ((v - x.double()).abs() <= slack + 1e-12).all()
    assert c.min() == 0 and c.max() == 15
    assert torch.equal(kr.unpack(kr.pack(c)).double(), c)


def test_rope_axes_sections():
    assert list(pa.rope_axes((2, 1, 3))) == [0, 0, 1, 2, 2, 2]
    assert list(pa.rope_axes((4, 2, 2), alternate=True)) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert list(pa.rope_axes((3,), alternate=True)) == [0, 0, 0]
    assert list(pa.rope_axes((0, 3))) == [1, 1, 1]
    for bad in ((), (3, -1)):
        with pytest.raises(pa.PaError):
            pa.rope_axes(bad)
    with pytest.raises(pa.PaError):
        pa.rope_axes((1, 3), alternate=True)   # pair 5 of 4


# ---------------------------------------------------------------- refusals

def _axes(L, p, axes, **kw):
    names = ["q", "k", "v", "wq", "wk", "cs", "pos", "slots", "qo", "ko", "vo", "kc", "vc",
             "status"]
    at = dict(zip(names, A), ko=0, vo=0, status=0)
    at.update(kw)
    return L.pa_qk_norm_rope_axes(ctypes.byref(p) if p else None,
                                  ctypes.byref(axes) if axes else None,
                                  *[at[n] for n in names], None)


def test_qk_norm_rope_axes_refusals(L):
    ok = dict(num_tokens=3, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
              num_blocks=10, rotary_dim=128, max_position=100, q_stride=1024, k_stride=256,
              v_stride=256, dtype=pa.PA_BF16, flags=0, eps=1e-6, weight_offset=0.0)
    P = lambda **kw: pa.RopeParams(**{**ok, **kw})

    def X(n, of):
        return pa.RopeAxes(n, (ctypes.c_uint8 * 128)(*of))

    three = X(3, [j % 3 for j in range(64)])
    assert _axes(L, None, three) == BAD
    assert _axes(L, P(), None) == BAD
    for x in (X(0, [0] * 64), X(5, [0] * 64), X(-1, [0] * 64), X(2, [0] * 63 + [2]),
              X(1, [1] + [0] * 63)):
        assert _axes(L, P(), x) == BAD
    # everything pa_qk_norm_rope refuses
    for kw in (dict(num_tokens=-1), dict(rotary_dim=8), dict(max_position=0), dict(q_stride=1016)):
        assert _axes(L, P(**kw), three) == BAD, kw
    assert _axes(L, P(head_dim=96), three) == NO
    for name in ("q", "k", "v", "slots", "qo", "cs", "pos", "wq", "kc"):
        assert _axes(L, P(), three, **{name: 0}) == BAD, name
    assert _axes(L, P(), three, pos=0x40000002) == ALIGN
    # an output over the positions of the last axis: three rows of three
    assert _axes(L, P(), three, status=A[6] + 32) == BAD
    # entries past the last pair are not looked at
    assert _axes(L, P(num_tokens=0), X(3, [2] * 64 + [9] * 64)) == pa.PA_OK


def _store(L, p, **kw):
    names = ["k", "v", "slots", "kc", "vc", "ks", "vs", "ko", "vo", "status"]
    at = dict(zip(names, A), ko=0, vo=0, status=0)
    at.update(kw)
    return L.pa_store_kv4(ctypes.byref(p) if p else None, *[at[n] for n in names], None)


def test_store_kv4_refusals(L):
    ok = dict(num_tokens=3, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=10,
              group_size=64, k_stride=256, v_stride=512, dtype=pa.PA_BF16)
    P = lambda **kw: pa.StoreKv4Params(**{**ok, **kw})
    assert _store(L, None) == BAD
    for kw in (dict(num_tokens=-1), dict(num_kv_heads=0), dict(block_size=0), dict(num_blocks=0),
               dict(group_size=16), dict(group_size=96), dict(group_size=0), dict(group_size=256),
               dict(head_dim=64, group_size=128), dict(k_stride=255), dict(v_stride=0)):
        assert _store(L, P(**kw)) == BAD, kw
    for kw in (dict(head_dim=96), dict(dtype=4), dict(num_kv_heads=65536)):
        assert _store(L, P(**kw)) == NO, kw
    assert _store(L, P(k_stride=260)) == ALIGN
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert _store(L, P(), **{name: 0}) == BAD, name
    for name in ("k", "v", "kc", "vc", "ks", "vs", "ko", "vo"):
        assert _store(L, P(), **{name: 0x40000008}) == ALIGN, name
    assert _store(L, P(), slots=0x40000004) == ALIGN
    assert _store(L, P(), status=0x40000002) == ALIGN
    # outputs over inputs or over one another
    assert _store(L, P(), kc=A[0]) == BAD
    assert _store(L, P(), ko=A[0] + 512) == BAD
    assert _store(L, P(), vo=A[1]) == BAD               # in place, but the rows are strided
    assert _store(L, P(), vs=A[5]) == BAD
    assert _store(L, P(), vc=A[3] + 16 * 10 * 2 * 64 - 16) == BAD
    assert _store(L, P(), status=A[2] + 16) == BAD
    assert _store(L, P(num_tokens=0), k=0, v=0, slots=0, kc=0) == pa.PA_OK


def _load(L, p, **kw):
    names = ["kc", "vc", "ks", "vs", "bt", "sl", "to", "ko", "vo", "status"]
    at = dict(zip(names, A), status=0)
    at.update(kw)
    return L.pa_load_kv4(ctypes.byref(p) if p else None, *[at[n] for n in names], None)


def test_load_kv4_refusals(L):
    ok = dict(num_seqs=3, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=10,
              max_blocks_per_seq=5, num_out_blocks=12, max_out_blocks_per_seq=4, max_seq_len=64,
              group_size=32, dtype=pa.PA_F16)
    P = lambda **kw: pa.LoadKv4Params(**{**ok, **kw})
    assert _load(L, None) == BAD
    for kw in (dict(num_seqs=-1), dict(num_kv_heads=0), dict(block_size=0), dict(num_blocks=0),
               dict(num_out_blocks=0), dict(max_blocks_per_seq=0), dict(max_out_blocks_per_seq=0),
               dict(max_seq_len=-1), dict(max_seq_len=65), dict(max_blocks_per_seq=3),
               dict(group_size=48)):
        assert _load(L, P(**kw)) == BAD, kw
    for kw in (dict(head_dim=80), dict(dtype=7), dict(num_seqs=65536),
               dict(num_kv_heads=60000, block_size=1000)):
        assert _load(L, P(**kw)) == NO, kw
    for name in ("kc", "vc", "ks", "vs", "bt", "sl", "to", "ko", "vo"):
        assert _load(L, P(), **{name: 0}) == BAD, name
    for name in ("kc", "vc", "ks", "vs", "ko", "vo"):
        assert _load(L, P(), **{name: 0x40000008}) == ALIGN, name
    for name in ("bt", "sl", "to", "status"):
        assert _load(L, P(), **{name: 0x40000002}) == ALIGN, name
    assert _load(L, P(), ko=A[0]) == BAD
    assert _load(L, P(), vo=A[7] + 4096) == BAD
    assert _load(L, P(), status=A[5] + 8) == BAD
    assert _load(L, P(num_seqs=0), kc=0, ko=0) == pa.PA_OK


def _decode(L, p, g, ws_bytes=1 << 40, **kw):
    names = ["q", "kc", "vc", "ks", "vs", "bt", "sl", "ws"]
    at = dict(zip(names, A), out=A[9])
    at.update(kw)
    return L.pa_decode_kv4(ctypes.byref(p), ctypes.byref(g) if g else None,
                           *[at[n] for n in names], ws_bytes, at["out"], None)


def test_decode_kv4_refusals(L):
    G = pa.Kv4Params
    assert _decode(L, params(), None) == BAD
    for g in (0, 16, 96, 256, -32):
        assert _decode(L, params(), G(g)) == BAD
        assert pa.kv4_workspace_size(params(), g) == 0
    g = G(64)
    for kw in (dict(num_kv_heads=5), dict(partition_size=0), dict(max_seq_len=100001),
               dict(num_seqs=-1), dict(flags=128)):
        assert _decode(L, params(**kw), g) == BAD, kw
    for kw in (dict(head_dim=96), dict(flags=pa.PA_FLAG_SPLIT_X), dict(kv_dtype=5),
               dict(flags=pa.PA_FLAG_SELFTEST_STALL), dict(out_dtype=pa.PA_F16)):
        assert _decode(L, params(**kw), g) == NO, kw
    assert _decode(L, params(head_dim=64), G(128)) == BAD
    for name in ("q", "kc", "vc", "ks", "vs", "bt", "sl", "ws", "out"):
        assert _decode(L, params(), g, **{name: 0}) == BAD, name
    for name in ("q", "kc", "vc", "ks", "vs", "ws", "out"):
        assert _decode(L, params(), g, **{name: 0x40000008}) == ALIGN, name
    assert _decode(L, params(), g, bt=0x40000002) == ALIGN
    n = pa.kv4_workspace_size(params(), 64)
    assert n > 1024
    assert _decode(L, params(), g, ws_bytes=n - 1) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert _decode(L, params(num_seqs=0), g, q=0, ws=0) == pa.PA_OK


@pytest.mark.parametrize("hq, hkv, d", [(8, 1, 128), (32, 8, 128), (24, 4, 256), (32, 2, 64)])
def test_a_workspace_serves_smaller_batches(hq, hkv, d):
    def size(B, n):
        return pa.kv4_workspace_size(
            pa.Params(num_seqs=B, num_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16,
                      num_blocks=1 << 20, max_blocks_per_seq=1 << 16, max_seq_len=n,
                      partition_size=1024, scale=1.0, kv_dtype=pa.PA_BF16, out_dtype=pa.PA_BF16),
            64)

    for n in (1, 200, 5000, 100000):
        got = [size(B, n) for B in range(1, 1000)]
        assert min(got) > 0 and got == sorted(got)
    for B in (1, 3, 19, 40, 300):
        got = [size(B, n) for n in range(1, 9000, 37)]
        assert got == sorted(got)


def test_bindings_refuse_before_the_library():
    k = torch.zeros(2, 4, 64)
    slots = torch.zeros(2, dtype=torch.int64)
    kc, vc, ks, vs = pa.alloc_kv4_cache(3, 4, 16, 64, dtype=torch.float32, device="cpu")
    assert kc.shape == (3, 4, 16, 32) and ks.shape == (3, 4, 16, 1, 2)
    with pytest.raises(pa.PaError):                     # CPU tensors
        pa.store_kv4(k, k, slots, kc, vc, ks, vs)
    for kw in (dict(group_size=48), dict(group_size=128), dict(dtype=torch.int8)):
        with pytest.raises(pa.PaError):
            pa.alloc_kv4_cache(3, 4, 16, 64, device="cpu", **kw)
    x = torch.zeros(3, 2, dtype=torch.int32)
    for of in ("0", [300], None, [-1], 32):
        with pytest.raises(pa.PaError):
            pa.qk_norm_rope_axes(k, k, k, x, slots, torch.zeros(9, 64), k, axis_of=of)
