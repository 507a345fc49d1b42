"""Refusals of the serving-step entry points (CPU only: every call fails a
host check, or is an empty batch, before anything is enqueued; the fake
addresses are never dereferenced)."""
import ctypes

import pytest

import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build
from test_abi_host import params


@pytest.fixture(scope="module")
def L():
    pa_build.build()
    return pa.lib()


A = [0x100000 * (i + 1) for i in range(20)]      # distinct, aligned, never dereferenced


def _plan(L, p, **kw):
    names = ["ctx", "new", "free", "count", "base", "tables", "start", "lens", "pos", "slots",
             "left", "status"]
    at = dict(zip(names, A), base=0, status=0)
    at.update(kw)
    return L.pa_plan_step(ctypes.byref(p) if p else None, *[at[n] for n in names], None)


def test_plan_step_refusals(L):
    ok = dict(num_seqs=4, block_size=16, num_blocks=100, max_blocks_per_seq=8, max_tokens=32,
              max_free=10)
    P = lambda **kw: pa.PlanParams(**{**ok, **kw})
    bad = pa.PA_ERR_INVALID_ARG
    assert _plan(L, None) == bad
    for kw in (dict(num_seqs=-1), dict(block_size=0), dict(num_blocks=0),
               dict(max_blocks_per_seq=0), dict(max_tokens=-1), dict(max_free=-1)):
        assert _plan(L, P(**kw)) == bad
    assert _plan(L, P(max_blocks_per_seq=1 << 27)) == pa.PA_ERR_UNSUPPORTED
    assert _plan(L, P(num_seqs=65536)) == pa.PA_ERR_UNSUPPORTED
    for name in ("ctx", "new", "free", "count", "tables", "start", "lens", "pos", "slots", "left"):
        assert _plan(L, P(), **{name: 0}) == bad, name
    for name in ("ctx", "new", "free", "count", "base", "tables", "start", "lens", "pos", "left",
                 "status"):
        assert _plan(L, P(), **{name: 0x40000002}) == pa.PA_ERR_MISALIGNED, name
    assert _plan(L, P(), slots=0x40000004) == pa.PA_ERR_MISALIGNED
    # outputs over inputs or over one another
    assert _plan(L, P(), lens=A[0]) == bad
    assert _plan(L, P(), left=A[3]) == bad
    assert _plan(L, P(), pos=A[1] + 12) == bad
    assert _plan(L, P(), start=A[7] + 12) == bad


def _rope(L, p, **kw):
    names = ["q", "k", "v", "wq", "wk", "cs", "pos", "slots", "qo", "ko", "vo", "kc", "vc",
             "status"]
    at = dict(zip(names, A), ko=0, vo=0, status=0)
    at.update(kw)
    return L.pa_qk_norm_rope(ctypes.byref(p) if p else None, *[at[n] for n in names], None)


def test_qk_norm_rope_refusals(L):
    ok = dict(num_tokens=3, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
              num_blocks=10, rotary_dim=128, max_position=100, q_stride=1024, k_stride=256,
              v_stride=256, dtype=pa.PA_BF16, flags=0, eps=1e-6, weight_offset=0.0)
    P = lambda **kw: pa.RopeParams(**{**ok, **kw})
    bad, no = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert _rope(L, None) == bad
    for kw in (dict(num_tokens=-1), dict(num_heads=0), dict(num_kv_heads=0), dict(block_size=0),
               dict(num_blocks=0), dict(flags=1), dict(rotary_dim=8), dict(rotary_dim=144),
               dict(rotary_dim=-16), dict(max_position=0), dict(q_stride=1016),
               dict(k_stride=255), dict(v_stride=0), dict(eps=float("nan")), dict(eps=-1.0)):
        assert _rope(L, P(**kw)) == bad, kw
    for kw in (dict(head_dim=96), dict(dtype=5), dict(num_heads=65536)):
        assert _rope(L, P(**kw)) == no, kw
    assert _rope(L, P(q_stride=1028)) == pa.PA_ERR_MISALIGNED
    for name in ("q", "k", "v", "slots", "qo", "cs", "pos", "wq", "wk", "kc", "vc"):
        assert _rope(L, P(), **{name: 0}) == bad, name
    for name in ("q", "k", "v", "wq", "wk", "cs", "qo", "ko", "vo", "kc", "vc"):
        assert _rope(L, P(), **{name: 0x40000008}) == pa.PA_ERR_MISALIGNED, name
    assert _rope(L, P(), slots=0x40000004) == pa.PA_ERR_MISALIGNED
    assert _rope(L, P(), pos=0x40000002) == pa.PA_ERR_MISALIGNED
    assert _rope(L, P(q_stride=2048), qo=A[0]) == bad       # in place over strided rows
    assert _rope(L, P(num_tokens=0), q=0, k=0, v=0, slots=0, qo=0) == pa.PA_OK


def _win(L, p, w, ws_bytes=1 << 40, **kw):
    names = ["q", "k", "v", "bt", "sl", "ws"]
    at = dict(zip(names, A), out=A[6])
    at.update(kw)
    return L.pa_decode_window(ctypes.byref(p), ctypes.byref(w) if w else None,
                              *[at[n] for n in names], ws_bytes, at["out"], None)


def test_decode_window_refusals(L):
    W = pa.WindowParams
    bad = pa.PA_ERR_INVALID_ARG
    assert _win(L, params(), None) == bad
    for w in (W(0, 0), W(-5, 0), W(10, -1)):
        assert _win(L, params(), w) == bad
        assert pa.lib().pa_window_workspace_size(ctypes.byref(params()), ctypes.byref(w)) == 0
    w = W(1000, 4)
    assert _win(L, params(partition_size=24), w) == bad
    assert _win(L, params(num_kv_heads=5), w) == bad
    assert _win(L, params(head_dim=96), w) == pa.PA_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "bt", "sl", "ws", "out"):
        assert _win(L, params(), w, **{name: 0}) == bad, name
    assert _win(L, params(), w, q=0x40000008) == pa.PA_ERR_MISALIGNED
    assert _win(L, params(), w, ws=0x40000010) == pa.PA_ERR_MISALIGNED
    n = pa.window_workspace_size(params(), 1000, 4)
    assert 1024 < n < pa.workspace_size(params())           # the window bounds the partials
    assert _win(L, params(), w, ws_bytes=n - 1) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert _win(L, params(num_seqs=0), w, q=0, ws=0) == pa.PA_OK


def test_prefill_window_refusals(L):
    ok = dict(num_seqs=2, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=50,
              max_blocks_per_seq=8, total_tokens=40, max_query_len=30, max_ctx_len=100,
              kv_dtype=pa.PA_BF16, out_dtype=pa.PA_F32, scale=0.1, flags=0)
    P = lambda **kw: pa.PrefillParams(**{**ok, **kw})

    def call(p, w=pa.WindowParams(10, 2), **kw):
        names = ["q", "k", "v", "kc", "vc", "bt", "qs", "cl", "out"]
        at = dict(zip(names, A))
        at.update(kw)
        return L.pa_prefill_window(ctypes.byref(p) if p else None, ctypes.byref(w) if w else None,
                                   *[at[n] for n in names], None)

    bad, no = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert call(None) == bad and call(P(), None) == bad
    for kw in (dict(num_heads=7), dict(num_seqs=-1), dict(max_ctx_len=129), dict(scale=0.0),
               dict(flags=256), dict(block_size=0), dict(max_query_len=-1)):
        assert call(P(**kw)) == bad, kw
    assert call(P(), pa.WindowParams(0, 1)) == bad
    for kw in (dict(head_dim=96), dict(kv_dtype=9), dict(out_dtype=pa.PA_F16)):
        assert call(P(**kw)) == no, kw
    for name in ("q", "k", "v", "kc", "vc", "bt", "qs", "cl", "out"):
        assert call(P(), **{name: 0}) == bad, name
    assert call(P(), k=0x40000008) == pa.PA_ERR_MISALIGNED
    assert call(P(), qs=0x40000002) == pa.PA_ERR_MISALIGNED
    for kw in (dict(num_seqs=0), dict(total_tokens=0), dict(max_query_len=0)):
        assert call(P(**kw), q=0, out=0) == pa.PA_OK


def test_decode_prefix_refusals(L):
    X = pa.PrefixParams

    def call(p, x=X(1000, 63), ws_bytes=1 << 40, **kw):
        names = ["q", "k", "v", "pb", "pl", "bt", "sl", "ws"]
        at = dict(zip(names, A), out=A[9])
        at.update(kw)
        return L.pa_decode_prefix(ctypes.byref(p), ctypes.byref(x) if x else None,
                                  *[at[n] for n in names], ws_bytes, at["out"], None)

    bad = pa.PA_ERR_INVALID_ARG
    assert call(params(), None) == bad
    for x in (X(-1, 10), X(100, -1), X(1009, 63)):
        assert call(params(), x) == bad
        assert pa.prefix_workspace_size(params(), x.max_prefix_len, x.max_prefix_blocks) == 0
    for name in ("q", "k", "v", "pb", "pl", "bt", "sl", "ws", "out"):
        assert call(params(), **{name: 0}) == bad, name
    assert call(params(), pb=0x40000002) == pa.PA_ERR_MISALIGNED
    assert call(params(), ws=0x40000010) == pa.PA_ERR_MISALIGNED
    n = pa.prefix_workspace_size(params(), 1000, 63)
    assert call(params(), ws_bytes=n - 1) == pa.PA_ERR_WORKSPACE_TOO_SMALL
    assert call(params(num_seqs=0), q=0, ws=0) == pa.PA_OK


def test_bindings_refuse_before_the_library():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(pa.PaError):                          # CPU tensors
        pa.plan_step(x, x, x, x[:1], x[:, None].contiguous(), torch.zeros(3, dtype=torch.int32),
                     x.clone(), x.clone(), torch.zeros(2, dtype=torch.int64), x[:1].clone(),
                     block_size=16, num_blocks=4)
    q = torch.zeros(2, 4, 64)
    with pytest.raises(pa.PaError):
        pa.qk_norm_rope(q, q[:, :2], q[:, 2:], x, torch.zeros(2, dtype=torch.int64), None,
                        torch.zeros_like(q))


@pytest.mark.parametrize("hq, hkv, d", [(8, 1, 128), (32, 8, 128), (24, 4, 256), (16, 16, 128)])
def test_a_workspace_serves_smaller_batches(hq, hkv, d):
    """The sizes never fall as sequences or lengths are added, so one workspace
    for the largest step serves every step."""
    def params(B, L):
        return pa.Params(num_seqs=B, num_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16,
                         num_blocks=1 << 20, max_blocks_per_seq=1 << 16, max_seq_len=L,
                         partition_size=512, scale=1.0, kv_dtype=pa.PA_BF16, out_dtype=pa.PA_BF16)

    sizes = (lambda B, L: pa.window_workspace_size(params(B, L), 4096, 4),
             lambda B, L: pa.prefix_workspace_size(params(B, 300), 20 * L, 20 * L // 16 + 1),
             lambda B, L: pa.prefix_workspace_size(params(B, L), 32000, 2000))
    for size in sizes:
        for L in (1, 200, 4100):
            got = [size(B, L) for B in range(1, 700)]
            assert min(got) > 0 and got == sorted(got)
        for B in (1, 3, 19, 40, 300):
            got = [size(B, L) for L in range(1, 5000, 37)]
            assert got == sorted(got)
