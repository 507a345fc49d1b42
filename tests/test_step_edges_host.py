"""Further checks of the serving-step operators that need no GPU: what the
sources must keep to, refusals, and the build of the two libraries."""
import glob
import os
import re
import sys

import pytest

import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build


def _code(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


SOURCES = sorted(glob.glob(os.path.join(pa_build.CSRC, "*.cu*")))


@pytest.mark.parametrize("path", [p for p in SOURCES
                                  if "cudaGridDependencySynchronize();" in _code(p)],
                         ids=os.path.basename)
def test_results_of_the_grid_before_are_read_coherently(path):
    """A programmatic dependent runs while the grid before it still writes, so
    what it reads after its wait is not read-only for the kernel's lifetime:
    no __ldg there."""
    for kernel in _code(path).split("__global__")[1:]:
        body = kernel.split("template <", 1)[0]
        if "cudaGridDependencySynchronize();" not in body:
            continue
        after = body.split("cudaGridDependencySynchronize();", 1)[1]
        assert "__ldg" not in after and "load_row" not in after
        assert "__ldcg" in after


def test_qk_norm_rope_refuses_outputs_over_inputs():
    """Addresses that are never dereferenced: every call is refused."""
    from test_step_host import A, _rope
    pa_build.build()
    L, bad = pa.lib(), pa.PA_ERR_INVALID_ARG
    T, hq, hkv, d = 5, 8, 2, 128
    row, base = (hq + 2 * hkv) * d, 0x7000000
    ok = dict(num_tokens=T, num_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16,
              num_blocks=10, rotary_dim=d, max_position=100, q_stride=row, k_stride=row,
              v_stride=row, dtype=pa.PA_BF16, flags=0, eps=1e-6, weight_offset=0.0)
    fused = dict(q=base, k=base + 2 * hq * d, v=base + 2 * (hq + hkv) * d)
    span = 2 * T * row                                     # bytes of the projection

    def call(params=(), **kw):
        return _rope(L, pa.RopeParams(**{**ok, **dict(params)}), **{**fused, **kw})

    # over the strided projection: in place, shifted, its first and last row
    for name in ("qo", "ko", "vo", "kc", "vc"):
        for at in (base, base + 2 * hq * d, base + 512, base + span - 256,
                   base - 256, base + 2 * row):
            assert call(**{name: at}) == bad, (name, at - base)
    for name in ("ko", "vo"):
        assert call(**{name: fused["k"]}) == bad and call(**{name: fused["v"]}) == bad
    # contiguous q, k, v: shifted by a row, or one's output over another
    flat = dict(q_stride=hq * d, k_stride=hkv * d, v_stride=hkv * d)
    q, k, v = A[0], A[1], A[2]
    for kw in (dict(qo=q + 2 * hq * d), dict(qo=q - 2 * hq * d), dict(ko=k + 512), dict(ko=v),
               dict(vo=k), dict(ko=q, vo=0), dict(vo=v + 16), dict(qo=k)):
        assert call(flat, **{**dict(q=q, k=k, v=v), **kw}) == bad, kw
    # over the weights, the table, positions, slots; outputs over one another; the pools
    names = ["q", "k", "v", "wq", "wk", "cs", "pos", "slots", "qo", "ko", "vo", "kc", "vc"]
    at = dict(zip(names, A))
    for out in ("qo", "ko", "vo", "kc", "vc"):
        for other in names[3:]:
            if other != out:
                assert call(**{"ko": at["ko"], "vo": at["vo"], out: at[other]}) == bad, (out, other)
    assert call(status=at["pos"] + 4) == bad and call(status=at["kc"] + 8) == bad
    assert call(vc=at["kc"] + 10 * 16 * hkv * d * 2 - 16) == bad
    assert call(dict(num_blocks=2 ** 31 - 1, block_size=2 ** 31 - 1), kc=256) == bad


def test_binding_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    """What _marshal.so was compiled against stands in the binary; a file that
    names something else is out of date however new it is."""
    pa_build.build()
    so = tmp_path / "_marshal.so"
    so.write_bytes(open(pa_build.MARSHAL, "rb").read())
    monkeypatch.setattr(pa_build, "MARSHAL", str(so))
    ran, run = [], pa_build.subprocess.run

    def fake(cmd, **kw):
        if "-o" not in cmd:
            return run(cmd, **kw)
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").write(b"new")
        return pa_build.subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(pa_build.subprocess, "run", fake)
    pa_build._build_marshal(False)
    assert not ran                                         # up to date as it is
    other = pa_build.binding_stamp().replace("torch ", "torch 1.")
    monkeypatch.setattr(pa_build, "binding_stamp", lambda: other)
    pa_build._build_marshal(False)
    assert len(ran) == 1 and any(other in a for a in ran[0]) and so.read_bytes() == b"new"


def test_binding_of_another_torch_is_not_used(monkeypatch):
    pa_build.build()
    assert pa._binding().built_for.startswith(pa_build.binding_stamp())
    monkeypatch.setattr(pa, "_marshal_mod", None)
    monkeypatch.setattr(pa_build, "binding_stamp", lambda: "torch 1.0, some Python, cxx11abi 0")
    with pytest.raises(RuntimeError, match="compiled for.*not for torch 1.0"):
        pa.plan_step(*[None] * 10, block_size=16, num_blocks=1)


@pytest.mark.parametrize("missing", ["torch", "headers", "compiler"])
def test_libpa_is_built_without_the_binding(monkeypatch, tmp_path, capsys, missing):
    """nvcc alone builds libpa.so for callers in C."""
    pa_build.build()                                       # libpa.so itself is up to date
    monkeypatch.setattr(pa_build, "MARSHAL", str(tmp_path / "_marshal.so"))

    class Spec:
        origin = str(tmp_path / "torch" / "__init__.py")

    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
        monkeypatch.setattr(pa_build.importlib.util, "find_spec", lambda name: None)
    elif missing == "headers":
        monkeypatch.setattr(pa_build.importlib.util, "find_spec", lambda name: Spec)
    else:
        monkeypatch.setenv("CXX", "no-such-compiler")
    assert pa_build.build() == pa_build.LIB
    assert "_marshal.so is not built" in capsys.readouterr().err
    assert not os.path.exists(pa_build.MARSHAL)
    assert pa_build.build(binding=False) == pa_build.LIB and capsys.readouterr().err == ""
