"""Checks of the rotation's arguments that need no GPU."""
import ctypes

import pytest

import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build


@pytest.mark.parametrize("sections", [[1] * 5, [1] * 300, [16, 16, 16, 16, 0]])
@pytest.mark.parametrize("alternate", [False, True])
def test_more_axes_than_a_call_takes(sections, alternate):
    with pytest.raises(pa.PaError):
        pa.rope_axes(sections, alternate)
    assert len(pa.rope_axes(sections[:4], alternate)) == sum(sections[:4])


def test_without_rows_no_address_is_looked_at():
    """An empty step's tensors have null addresses.  The sizes are still checked."""
    pa_build.build()
    L = pa.lib()
    ok = dict(num_tokens=0, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
              num_blocks=10, rotary_dim=128, max_position=100, q_stride=1024, k_stride=256,
              v_stride=256, dtype=pa.PA_BF16, flags=0, eps=1e-6, weight_offset=0.0)
    of = pa.RopeAxes(3, (ctypes.c_uint8 * 128)(*pa.rope_axes((24, 20, 20))))
    none = [None] * 15
    assert L.pa_qk_norm_rope(ctypes.byref(pa.RopeParams(**ok)), *none) == pa.PA_OK
    assert L.pa_qk_norm_rope_axes(ctypes.byref(pa.RopeParams(**ok)), ctypes.byref(of),
                                  *none) == pa.PA_OK
    for kw in (dict(max_position=0), dict(rotary_dim=8), dict(num_heads=0)):
        bad = ctypes.byref(pa.RopeParams(**{**ok, **kw}))
        assert L.pa_qk_norm_rope(bad, *none) == pa.PA_ERR_INVALID_ARG, kw
        assert L.pa_qk_norm_rope_axes(bad, ctypes.byref(of), *none) == pa.PA_ERR_INVALID_ARG, kw
