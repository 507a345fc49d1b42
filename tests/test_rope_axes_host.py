"""Refusals of the rotation with several axes that need no GPU."""
import pytest

import paged_attention_decode_v2_gb300 as pa


@pytest.mark.parametrize("sections", [[1] * 5, [1] * 300, [16, 16, 16, 16, 0]])
@pytest.mark.parametrize("alternate", [False, True])
def test_more_axes_than_a_call_takes(sections, alternate):
    with pytest.raises(pa.PaError):
        pa.rope_axes(sections, alternate)
    assert len(pa.rope_axes(sections[:4], alternate)) == sum(sections[:4])
