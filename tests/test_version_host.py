"""What a program can ask the library about itself."""
import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build


def test_the_version_tells_of_the_4_bit_cache():
    """0.3.0 brought pa_qk_norm_rope_axes and the calls on the 4-bit cache."""
    pa_build.build()
    assert pa.version() >= 300
