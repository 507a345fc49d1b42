"""The parts of a row of the 4-bit decode, as far as the workspace shows them: no GPU."""
import pytest

import paged_attention_decode_v2_gb300 as pa
from paged_attention_decode_v2_gb300 import build as pa_build

LONGEST = 1 << 17      # tokens of a part


@pytest.fixture(scope="module", autouse=True)
def L():
    pa_build.build()


def size(B, n, partition_size, hq=8, hkv=8, d=64):
    return pa.kv4_workspace_size(
        pa.Params(num_seqs=B, num_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=16,
                  num_blocks=1 << 20, max_blocks_per_seq=1 << 20, max_seq_len=n,
                  partition_size=partition_size, scale=1.0, kv_dtype=pa.PA_BF16,
                  out_dtype=pa.PA_BF16), 32)


@pytest.mark.parametrize("B,n", [(256, 1 << 20), (608, 1 << 20), (5000, 1 << 18), (700, 131073)])
def test_no_part_is_longer_than_the_longest(B, n):
    """A batch has at least the slots of its rows in parts of 2^17 tokens (a slot of a row and head
    is a partial of head_dim + 2 float32), however large the partition size."""
    least = B * -(-n // LONGEST) * 8 * (64 + 2) * 4
    for partition_size in (LONGEST, LONGEST + 1, 1 << 20, 1 << 30):
        assert size(B, n, partition_size) >= least
        assert size(B, n, partition_size) == size(B, n, LONGEST)
    assert size(B, n, 1024) > size(B, n, LONGEST)
