"""CPU checks of the 8-bit cache's size limits."""
import pytest

from packed_decode_attention_b200 import bgtq
from packed_decode_attention_b200 import build as pkg_build


@pytest.mark.parametrize("max_q,heads", [(16, 1 << 20), (15, 1118480), (1, 1 << 24)])
def test_query_rows_a_sequence(max_q, heads):
    """A row's offset among its sequence's (query, head, dimension) stays in an int32: at most 2^24 rows of 128."""
    pkg_build.build()
    base = dict(n_layers=1, max_batch=1, capacity_tokens=64, max_q_tokens=max_q)
    assert (heads // 16) * 16 * max_q <= 1 << 24 < (heads // 16 + 1) * 16 * max_q
    bgtq.bgtq_byte_required_bytes(bgtq.ByteConfig(n_kv_heads=heads // 16, n_q_heads=heads // 16 * 16, **base))
    more = heads // 16 + 1
    with pytest.raises(bgtq.BgtqError) as e:
        bgtq.bgtq_byte_required_bytes(bgtq.ByteConfig(n_kv_heads=more, n_q_heads=16 * more, **base))
    assert e.value.status == -1
