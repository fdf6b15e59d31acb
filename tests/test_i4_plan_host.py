"""The 4-bit decode's plan from host lengths, at widths up to the largest. No GPU."""
import pytest

import paged_kv_cache_196_gb300 as pk


@pytest.mark.parametrize("lens", [[1], [100] * 64, [4000] * 3, [196608] * 8, list(range(1, 4000, 37))])
def test_the_plan_does_not_depend_on_unused_columns(lens):
    """A table wider than the sequences leaves whole sequences whole, and asks for as many
    partitions of its rows as the longest one has pieces."""
    width = -(-max(lens) // 16)
    narrow = pk.kv_decode_plan_i4(lens, 4, width)
    for wide in (2 * width, 1024, 1025, 8192, 2 ** 27 - 1, 2 ** 31 - 4, 2 ** 31 - 1):
        if wide >= width:
            assert (pk.kv_decode_plan_i4(lens, 4, wide) == 1) == (narrow == 1)
            assert 1 <= pk.kv_decode_plan_i4(lens, 4, wide) <= narrow
