"""Calls over drafted tokens at the limits of their arguments."""
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _tree import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_columns_of_a_table(dtype):
    """A key tile's end has to be an int: 2^27 - 8 columns of 16 tokens end at 2^31 - 128."""
    case = TreeCase(dtype, 64, 1, 2, [20], [4])
    try:
        most = (1 << 27) - 8
        assert pk.kv_tree_workspace_size(case.pool, 1, 2, most, 4) > 0
        a = case.args("f32")
        for width in (most + 1, most + 7, most + 8):
            with pytest.raises(pk.KVError) as e:
                pk.kv_tree_workspace_size(case.pool, 1, 2, width, 4)
            assert e.value.status == -3
            with pytest.raises(pk.KVError) as e:
                pk.paged_tree_attention(case.pool, a["q"], a["cu"], 4, 4, a["parents"], a["tables"], width, a["lens"], 1, 2,
                                        1.0, a["out"], pk.KV_F32, None, a["ws"], 1 << 40)
            assert e.value.status == -3
        torch.cuda.synchronize()
        assert (a["out"] == 777).all()
    finally:
        case.close()


def test_a_sequence_in_a_table_of_the_most_columns():
    """One short sequence (the columns behind it are not read: a table of one row may end with the memory)."""
    for dtype in ("f32", "f16"):
        case = TreeCase(dtype, 64, 1, 2, [700], [9], width=44)
        try:
            a = case.args("f32")
            case.width = (1 << 27) - 8
            n = pk.kv_tree_workspace_size(case.pool, 1, case.hq, case.width, 9)
            a["ws"], a["ws_bytes"] = torch.empty(n // 4, device="cuda"), n
            case.call(a)
            case.check(a)
        finally:
            case.close()
