"""Calls over drafted tokens at the limits of their arguments."""
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _tree import TreeCase, views
from test_gpu_keep import KeepCase

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


def test_new_lengths_over_an_input():
    """A CTA of one layer writes a sequence's new length while those of others still read the call's inputs."""
    case = KeepCase("bf16", 64, 2, [20, 40, 3], [8, 5, 9], [3, 0, 4])
    try:
        a = case.args()
        held = {x: a[x].clone() for x in ("cu", "path", "count", "tables", "lens")}

        def call(new):
            pk.kv_keep_path(case.pools, a["cu"], 9, a["path"], case.max_path, a["count"], a["tables"], case.width, a["lens"],
                            3, new)
        for x in held:
            n = a[x].numel()
            start = a[x].data_ptr()
            for at in (0, 4 * (n - 1), -8):   # its beginning, its last entry, an array that ends in it
                with pytest.raises(pk.KVError) as e:
                    call(start + at)
                assert e.value.status == -1, (x, at)
        torch.cuda.synchronize()
        assert all(torch.equal(a[x], held[x]) for x in held)
        # behind an input, and before one
        buf = torch.full((9,), 77, dtype=torch.int32, device="cuda")
        buf[3:6] = a["count"]
        a["count"] = buf[3:6]
        for at in (6, 0):
            call(buf[at:at + 3])
            if at == 6:
                a["new"] = torch.cat([buf[6:9], a["new"][3:]])
                case.check(a)
                for p, kv in zip(case.pools, case.before):   # the rows as they were, for the other call
                    for x, y in zip(views(p, case.blocks, 2, 64, "bf16"), kv):
                        x.view(y.dtype).copy_(y)
        a["new"] = torch.cat([buf[0:3], a["new"][3:]])
        case.check(a)
    finally:
        case.close()


@pytest.mark.parametrize("width", [15, 16, 17, 32, 33])
@pytest.mark.parametrize("d,g,nodes", [(64, 1, 3), (64, 3, 40), (128, 8, 9)])
def test_fp32_tables_around_the_limit_of_whole_pairs(width, d, g, nodes):
    """Whole pairs need no workspace; cut ones, in runs down to a key tile, give what the formula gives."""
    for lens in ([16 * width - nodes], [16 * width - nodes, 0, 5, 100, 16 * width - nodes - 3]):
        case = TreeCase("f32", d, 2, g, lens, [nodes] * len(lens), width=width, seed=width)
        try:
            a = case.args("f32")
            assert (a["ws_bytes"] == 0) == (width <= 16)
            case.call(a)
            case.check(a)
        finally:
            case.close()
