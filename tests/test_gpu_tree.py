"""Attention of a tree of drafted tokens over the paged cache against the formula in 64 bits."""
import math
import threading
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _tree import DT, KV, TreeCase
from _gpu import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


def run(case, out_dtype=None, err=0, gone=(), **kw):
    """The call, under a table of few blocks (no sequence is cut) also under a wider one (they may be)."""
    try:
        a = case.args(out_dtype, **kw)
        case.call(a)
        case.check(a, err=err, gone=gone)
        if case.width <= 32:
            case.widen(33)
            a = case.args(out_dtype, **kw)
            case.call(a)
            case.check(a, err=err, gone=gone)
    finally:
        case.close()


# types, head layouts, lengths around a block, a key tile and a run; ragged trees, none at all
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g,hkv", [(1, 1), (4, 2), (7, 1), (8, 3)])
def test_types_and_heads(dtype, d, g, hkv):
    run(TreeCase(dtype, d, hkv, g, [0, 3, 130, 257], [1, 9, 0, 5], seed=g + d))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cached", [0, 1, 15, 16, 17, 112, 120, 127, 128, 129, 255, 256, 640, 1300])
def test_lengths(dtype, cached):
    run(TreeCase(dtype, 128, 2, 3, [cached, cached + 5], [16, 7], seed=cached), out_dtype="f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nodes", [1, 2, 4, 5, 8, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256])
def test_tree_sizes(dtype, nodes):
    run(TreeCase(dtype, 64 if nodes % 2 else 128, 1, 2 + nodes % 3, [77, 0], [nodes, max(1, nodes // 3)], seed=nodes))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("kind", ["chain", "star", "tree", "forest"])
@pytest.mark.parametrize("nodes,g", [(40, 1), (100, 4)])
def test_tree_shapes(dtype, kind, nodes, g):
    run(TreeCase(dtype, 128, 2, g, [200, 90], [nodes, nodes - 7], kind=kind, seed=3), out_dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_chains_without_parents(dtype):
    run(TreeCase(dtype, 128, 2, 4, [300, 0, 31], [6, 33, 1], kind="chain"), chain=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch", [1, 5, 64, 300])
def test_batches(dtype, batch):
    rng = np.random.default_rng(batch)
    run(TreeCase(dtype, 64, 2, 2, rng.integers(0, 400, batch), rng.integers(0, 9, batch), seed=batch), rows=5)


# one sequence over many CTAs, beside short ones; wide scores (a few keys carry a row)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("q_size", [0.02, 1.0, 6.0])
def test_long_and_short(dtype, q_size):
    run(TreeCase(dtype, 128, 2, 4, [9000, 3, 500, 0], [13, 8, 1, 2], q_size=q_size, seed=5), out_dtype="f32")


# the output that shows how the weights are held; many pieces to a CTA and many CTAs to a sequence
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [3, 16, 40, 90])
@pytest.mark.parametrize("batch,cached", [(2, 2500), (50, 300)])
def test_output_in_32_bits(dtype, d, nodes, batch, cached):
    rng = np.random.default_rng(nodes)
    run(TreeCase(dtype, d, 4, 4 if batch == 2 else 2, rng.integers(0, cached, batch),
                 rng.integers(1 if batch == 2 else 0, nodes + 1, batch), width=40, seed=nodes), out_dtype="f32",
        max_q_len=nodes)


def test_table_wider_than_the_sequences():
    run(TreeCase("bf16", 128, 2, 4, [40, 700], [8, 8], width=5000))


# NaN and infinities in drafts that a row does not see, in the slots behind a sequence and in blocks of others
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("width,g", [(0, 4), (33, 4), (33, 1), (33, 8)])
def test_masked_keys_reach_nobody(dtype, d, bad, width, g):
    case = TreeCase(dtype, d, 2, g, [100, 250], [20, 11], kind="star", seed=9, garbage=bad, width=width)
    case.k[0][100 + 7] = bad   # node 7 of the first tree: only its own rows see it
    case.v[0][100 + 9] = bad   # node 9
    case.v[1][250 + 4, :, 5] = bad
    for b in range(2):
        case.write(b)
    try:
        a = case.args("f32")
        case.call(a)
        rows = np.ones(case.total, bool)
        rows[[7, 9, 20 + 4]] = False
        case.check(a, rows=rows)
        out = a["out"].cpu().numpy()
        assert np.isnan(out[7]).all() if bad != -math.inf else True
        assert not np.isfinite(out[9]).any()
        assert not np.isfinite(out[20 + 4][:, 5]).any() and np.isfinite(np.delete(out[20 + 4], 5, axis=1)).all()
    finally:
        case.close()


@pytest.mark.parametrize("width", [0, 33])
def test_nan_in_a_cached_key_reaches_every_row(width):
    case = TreeCase("bf16", 128, 1, 4, [300], [12], seed=2, width=width)
    case.k[0][17] = math.nan
    case.write(0)
    try:
        a = case.args("f32")
        case.call(a)
        torch.cuda.synchronize()
        assert torch.isnan(a["out"]).all() and torch.isnan(a["lse"]).all()
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [0, 33])
def test_blocks_out_of_range(dtype, width):
    case = TreeCase(dtype, 128, 2, 2, [200, 0], [9, 4], seed=4, width=width)
    case.tables[0, 3] = case.blocks
    case.tables[0, 12] = -5      # the tree's own block: tokens 192 .. 207
    case.tables[1, 0] = 1 << 30  # all that the second sequence has
    try:
        a = case.args("f32")
        case.call(a)
        case.check(a, gone=[(0, 3), (0, 12), (1, 0)], err=0x1)
        assert (a["out"][9:] == 0).all() and (a["lse"][9:] == -math.inf).all()
    finally:
        case.close()


def test_parents_out_of_order():
    case = TreeCase("bf16", 128, 1, 2, [50], [6], kind="chain")
    bad = [-1, 0, 2, 7, -3, 4]   # nodes 2, 3 and 4 name no node before them
    case.parents = [[-1, 0, -1, -1, -1, 4]]
    try:
        a = case.args("f32")
        a["parents"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        case.call(a)
        case.check(a, err=0x40)
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sequences_out_of_range_are_left_out(dtype):
    case = TreeCase(dtype, 64, 1, 2, [50, 20, 30], [6, 5, 4])
    try:
        a = case.args("f32")
        lens = list(case.lens)
        for wrong, rows in (([lens[0], 3, lens[2]], slice(6, 11)), ([lens[0], 16 * case.width + 1, lens[2]], slice(6, 11)),
                            ([-1, lens[1], lens[2]], slice(0, 6))):
            a["lens"] = torch.tensor(wrong, dtype=torch.int32, device="cuda")
            a["out"].fill_(777)
            a["lse"].fill_(777)
            case.call(a)
            keep = np.ones(case.total, bool)
            keep[rows] = False
            case.check(a, err=0x1, rows=keep)
            assert (a["out"][rows] == 777).all() and (a["lse"][rows] == 777).all()
        # a tree longer than max_q_len; rows past total_q
        a["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for change in (dict(max_q_len=5), dict(total=11)):
            a["out"].fill_(777)
            a["lse"].fill_(777)
            case.call({**a, **change})
            keep = np.ones(case.total, bool)
            keep[slice(0, 6) if "max_q_len" in change else slice(11, 15)] = False
            case.check(a, err=0x1, rows=keep)
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_same_bits_every_time_and_without_lse(dtype):
    case = TreeCase(dtype, 128, 2, 4, [3000, 100, 7], [20, 3, 11])
    try:
        a = case.args("f32")
        case.call(a)
        torch.cuda.synchronize()
        first, lse = a["out"].clone(), a["lse"].clone()
        for _ in range(3):
            a["out"].fill_(0)
            a["lse"].fill_(0)
            a["ws"].fill_(math.nan)
            case.call(a)
            assert torch.equal(first, a["out"]) and torch.equal(lse, a["lse"])
        a["lse"].fill_(5)
        case.call(a, lse=False)
        assert torch.equal(first, a["out"]) and (a["lse"] == 5).all()
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_while_lengths_change(dtype):
    case = TreeCase(dtype, 128, 2, 4, [2000, 100, 900], [20, 3, 11])
    try:
        a = case.args("f32")
        case.call(a)  # first use outside a capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            case.call(a)
        keep = list(case.lens)
        for drop in ((0, 0, 0), (1500, 0, 890), (0, 90, 300)):
            # shorter caches: the trees are then the last tokens of what is left
            case.lens = [n - x for n, x in zip(keep, drop)]
            full = case.k, case.v
            case.k = [k[:n] for k, n in zip(case.k, case.lens)]
            case.v = [v[:n] for v, n in zip(case.v, case.lens)]
            a["lens"].copy_(torch.tensor(case.lens, dtype=torch.int32))
            a["out"].fill_(777)
            graph.replay()
            case.check(a)
            case.k, case.v = full
    finally:
        case.close()


def test_two_graphs_share_a_workspace():
    one = TreeCase("bf16", 128, 2, 4, [3000, 100], [20, 3], seed=1)
    two = TreeCase("bf16", 128, 2, 4, [50, 4000], [64, 9], seed=2)
    try:
        a, b = one.args("f32"), two.args("f32")
        n = max(a["ws_bytes"], b["ws_bytes"])
        ws = torch.full((n // 4,), math.nan, device="cuda")
        a["ws"] = b["ws"] = ws
        graphs = []
        for case, args in ((one, a), (two, b)):
            case.call(args)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                case.call(args)
            graphs.append(g)
        for _ in range(2):
            for g in graphs:
                g.replay()
        one.check(a)
        two.check(b)
    finally:
        one.close()
        two.close()


@pytest.mark.parametrize("d,nodes", [(64, 9), (128, 9), (128, 30), (128, 70), (64, 70)])
def test_waits_that_run_out(d, nodes):
    case = TreeCase("bf16", d, 2, 4, [2000, 40], [nodes, 3], seed=8)
    try:
        a = case.args("f32")
        case.call(a)
        case.check(a)
        pk.kv_debug_set_wait_limit_ns(0)
        try:
            case.call(a)
            torch.cuda.synchronize()
            assert pk.kv_get_device_error(case.pool) & 0x4
        finally:
            pk.kv_debug_set_wait_limit_ns(pk.KV_WAIT_LIMIT_DEFAULT_NS)
        a["out"].fill_(777)
        case.call(a)
        case.check(a)
    finally:
        case.close()


def test_on_a_stream_of_its_own():
    case = TreeCase("f16", 128, 2, 4, [700, 20], [9, 3])
    try:
        a = case.args("f32")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        case.call(a, stream=s)
        s.synchronize()
        case.check(a)
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_calls_at_once(dtype):
    """One pool, two streams, a workspace each."""
    case = TreeCase(dtype, 128, 2, 4, [3000, 20, 900], [40, 3, 64], seed=12)
    try:
        a, b = case.args("f32"), case.args("f32")
        torch.cuda.synchronize()
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(8):
            case.call(a, stream=s)
            case.call(b, stream=t)
        torch.cuda.synchronize()
        case.check(a)
        case.check(b)
        assert torch.equal(a["out"], b["out"])
    finally:
        case.close()


@pytest.mark.parametrize("seed", range(4))
def test_first_calls_of_two_host_threads(seed):
    """They make what the pool keeps for its calls (its tensor maps) together."""
    case = TreeCase("bf16", 128, 2, 4, [700, 20], [9, 3], seed=seed, width=40)
    try:
        a = [case.args("f32") for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        start = threading.Barrier(2)

        def one(i):
            start.wait(timeout=30)
            case.call(a[i], stream=streams[i])
        with ThreadPoolExecutor(2) as pool:
            list(pool.map(one, range(2)))
        torch.cuda.synchronize()
        case.check(a[0])
        case.check(a[1])
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_sequences_of_few_tokens(dtype):
    # more than a thread of a CTA has to scan one by one; sequences without nodes in between
    rng = np.random.default_rng(3)
    run(TreeCase(dtype, 64, 1, 2, rng.integers(0, 20, 3000), rng.integers(0, 3, 3000), seed=6))


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    dtype, d = ("f32", "bf16", "f16")[rng.integers(3)], (64, 128)[rng.integers(2)]
    batch, g, hkv = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 5))
    most = int(np.exp(rng.uniform(0, np.log(256))))
    top = int(np.exp(rng.uniform(0, np.log(4000))))
    run(TreeCase(dtype, d, hkv, g, rng.integers(0, top + 1, batch), rng.integers(0, most + 1, batch),
                 kind=("chain", "star", "tree", "forest")[rng.integers(4)], seed=seed, q_size=float(rng.choice([0.3, 1.0, 3.0]))),
        out_dtype=(dtype, "f32")[rng.integers(2)], rows=int(rng.integers(0, 4)))


def test_offsets_past_32_bits():
    # blocks at the far end of pools of more than 2^32 bytes each
    for dtype, d, hkv in (("bf16", 128, 8), ("f32", 64, 8)):
        blocks = 140000
        pool = pk.kv_pool_create(blocks, 16, hkv, d, KV[dtype])
        small = TreeCase(dtype, d, hkv, 2, [300], [9], seed=3)
        try:
            from _tree import views
            k, v = views(pool, blocks, hkv, d, dtype)
            far = blocks - small.blocks
            k[far:].copy_(small.k_view)
            v[far:].copy_(small.v_view)
            a = small.args("f32")
            a["tables"] = torch.where(a["tables"] >= 0, a["tables"] + far, a["tables"])
            own, small.pool = small.pool, pool
            small.call(a)
            small.check(a)
            small.pool = own
        finally:
            small.close()
            pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("nodes", [3, 30, 70])
def test_output_aligned_to_16_bytes_only(dtype, out_dtype, nodes):
    case = TreeCase(dtype, 64, 2, 4, [300], [nodes])
    try:
        a = case.args(out_dtype)
        n = 16 // a["out"].element_size()
        buf = torch.full((a["out"].numel() + n,), 777.0, dtype=a["out"].dtype, device="cuda")
        a["out"] = buf[n:].view(a["out"].shape)
        q = torch.zeros(a["q"].numel() + 16 // a["q"].element_size(), dtype=a["q"].dtype, device="cuda")
        q[16 // q.element_size():] = a["q"].flatten()
        a["q"] = q[16 // q.element_size():].view(a["q"].shape)
        assert a["out"].data_ptr() % 32 == 16 and a["q"].data_ptr() % 32 == 16
        case.call(a)
        case.check(a)
        assert (buf[:n] == 777).all()
    finally:
        case.close()


def test_no_workspace_under_few_blocks():
    case = TreeCase("f16", 128, 2, 4, [300, 0, 77], [6, 33, 1], width=32)
    try:
        a = case.args("f32")
        assert a["ws_bytes"] == 0 and pk.kv_tree_workspace_size(case.pool, 3, case.hq, 33, 33) > 0
        a["ws"] = None
        case.call(a)
        case.check(a)
    finally:
        case.close()


def test_nothing_to_do():
    case = TreeCase("bf16", 128, 1, 1, [5], [0])
    try:
        a = case.args("f32", rows=3)
        case.call(a)
        case.check(a)
        assert pk.kv_tree_workspace_size(case.pool, 0, 1, 4, 8) == 0
        pk.paged_tree_attention(case.pool, None, None, 0, 0, None, None, 0, None, 0, 1, 1.0, None, pk.KV_F32)
    finally:
        case.close()


def test_refusals():
    case = TreeCase("bf16", 128, 2, 2, [20], [4], width=33)
    i4 = pk.kv_pool_create(4, 16, 2, 128, pk.KV_I4)
    try:
        a = case.args("f32")

        def refused(status, **change):
            x = dict(pool=case.pool, q=a["q"], cu=a["cu"], total=a["total"], max_q_len=4, parents=a["parents"],
                     tables=a["tables"], width=case.width, lens=a["lens"], batch=1, hq=4, scale=1.0, out=a["out"],
                     out_dt=pk.KV_F32, ws=a["ws"], n=a["ws_bytes"])
            x.update(change)
            with pytest.raises(pk.KVError) as e:
                pk.paged_tree_attention(x["pool"], x["q"], x["cu"], x["total"], x["max_q_len"], x["parents"], x["tables"],
                                        x["width"], x["lens"], x["batch"], x["hq"], x["scale"], x["out"], x["out_dt"],
                                        None, x["ws"], x["n"])
            assert e.value.status == status, change
        for change in (dict(pool=None), dict(q=None), dict(cu=None), dict(tables=None), dict(lens=None), dict(out=None),
                       dict(ws=None), dict(batch=-1), dict(total=-1), dict(max_q_len=-1), dict(width=-1), dict(hq=3),
                       dict(hq=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
                       dict(n=a["ws_bytes"] - 1), dict(q=a["q"].data_ptr() + 2), dict(out=a["out"].data_ptr() + 4),
                       dict(ws=a["ws"].data_ptr() + 4)):
            refused(-1, **change)
        for change in (dict(pool=i4), dict(out_dt=pk.KV_F16), dict(hq=18), dict(max_q_len=257), dict(width=1 << 27)):
            refused(-3, **change)
        for args, status in (((case.pool, -1, 4, 4, 4), -1), ((case.pool, 1, 3, 4, 4), -1), ((case.pool, 1, 4, 4, 257), -3),
                             ((i4, 1, 4, 4, 4), -3), ((case.pool, 1, 18, 4, 4), -3), ((None, 1, 4, 4, 4), -1)):
            with pytest.raises(pk.KVError) as e:
                pk.kv_tree_workspace_size(*args)
            assert e.value.status == status
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(case.pool) == 0
        assert (a["out"] == 777).all()
    finally:
        case.close()
        pk.kv_pool_destroy(i4)
