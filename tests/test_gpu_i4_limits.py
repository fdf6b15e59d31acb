"""Sizes at the ends of the 4-bit calls' ranges, and inputs whose results must not
depend on which kernel a call takes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _i4 import Cache, attend, check_attention, f64

pytestmark = pytest.mark.gpu


def test_prefill_workspace_with_an_unbounded_chunk_length():
    """Any upper bound of the chunks' lengths may be given, the largest int too: the
    workspace is the one for chunks as long as the table."""
    require_cuda()
    pool = pk.kv_pool_create(4, 16, 8, 128, pk.KV_I4)
    for width in (1, 40, 16384):
        size = [pk.kv_prefill_i4_workspace_size(pool, 1, 16, width, m) for m in (16 * width, 2 ** 30, 2 ** 31 - 1)]
        assert size[1] == size[2] and (width < 40 or size[0] == size[1])
        assert size[2] > 2 * width * 8 * 16 * 128 * 2  # the K and V tiles alone
    pk.kv_pool_destroy(pool)


def test_prefill_with_an_unbounded_chunk_length():
    """The same results as with the chunks' own longest length."""
    c = Cache([300, 129, 45], 2, 128, seed=31)
    cu = np.array([0, 60, 189, 222])
    q = c.queries(222, 8, "bf16")
    out, lse = c.prefill(q, "bf16", "bf16", cu, 2 ** 31 - 1)
    good, lse2 = c.prefill(q, "bf16", "bf16", cu, 129)
    assert torch.equal(out, good) and torch.equal(lse, lse2)
    c.close()


@pytest.mark.parametrize("lens,g,T", [
    ([200, 90], 2, 5),        # by columns
    ([200, 90], 2, 60),       # expanded tiles
    ([9000], 1, 300),         # expanded tiles, their keys cut into pieces
])
def test_prefill_lse_of_a_nan_row_is_nan(lens, g, T):
    """A NaN in q or in a key: the rows that meet it have a NaN log-sum-exp beside their NaN
    output, on every path; -inf would say that they saw no key."""
    c = Cache(lens, 2, 128, seed=14)
    cu = np.arange(len(lens) + 1) * T
    q = c.queries(int(cu[-1]), 2 * g, "bf16")
    ref, lref = c.prefill(q, "bf16", "bf16", cu, T)
    bad = q.clone()
    bad[2, 1, 7] = float("nan")
    out, lse = c.prefill(bad, "bf16", "bf16", cu, T)
    hit = torch.zeros(int(cu[-1]), 2 * g, dtype=torch.bool, device="cuda")
    hit[2, 1] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], ref[~hit]) and torch.equal(lse[~hit], lref[~hit])
    at = lens[0] - T + 3  # a key of the chunk
    k = c.k[0][at:at + 1].clone()
    k[0, 1, 3] = float("nan")
    pk.kv_append_rope(c.pool, k.cuda(), c.v[0][at:at + 1].cuda(), pk.KV_BF16, torch.from_numpy(c.slots[0][at:at + 1]).cuda(), 1)
    out, lse = c.prefill(q, "bf16", "bf16", cu, T)
    hit.zero_()
    hit[3:T, g:] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], ref[~hit]) and torch.equal(lse[~hit], lref[~hit])
    c.close()


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "past"])
@pytest.mark.parametrize("lens,hkv,g,T", [
    ([100, 90], 2, 2, 4),        # by columns
    ([100, 90], 2, 2, 60),       # expanded tiles
    ([700, 300], 1, 4, 260),     # several key tiles
    ([9000], 1, 2, 260),         # keys cut into pieces, some without a block that is not there
])
def test_prefill_leaves_out_the_keys_of_bad_blocks(lens, hkv, g, T, bad):
    """A block id out of range: its keys have no weight, on every path. Blocks of the cached
    part, of the chunk and a whole key tile are missing."""
    c = Cache(lens, hkv, 128, seed=16)
    cu = np.arange(len(lens) + 1) * T
    q = c.queries(int(cu[-1]), hkv * g, "bf16")
    tables = c.tables.copy()
    gone = [0, (lens[0] - T // 2) // 16] + (list(range(8, 16)) if lens[0] > 400 else [])
    tables[0, gone] = c.nb if bad == "past" else bad
    out, lse = c.prefill(q, "bf16", "f32", cu, T, tables=torch.from_numpy(tables).cuda(), expect=0x1)
    o64, l64, q64 = f64(out), f64(lse), f64(q)
    for b, n in enumerate(lens):
        there = np.ones(n, bool)
        if b == 0:
            for i in gone:
                there[16 * i:16 * i + 16] = False
        rows = slice(cu[b], cu[b + 1])
        seen = [int(there[:n - T + i + 1].sum()) for i in range(T)]
        ref = attend(q64[rows], c.kv[b][there], c.vv[b][there], 128 ** -0.5, seen)
        check_attention(o64[rows], l64[rows], ref, 128 ** -0.5, n, "f32", 2.0 ** -11, f"seq {b}", floor=2.0 ** -24)
    c.close()


@pytest.mark.parametrize("T", [4, 60])
def test_prefill_without_a_block_that_is_there(T):
    """No key left: rows of zeros and a log-sum-exp of -inf, as an empty sequence's."""
    c = Cache([60], 2, 128, seed=17)
    q = c.queries(T, 4, "f16")
    out, lse = c.prefill(q, "f16", "f16", [0, T], T, tables=torch.full_like(c.t_tables, -1), expect=0x1)
    assert torch.all(out == 0) and torch.isneginf(lse).all()
    c.close()


@pytest.mark.parametrize("batch", [40, 400, 4100])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_one_split_under_a_wide_table(batch, d):
    """One split means whole sequences, without a workspace, for a table of a long-context
    model's width too: the bits of the narrow table's call, below and above the number of
    pairs that one wave takes and past the batch that the device cuts."""
    c = Cache([500], 2, d, seed=18)
    lens = torch.tensor([(37 * b) % 501 for b in range(batch)], dtype=torch.int32, device="cuda")
    q = c.queries(batch, 8, "bf16")
    outs = []
    for width in (c.width, 8192):
        tables = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        tables[:, :c.width] = c.t_tables[0]
        out, lse = torch.empty_like(q), torch.empty(batch, 8, device="cuda")
        pk.paged_decode_attention_i4(c.pool, q, pk.KV_BF16, tables, width, lens, batch, 8, d ** -0.5, out, pk.KV_BF16, lse, 1)
        assert pk.kv_get_device_error(c.pool) == 0
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for b in range(0, batch, max(1, batch // 12)):
        n = int(lens[b])
        ref = attend(f64(q[b:b + 1]), c.kv[0][:n], c.vv[0][:n], d ** -0.5, [n])
        check_attention(f64(outs[1][0][b:b + 1]), f64(outs[1][1][b:b + 1]), ref, d ** -0.5, n, "bf16", 2.0 ** -11, f"seq {b}")
    c.close()


@pytest.mark.parametrize("splits", [2, 5, 40])
def test_decode_of_long_sequences_under_a_wide_table(splits):
    """More splits than one: planned over the table's width, within the workspace of the
    general rule."""
    c = Cache([20000, 33, 0, 4100], 1, 128, seed=19)
    width = 16384
    tables = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    tables[:, :c.width] = c.t_tables
    q = c.queries(4, 4, "bf16")
    out, lse = torch.empty(4, 4, 128, device="cuda"), torch.empty(4, 4, device="cuda")
    n = pk.kv_decode_workspace_size(4, 4, 1, 128, width, splits)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pk.paged_decode_attention_i4(c.pool, q, pk.KV_BF16, tables, width, c.t_lens, 4, 4, 128 ** -0.5, out, pk.KV_F32, lse, splits, ws, n)
    assert pk.kv_get_device_error(c.pool) == 0
    for b, m in enumerate(c.lens):
        ref = attend(f64(q)[b:b + 1], c.kv[b], c.vv[b], 128 ** -0.5, [int(m)])
        check_attention(f64(out)[b:b + 1], f64(lse)[b:b + 1], ref, 128 ** -0.5, int(m), "f32", 2.0 ** -21, f"seq {b}")
    c.close()


def test_prefill_of_many_drafts():
    """40000 sequences of up to 4 drafted tokens with 8 heads per kv head: two groups of
    columns each, more (sequence, group) pairs than a grid's second dimensions hold."""
    c = Cache([60], 1, 128, seed=20)
    B, T = 40000, 4
    t = np.array([(b % 5) for b in range(B)])
    t[[0, B - 1]] = T
    cu = np.concatenate([[0], np.cumsum(t)])
    lens = np.array([4 + (7 * b) % 57 for b in range(B)], np.int32)
    q = c.queries(1, 8, "bf16").expand(int(cu[-1]), -1, -1).contiguous()
    q *= torch.linspace(0.5, 1.5, q.shape[0], device="cuda")[:, None, None].to(q.dtype)
    out, lse = c.prefill(q, "bf16", "f32", cu, T, tables=c.t_tables.expand(B, -1).contiguous(), lens=torch.from_numpy(lens).cuda())
    for b in list(range(0, B, 1999)) + [32767, 32768, 32769, B - 2, B - 1]:
        n, rows = int(lens[b]), slice(int(cu[b]), int(cu[b + 1]))
        if not t[b]:
            continue
        ref = attend(f64(q[rows]), c.kv[0][:n], c.vv[0][:n], 128 ** -0.5, [n - t[b] + i + 1 for i in range(t[b])])
        check_attention(f64(out[rows]), f64(lse[rows]), ref, 128 ** -0.5, n, "f32", 2.0 ** -11, f"seq {b}", floor=2.0 ** -24)
    c.close()


def test_prefill_size_and_call_refuse_the_same():
    """What the call cannot do its workspace query refuses too."""
    require_cuda()
    pool = pk.kv_pool_create(4, 16, 8, 128, pk.KV_I4)
    t = torch.zeros(1 << 14, dtype=torch.float32, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")

    def both(batch, hq, width, most):
        with pytest.raises(pk.KVError) as e:
            pk.kv_prefill_i4_workspace_size(pool, batch, hq, width, most)
        assert e.value.status == -3
        with pytest.raises(pk.KVError) as e:
            pk.paged_prefill_attention_i4(pool, t, pk.KV_BF16, i, 1, most, i, width, i, batch, hq, 1.0, t, pk.KV_F32, None, t, 2 ** 62)
        assert e.value.status == -3

    both(3, 8, 6_000_000, 400)              # expanded: rows of the tiles past 2^31
    both(65535, 8, 2 ** 31 - 1, 2 ** 31 - 1)
    both(1, 8, 2 ** 27, 4)                  # by columns: keys past 2^31
    both(65535, 64, 2 ** 27 - 1, 4)         # a grid of as many CTAs
    both(65536, 8, 3, 4)
    both(1, 72, 3, 4)
    assert pk.kv_prefill_i4_workspace_size(pool, 3, 8, 5_000_000, 400) > 3 * 5_000_000 * 8 * 8192
    assert pk.kv_get_device_error(pool) == 0
    pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_scale_that_is_no_number(scale, d):
    """Every row with a key is NaN, as the formula has it; an empty sequence keeps its 0."""
    c = Cache([700, 0, 33], 2, d, seed=22)
    q = c.queries(3, 4, "bf16")
    for splits in (1, 3):
        out, lse = c.decode(q, "bf16", "f32", splits, scale=scale)
        assert torch.isnan(out[[0, 2]]).all() and torch.isnan(lse[[0, 2]]).all()
        assert torch.all(out[1] == 0) and torch.isneginf(lse[1]).all()
    c.close()


@pytest.mark.parametrize("most", [4, 400])
def test_prefill_refuses_a_scale_that_is_no_number(most):
    require_cuda()
    pool = pk.kv_pool_create(4, 16, 2, 128, pk.KV_I4)
    pk.kv_pool_set_i4_scales(pool, 2.0 ** 20, 1.0)
    t = torch.zeros(1 << 14, dtype=torch.float32, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")
    for scale in (float("nan"), float("inf"), 3e38, 2e30):  # the last: times the pool's scale past fp32
        with pytest.raises(pk.KVError) as e:
            pk.paged_prefill_attention_i4(pool, t, pk.KV_BF16, i, 1, most, i, 3, i, 1, 4, scale, t, pk.KV_F32, None, t, 2 ** 62)
        assert e.value.status == -1
    pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("q_dtype", ["bf16", "f16"])
@pytest.mark.parametrize("columns", [8, 21, 24, 32, 96])
def test_prefill_by_columns_has_the_decodes_weights(columns, q_dtype):
    """fp32 output by columns keeps weights of two fp16 parts, 2^-21, at every width; the
    same rows over expanded tiles weights of one, and the log-sum-exp of the decode's bound."""
    c = Cache([6000, 33, 700], 1, 128, seed=columns + 1)
    g = 8 if columns % 8 == 0 else 7
    T = columns // g
    cu = np.array([0, T, T, 2 * T])
    q = c.queries(2 * T, g, q_dtype)
    for most, step, floor in ((T, 2.0 ** -21, 2.0 ** -31), (97, 2.0 ** -11, 2.0 ** -24)):
        out, lse = c.prefill(q, q_dtype, "f32", cu, most)
        for b, n in enumerate(c.lens):
            t, rows = int(cu[b + 1] - cu[b]), slice(int(cu[b]), int(cu[b + 1]))
            if t:
                ref = attend(f64(q[rows]), c.kv[b], c.vv[b], 128 ** -0.5, [int(n) - t + i + 1 for i in range(t)])
                check_attention(f64(out[rows]), f64(lse[rows]), ref, 128 ** -0.5, int(n), "f32", step, f"most {most} seq {b}",
                                floor=floor)
    c.close()


def test_prefill_workspace_of_nothing():
    """No sequence, no query token or no table column: an answer, and a call without work."""
    require_cuda()
    pool = pk.kv_pool_create(4, 16, 2, 128, pk.KV_I4)
    for batch, width, most in ((0, 3, 4), (0, 3, 400), (2, 3, 0), (0, 0, 0), (2, 0, 0), (2, 0, 4)):
        n = pk.kv_prefill_i4_workspace_size(pool, batch, 8, width, most)
        assert n == 0 or most > 96 // 4
    t = torch.zeros(1 << 12, dtype=torch.float32, device="cuda")
    i = torch.zeros(8, dtype=torch.int32, device="cuda")
    for batch, rows, most in ((0, 0, 0), (0, 5, 5), (2, 0, 0), (2, 0, 5), (2, 5, 0)):
        pk.paged_prefill_attention_i4(pool, t, pk.KV_BF16, i, rows, most, i, 3, i, batch, 8, 1.0, t, pk.KV_F32)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0 and torch.all(t == 0)
    pk.kv_pool_destroy(pool)
