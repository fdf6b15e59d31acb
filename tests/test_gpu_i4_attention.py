"""Decode and prefill attention over a 4-bit pool on the GPU against 64-bit
attention over what the pool stands for; the bounds are derived in
_i4.check_attention.  Unused slots hold codes of 7 under NaN scales throughout."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _i4 import KV, TORCH, Cache, attend, check_attention, f64, raw_bytes, rope_table, rotate32, stored

pytestmark = pytest.mark.gpu

# rounding of a softmax weight: fp16, or two fp16 parts (fp32 output)
STEP = {"f32": 2.0 ** -21, "bf16": 2.0 ** -11, "f16": 2.0 ** -11}


def check_decode(c, q, out, lse, out_type, what="", lens=None):
    lens = c.lens if lens is None else lens
    q64, o64, l64 = f64(q), f64(out), f64(lse)
    for b, n in enumerate(lens):
        ref = attend(q64[b:b + 1], c.kv[b], c.vv[b], c.d ** -0.5, [int(n)])
        check_attention(o64[b:b + 1], l64[b:b + 1], ref, c.d ** -0.5, int(n), out_type, STEP[out_type], f"{what} seq {b}")
        if n == 0:
            assert np.all(o64[b] == 0)


@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_dtype,out_type", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_decode_ragged(g, d, q_dtype, out_type):
    c = Cache([1, 15, 16, 17, 35, 100, 257, 0, 64], 2, d, seed=g + d)
    q = c.queries(len(c.lens), 2 * g, q_dtype)
    for splits in (1, 4, 0):
        out, lse = c.decode(q, q_dtype, out_type, splits)
        check_decode(c, q, out, lse, out_type, f"splits {splits}")
    c.close()


@pytest.mark.parametrize("splits", [1, 3, 32, 33, 150])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_every_merge(splits, d):
    """One partition, merged by the last CTA (up to 32), by the merge kernel."""
    c = Cache([9600, 5, 0, 2500], 1, d, seed=splits)
    q = c.queries(4, 4, "bf16")
    out, lse = c.decode(q, "bf16", "f32", splits)
    check_decode(c, q, out, lse, "f32")
    again, lse2 = c.decode(q, "bf16", "f32", splits)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    c.close()


def test_decode_more_pairs_than_counters():
    """batch x kv heads past the pool's arrival counters: the merge kernel takes over."""
    c = Cache([300], 8, 64, seed=3)
    B = 8300
    tables = c.t_tables.expand(B, -1).contiguous()
    lens = torch.full((B,), 300, dtype=torch.int32, device="cuda")
    q = c.queries(1, 8, "f16")
    one, lse1 = c.decode(q, "f16", "f16", 3)
    out, lse = c.decode(q.expand(B, -1, -1).contiguous(), "f16", "f16", 3, tables=tables, lens=lens)
    # cut and merged otherwise, so each is held to the reference; equal rows are equal
    check_decode(c, q, one, lse1, "f16")
    check_decode(c, q, out[:1], lse[:1], "f16")
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    c.close()


def test_decode_placement_and_order_do_not_matter():
    lens = [35, 170, 1, 90, 16]
    a, b = Cache(lens, 2, 128, seed=7, extra=2), Cache(lens, 2, 128, seed=7, extra=40)
    q = a.queries(5, 8, "bf16")
    order = torch.tensor([4, 1, 0, 3, 2], dtype=torch.int32, device="cuda")
    # the caches of one seed hold the same rows only if drawn alike: append a's rows to b
    for s, k, v in zip(b.slots, a.k, a.v):
        pk.kv_append_rope(b.pool, k.cuda(), v.cuda(), pk.KV_BF16, torch.from_numpy(s).cuda(), len(s))
    for splits in (1, 3):
        x, lx = a.decode(q, "bf16", "bf16", splits)
        y, ly = b.decode(q, "bf16", "bf16", splits, order=order)
        assert torch.equal(x, y) and torch.equal(lx, ly)
    a.close()
    b.close()


@pytest.mark.parametrize("bad", [-1, -2, -2 ** 31, 2 ** 31 - 1])
def test_decode_bad_blocks_are_skipped_and_flagged(bad):
    c = Cache([100, 64], 2, 128, seed=9)
    q = c.queries(2, 4, "bf16")
    tables = c.tables.copy()
    tables[0, 2], tables[1, 0] = c.nb, bad
    out, lse = c.decode(q, "bf16", "f32", 2, tables=torch.from_numpy(tables).cuda(), expect=0x1)
    c.kv = [np.delete(c.kv[0], np.s_[32:48], 0), c.kv[1][16:]]
    c.vv = [np.delete(c.vv[0], np.s_[32:48], 0), c.vv[1][16:]]
    check_decode(c, q, out, lse, "f32", lens=[84, 48])
    # a length past the table is clamped to it
    lens = torch.tensor([16 * c.width + 1, 0], dtype=torch.int32, device="cuda")
    c.decode(q, "bf16", "f32", 1, lens=lens, tables=torch.zeros_like(c.t_tables), expect=0x1)
    c.decode(q, "bf16", "f32", 1, order=torch.tensor([0, 7], dtype=torch.int32, device="cuda"), expect=0x1)
    c.close()


@pytest.mark.parametrize("size", [1e-30, 1e-6, 300.0, 3e4])
def test_decode_query_magnitudes(size):
    """bf16 queries far outside fp16's range, and one dominating element."""
    c = Cache([40, 90], 1, 128, seed=2)
    q = c.queries(2, 8, "bf16").float()
    q[0, 1, 5] *= 1000
    q = (q * size).to(torch.bfloat16)
    scale = 128 ** -0.5 / size
    out, lse = c.decode(q, "bf16", "f32", 1, scale=scale)
    for b, n in enumerate(c.lens):
        ref = attend(f64(q)[b:b + 1], c.kv[b], c.vv[b], scale, [int(n)])
        check_attention(f64(out)[b:b + 1], f64(lse)[b:b + 1], ref, scale, int(n), "f32", STEP["f32"])
    c.close()


def test_decode_nan_stays_in_its_rows():
    c = Cache([40, 40], 2, 128, seed=4)
    q = c.queries(2, 4, "bf16")
    ref, lref = c.decode(q, "bf16", "bf16", 2)
    bad = q.clone()
    bad[0, 1, 7] = float("nan")
    out, lse = c.decode(bad, "bf16", "bf16", 2)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], lref[keep])
    # a NaN key group reaches every query head of its kv head, no other
    k = c.k[1][39:].clone()
    k[0, 1, 3] = float("nan")
    pk.kv_append_rope(c.pool, k.cuda(), c.v[1][39:].cuda(), pk.KV_BF16, torch.from_numpy(c.slots[1][39:]).cuda(), 1)
    out, lse = c.decode(q, "bf16", "bf16", 2)
    assert torch.isnan(out[1, 2:]).all() and torch.equal(out[0], ref[0]) and torch.equal(out[1, :2], ref[1, :2])
    c.close()


def test_decode_past_32_bit_offsets():
    """Blocks whose tiles lie past 4 GiB of the pool."""
    c = Cache([70, 33], 8, 128, seed=6, num_blocks=480_000, poison=False)
    assert int(c.tables.max()) * 8 * 9 * 128 > 2 ** 32
    q = c.queries(2, 32, "bf16")
    out, lse = c.decode(q, "bf16", "bf16", 2)
    check_decode(c, q, out, lse, "bf16")
    ko, vo = (torch.empty(33, 8, 128, device="cuda") for _ in "kv")
    pk.kv_read_tokens(c.pool, torch.from_numpy(c.slots[1]).cuda(), 33, ko, vo, pk.KV_F32)
    np.testing.assert_array_equal(f64(ko), c.kv[1])
    cu = [0, 40, 73]
    q = c.queries(73, 16, "bf16")
    out, lse = c.prefill(q, "bf16", "bf16", cu, 40)
    check_prefill(c, q, out, lse, cu, "bf16")
    c.close()


def test_decode_wait_limit():
    """A wait that runs out is reported; the pool works again afterwards."""
    c = Cache([3000, 800], 8, 128, seed=5, num_blocks=16384, poison=False)
    raw_bytes(pk.kv_pool_ptrs(c.pool)[0], (c.nb - c.width - 50) * 8 * 18 * 128).fill_(0)  # the other blocks: zeros
    # more bytes than L2 holds: some first copy is not there when it is looked for
    B, width = 64, 250
    tables = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    lens = torch.full((B,), 16 * width, dtype=torch.int32, device="cuda")
    q = c.queries(B, 32, "bf16")
    out = torch.empty(B, 32, 128, dtype=torch.bfloat16, device="cuda")
    n = pk.kv_decode_workspace_size(B, 32, 8, 128, width, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pk.kv_debug_set_wait_limit_ns(0)
    try:
        seen = 0
        for _ in range(3):  # the first launch after the setting starts slowly enough for its copies to come in time
            pk.paged_decode_attention_i4(c.pool, q, pk.KV_BF16, tables, width, lens, B, 32, 0.1, out, pk.KV_BF16, None, 2, ws, n)
            torch.cuda.synchronize()
            seen |= pk.kv_get_device_error(c.pool)
        assert seen == 0x4
    finally:
        pk.kv_debug_set_wait_limit_ns(pk.KV_WAIT_LIMIT_DEFAULT_NS)
    q = c.queries(2, 32, "bf16")
    out, lse = c.decode(q, "bf16", "bf16", 3)
    check_decode(c, q, out, lse, "bf16")
    c.close()


def test_two_graphs_share_a_workspace():
    """Two captured steps over one pool and one workspace, replayed in turn, and a
    length that changes between replays: the cut is made on the device."""
    a, lens2 = Cache([900, 40, 2000, 333], 2, 128, seed=21), [500, 40, 1200, 16]
    q1, q2 = a.queries(4, 8, "bf16", seed=1), a.queries(4, 8, "bf16", seed=2)
    lens = a.t_lens.clone()
    outs = [torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.empty(4, 8, device="cuda") for _ in range(2)]
    n = pk.kv_decode_workspace_size(4, 8, 2, 128, a.width, 8)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs = []
    for q, out, lse in zip((q1, q2), outs, lses):
        def step():
            pk.paged_decode_attention_i4(a.pool, q, pk.KV_BF16, a.t_tables, a.width, lens, 4, 8, 128 ** -0.5, out, pk.KV_BF16, lse, 8,
                                         ws, n)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for now in (a.lens, np.array(lens2, np.int32), a.lens):
        lens.copy_(torch.from_numpy(now))
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for q, out, lse in zip((q1, q2), outs, lses):
            for b, m in enumerate(now):
                ref = attend(f64(q)[b:b + 1], a.kv[b][:m], a.vv[b][:m], 128 ** -0.5, [int(m)])
                check_attention(f64(out)[b:b + 1], f64(lse)[b:b + 1], ref, 128 ** -0.5, int(m), "bf16", STEP["bf16"])
    assert pk.kv_get_device_error(a.pool) == 0
    a.close()


@pytest.mark.parametrize("batch", [255, 257, 1100, 4096, 4097])
def test_decode_many_sequences(batch):
    """Batches around the scan's slices and past the largest that it takes."""
    lens = [(i * 37) % 40 for i in range(batch)]
    lens[batch // 2] = 700
    one = Cache([700], 1, 64, seed=8)
    tables = one.t_tables.expand(batch, -1).contiguous()
    t_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = one.queries(batch, 2, "f16")
    for splits in (1, 3):
        out, lse = one.decode(q, "f16", "f32", splits, tables=tables, lens=t_lens)
        o64, l64, q64 = f64(out), f64(lse), f64(q)
        for b in list(range(0, batch, 41)) + [batch // 2, batch - 1]:
            ref = attend(q64[b:b + 1], one.kv[0][:lens[b]], one.vv[0][:lens[b]], 64 ** -0.5, [lens[b]])
            check_attention(o64[b:b + 1], l64[b:b + 1], ref, 64 ** -0.5, lens[b], "f32", STEP["f32"], f"seq {b}")
    one.close()


@pytest.mark.parametrize("d", [64, 128])
def test_decode_runs_of_whole_sequences(d):
    """One split and more (sequence, kv head) pairs than two for every CTA: a CTA takes
    several pairs in turn, and each result equals that of its own CTA bit for bit."""
    c = Cache([2500], 2, d, seed=16)
    B = 700
    lens = torch.tensor([(i * 911) % 2500 if i % 5 == 0 else (i * 37) % 60 for i in range(B)], dtype=torch.int32, device="cuda")
    tables = c.t_tables.expand(B, -1).contiguous()
    q = c.queries(B, 8, "bf16")
    out, lse = c.decode(q, "bf16", "bf16", 1, tables=tables, lens=lens)
    for at in range(0, B, 70):
        part = slice(at, at + 70)
        o, l = c.decode(q[part].contiguous(), "bf16", "bf16", 1, tables=tables[part].contiguous(), lens=lens[part].contiguous())
        assert torch.equal(out[part], o) and torch.equal(lse[part], l)
    bad = lens.clone()
    bad[333] = 16 * c.width + 1  # read as far as the table goes
    out2, _ = c.decode(q, "bf16", "bf16", 1, tables=tables, lens=bad, expect=0x1)
    keep = torch.arange(B, device="cuda") != 333
    assert torch.equal(out2[keep], out[keep])
    c.close()


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_decode_scale_of_zero_and_below(scale):
    c = Cache([100, 33], 2, 128, seed=14)
    q = c.queries(2, 4, "bf16")
    out = torch.empty(2, 4, 128, device="cuda")
    lse = torch.empty(2, 4, device="cuda")
    pk.paged_decode_attention_i4(c.pool, q, pk.KV_BF16, c.t_tables, c.width, c.t_lens, 2, 4, scale, out, pk.KV_F32, lse, 1)
    for b, n in enumerate(c.lens):
        ref = attend(f64(q)[b:b + 1], c.kv[b], c.vv[b], scale, [int(n)])
        check_attention(f64(out)[b:b + 1], f64(lse)[b:b + 1], ref, scale, int(n), "f32", STEP["f32"])
    c.close()


# ------------------------------------------------------------------ prefill
def check_prefill(c, q, out, lse, cu, out_type, what=""):
    q64, o64, l64 = f64(q), f64(out), f64(lse)
    for b, n in enumerate(c.lens):
        T = cu[b + 1] - cu[b]
        rows = slice(cu[b], cu[b + 1])
        seen = [int(n) - T + i + 1 for i in range(T)]
        ref = attend(q64[rows], c.kv[b], c.vv[b], c.d ** -0.5, seen)
        # the tcgen05 kernel's weights are fp16 for every output type, and rounded
        # to 2^-25 of a reference weight of at least 1
        check_attention(o64[rows], l64[rows], ref, c.d ** -0.5, int(n), out_type, 2.0 ** -11, f"{what} seq {b}",
                        floor=2.0 ** -24)


@pytest.mark.parametrize("q_dtype,out_type", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("g,hkv", [(4, 2), (7, 1), (1, 3)])
@pytest.mark.parametrize("lens,chunks", [
    ([3, 40, 130, 17], [3, 2, 1, 0]),          # few query tokens: a column each
    ([200, 33], [8, 4]),
    ([300, 129, 45], [50, 129, 33]),           # expanded tiles, one chunk that starts its sequence
    ([400], [300]),
    ([40, 300, 97], [20, 11, 1]),              # between the two: by columns, or expanded
])
def test_prefill(q_dtype, out_type, g, hkv, lens, chunks):
    c = Cache(lens, hkv, 128, seed=sum(lens) + g)
    cu = np.concatenate([[0], np.cumsum(chunks)])
    q = c.queries(int(cu[-1]) + 2, g * hkv, q_dtype)  # two rows no chunk covers
    out, lse = c.prefill(q, q_dtype, out_type, cu, max(chunks))
    check_prefill(c, q[:-2], out[:-2], lse[:-2], cu, out_type)
    assert torch.all(out[-2:] == 7) and torch.all(lse[-2:] == 7)
    c.close()


@pytest.mark.parametrize("columns", [8, 9, 16, 17, 24, 32, 48, 96])
def test_prefill_few_columns_long_context(columns):
    """Each width of the column form, cut into partitions that are merged."""
    c = Cache([6000, 700, 16 * 40], 1, 128, seed=columns)
    T = columns if columns % 2 else columns // 2
    g = columns // T
    cu = np.array([0, T, T, T + 1 + T // 2])  # the middle sequence has no query
    q = c.queries(int(cu[-1]), g, "bf16")
    out, lse = c.prefill(q, "bf16", "bf16", cu, T)
    check_prefill(c, q, out, lse, cu, "bf16")
    # the same rows through the expanding path: equal within the two forms' bounds
    out2, _ = c.prefill(q, "bf16", "f32", cu, 97)
    check_prefill(c, q, out2, lse, cu, "f32")
    c.close()


@pytest.mark.parametrize("T", [4, 40, 60])
def test_prefill_flags_bad_blocks_and_lengths(T):
    c = Cache([100, 90], 2, 128, seed=9)
    q = c.queries(2 * T, 4, "bf16")
    tables = c.tables.copy()
    tables[0, 1] = c.nb + 3
    cu = [0, T, 2 * T]
    out, _ = c.prefill(q, "bf16", "bf16", cu, T, tables=torch.from_numpy(tables).cuda(), expect=0x1)
    good, _ = c.prefill(q, "bf16", "bf16", cu, T)
    assert torch.equal(out[T:], good[T:]) and torch.isfinite(out).all()
    for lens in ([T - 1, 90], [16 * c.width + 1, 90]):
        out, _ = c.prefill(q, "bf16", "bf16", cu, T, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), expect=0x1)
        assert torch.all(out[:T] == 7) and torch.equal(out[T:], good[T:])  # the sequence is left out
    c.close()


@pytest.mark.parametrize("out_type", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,g,lens,chunks", [
    (1, 1, [9000], [300]),                 # two query tiles, their keys cut into many pieces
    (1, 8, [5000, 700, 130, 4100], [40, 700, 129, 33]),
    (2, 4, [8000, 20, 0, 3000], [130, 20, 0, 41]),
    (1, 3, [3000, 600], [2600, 90]),       # rows that see none of a piece's keys
])
def test_prefill_keys_cut(hkv, g, lens, chunks, out_type):
    c = Cache(lens, hkv, 128, seed=sum(lens) + g)
    cu = np.concatenate([[0], np.cumsum(chunks)])
    q = c.queries(int(cu[-1]), g * hkv, "bf16")
    out, lse = c.prefill(q, "bf16", out_type, cu, max(chunks))
    check_prefill(c, q, out, lse, cu, out_type)
    for _ in range(3):  # the last piece to arrive differs, the result does not
        again, lse2 = c.prefill(q, "bf16", out_type, cu, max(chunks))
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    c.close()


def test_prefill_more_sequences_than_are_ordered_at_once():
    B = 600
    one = Cache([1500], 1, 128, seed=6)
    lens = torch.tensor([1500 if b % 199 == 7 else 33 + b % 90 for b in range(B)], dtype=torch.int32)
    T = [0 if b % 11 == 3 else 33 if b % 199 == 7 else 1 + b % 33 for b in range(B)]
    cu = np.concatenate([[0], np.cumsum(T)])
    q = one.queries(int(cu[-1]), 1, "f16")
    out, lse = one.prefill(q, "f16", "f16", cu, 33, tables=one.t_tables.expand(B, -1).contiguous(), lens=lens.cuda())
    q64, o64, l64 = f64(q), f64(out), f64(lse)
    for b in list(range(0, B, 37)) + [7, 206, B - 1]:
        n, rows = int(lens[b]), slice(cu[b], cu[b + 1])
        ref = attend(q64[rows], one.kv[0][:n], one.vv[0][:n], 128 ** -0.5, [n - T[b] + i + 1 for i in range(T[b])])
        check_attention(o64[rows], l64[rows], ref, 128 ** -0.5, n, "f16", 2.0 ** -11, f"seq {b}", floor=2.0 ** -24)
    one.close()


def test_prefill_longer_than_announced_is_left_out():
    c = Cache([300, 200], 1, 128, seed=3)
    cu = [0, 120, 220]
    q = c.queries(220, 4, "bf16")
    out, _ = c.prefill(q, "bf16", "bf16", cu, 100, expect=0x1)
    good, _ = c.prefill(q, "bf16", "bf16", cu, 120)
    assert torch.all(out[:120] == 7) and torch.all(torch.isfinite(out[120:]))
    assert torch.equal(out[120:], good[120:])
    c.close()


@pytest.mark.parametrize("T", [5, 60])
def test_prefill_nan_stays_in_its_rows(T):
    c = Cache([200, 90], 2, 128, seed=4)
    cu = [0, T, 2 * T]
    q = c.queries(2 * T, 4, "bf16")
    ref, lref = c.prefill(q, "bf16", "bf16", cu, T)
    bad = q.clone()
    bad[2, 1, 7] = float("nan")
    out, lse = c.prefill(bad, "bf16", "bf16", cu, T)
    assert torch.isnan(out[2, 1]).all()
    keep = torch.ones(2 * T, 4, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], lref[keep])
    # a key inside the chunk: the rows before it do not see it
    at = 200 - T + 3
    k = c.k[0][at:at + 1].clone()
    k[0, 1, 3] = float("nan")
    pk.kv_append_rope(c.pool, k.cuda(), c.v[0][at:at + 1].cuda(), pk.KV_BF16, torch.from_numpy(c.slots[0][at:at + 1]).cuda(), 1)
    out, lse = c.prefill(q, "bf16", "bf16", cu, T)
    assert torch.isnan(out[3:T, 2:]).all()
    keep = torch.ones(2 * T, 4, dtype=torch.bool, device="cuda")
    keep[3:T, 2:] = False
    assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], lref[keep])
    c.close()


@pytest.mark.parametrize("lens,T", [([3000, 200], 60), ([400, 300], 300)])
def test_prefill_wait_limit(lens, T):
    """As for the decode, with keys cut and whole: a wait that runs out is reported, the
    next call is right."""
    c = Cache(lens, 2, 128, seed=15)
    cu = [0, T, 2 * T]
    q = c.queries(2 * T, 8, "bf16")
    n = pk.kv_prefill_i4_workspace_size(c.pool, 2, 8, c.width, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    t_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pk.kv_debug_set_wait_limit_ns(0)
    try:
        seen = 0
        for _ in range(3):
            pk.paged_prefill_attention_i4(c.pool, q, pk.KV_BF16, t_cu, 2 * T, T, c.t_tables, c.width, c.t_lens, 2, 8, 0.1, out,
                                          pk.KV_BF16, None, ws, n)
            torch.cuda.synchronize()
            seen |= pk.kv_get_device_error(c.pool)
        assert seen == 0x4
    finally:
        pk.kv_debug_set_wait_limit_ns(pk.KV_WAIT_LIMIT_DEFAULT_NS)
    got, lse = c.prefill(q, "bf16", "bf16", cu, T)
    check_prefill(c, q, got, lse, cu, "bf16")
    c.close()


@pytest.mark.parametrize("T", [8, 64])
def test_prefill_captured_while_lengths_change(T):
    """The columns' runs and the list of items are made on the device: a replayed graph
    follows the lengths and the chunks' bounds as a new call would."""
    c = Cache([4000, 300, 900], 2, 128, seed=12)
    q = c.queries(3 * T, 8, "bf16")
    cu, lens = torch.tensor([0, T, 2 * T, 3 * T], dtype=torch.int32, device="cuda"), c.t_lens.clone()
    out, lse = torch.empty_like(q), torch.empty(3 * T, 8, device="cuda")
    n = pk.kv_prefill_i4_workspace_size(c.pool, 3, 8, c.width, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(o, l):
        pk.paged_prefill_attention_i4(c.pool, q, pk.KV_BF16, cu, 3 * T, T, c.t_tables, c.width, lens, 3, 8, 128 ** -0.5, o, pk.KV_BF16, l,
                                      ws, n)

    step(out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, lse)
    for now, bounds in (([4000, 300, 900], [0, T, 2 * T, 3 * T]), ([T, 300, 70], [0, T, T + 1, 2 * T + 1]),
                        ([3000, 0, 900], [0, 3, 3, 3 + T]), ([4000, 300, 900], [0, T, 2 * T, 3 * T])):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        cu.copy_(torch.tensor(bounds, dtype=torch.int32))
        out.fill_(7)
        lse.fill_(7)
        g.replay()
        again, lse2 = torch.full_like(out, 7), torch.full_like(lse, 7)
        step(again, lse2)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        for b, m in enumerate(now):
            rows = slice(bounds[b], bounds[b + 1])
            t = bounds[b + 1] - bounds[b]
            if t:
                ref = attend(f64(q)[rows], c.kv[b][:m], c.vv[b][:m], 128 ** -0.5, [m - t + i + 1 for i in range(t)])
                check_attention(f64(out)[rows], f64(lse)[rows], ref, 128 ** -0.5, m, "bf16", 2.0 ** -11, f"seq {b}", floor=2.0 ** -24)
    assert pk.kv_get_device_error(c.pool) == 0
    c.close()


def test_prefill_past_32_bit_offsets():
    """Expanded tiles past 2^32 bytes: a wide table, mostly unused."""
    c = Cache([700], 8, 128, seed=5)
    width = 48000
    tables = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    tables[0, :c.width] = tables[2, :c.width] = c.t_tables[0]
    lens = torch.tensor([700, 0, 650], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 30, 30, 130], dtype=torch.int32, device="cuda")
    q = c.queries(130, 8, "f16")
    out, lse = torch.empty(130, 8, 128, device="cuda"), torch.empty(130, 8, device="cuda")
    n = pk.kv_prefill_i4_workspace_size(c.pool, 3, 8, width, 100)
    assert n > 2 * 2 ** 32
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    pk.paged_prefill_attention_i4(c.pool, q, pk.KV_F16, cu, 130, 100, tables, width, lens, 3, 8, 128 ** -0.5, out, pk.KV_F32, lse, ws, n)
    for rows, m in ((slice(0, 30), 700), (slice(30, 130), 650)):
        t = rows.stop - rows.start
        ref = attend(f64(q)[rows], c.kv[0][:m], c.vv[0][:m], 128 ** -0.5, [m - t + i + 1 for i in range(t)])
        check_attention(f64(out)[rows], f64(lse)[rows], ref, 128 ** -0.5, m, "f32", 2.0 ** -11, floor=2.0 ** -24)
    assert pk.kv_get_device_error(c.pool) == 0
    c.close()


@pytest.mark.parametrize("T", [4, 400])
def test_prefill_without_a_table_column(T):
    """No sequence can have a key: each with a query is left out and flagged."""
    c = Cache([20], 2, 128, seed=2)
    n = pk.kv_prefill_i4_workspace_size(c.pool, 1, 4, 0, T)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    q = c.queries(T, 4, "bf16")
    out = torch.full_like(q, 7)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for length in (0, T):
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        pk.paged_prefill_attention_i4(c.pool, q, pk.KV_BF16, cu, T, T, c.t_tables, 0, lens, 1, 4, 1.0, out, pk.KV_BF16, None, ws, n)
        assert pk.kv_get_device_error(c.pool) == 0x1
        assert torch.all(out == 7)
    c.close()


def test_refusals():
    c = Cache([40], 2, 128, seed=1)
    d64 = Cache([40], 2, 64, seed=1)
    bf = pk.kv_pool_create(4, 16, 2, 128, pk.KV_BF16)
    t = torch.zeros(1 << 14, dtype=torch.float32, device="cuda")
    i = torch.zeros(64, dtype=torch.int32, device="cuda")

    def refused(status, f, *a, **k):
        with pytest.raises(pk.KVError) as e:
            f(*a, **k)
        assert e.value.status == status, (e.value.status, a, k)

    def dec(pool=c.pool, q=t, qt=pk.KV_BF16, tab=i, mb=3, lens=i, B=1, hq=4, out=t, ot=pk.KV_F32, **k):
        return (pk.paged_decode_attention_i4, pool, q, qt, tab, mb, lens, B, hq, 1.0, out, ot), k

    for status, case in ((-3, dec(pool=bf)), (-3, dec(qt=pk.KV_F32)), (-3, dec(ot=pk.KV_F16)), (-1, dec(hq=3)), (-1, dec(hq=0)),
                         (-3, dec(hq=18)), (-1, dec(q=None)), (-1, dec(out=None)), (-1, dec(lens=None)), (-1, dec(tab=None)),
                         (-1, dec(B=-1)), (-1, dec(mb=-1)), (-1, dec(num_splits=-1)), (-1, dec(q=t.data_ptr() + 8)),
                         (-1, dec(mb=64, num_splits=3)), (-1, dec(mb=64, num_splits=3, workspace=t, workspace_bytes=64)),
                         (-3, dec(B=70000))):
        refused(status, *case[0], **case[1])

    def pre(pool=c.pool, q=t, qt=pk.KV_BF16, cu=i, rows=1, most=400, tab=i, mb=3, lens=i, B=1, hq=4, out=t, ot=pk.KV_F32, ws=t,
            n=1 << 16, scale=1.0):
        return pk.paged_prefill_attention_i4, pool, q, qt, cu, rows, most, tab, mb, lens, B, hq, scale, out, ot, None, ws, n

    for status, case in ((-3, pre(pool=bf)), (-3, pre(pool=d64.pool)), (-3, pre(qt=pk.KV_F32)), (-3, pre(ot=pk.KV_F16)),
                         (-1, pre(hq=3)), (-1, pre(q=None)), (-1, pre(cu=None)), (-1, pre(tab=None)), (-1, pre(lens=None)),
                         (-1, pre(out=None)), (-1, pre(ws=None)), (-1, pre(n=1000)), (-1, pre(rows=-1)), (-1, pre(most=-1)),
                         (-1, pre(ws=t.data_ptr() + 8)), (-3, pre(B=70000)), (-1, pre(scale=0.0)), (-1, pre(scale=-1.0)),
                         (-1, pre(scale=float("nan")))):
        refused(status, *case)
    refused(-3, pk.kv_prefill_i4_workspace_size, bf, 1, 4, 3, 40)
    refused(-3, pk.kv_prefill_i4_workspace_size, d64.pool, 1, 4, 3, 40)
    refused(-1, pk.kv_prefill_i4_workspace_size, c.pool, 1, 3, 3, 40)
    refused(-3, pk.kv_prefill_i4_workspace_size, c.pool, 70000, 4, 3, 40)
    pk.paged_decode_attention_i4(c.pool, None, pk.KV_BF16, None, 3, None, 0, 4, 1.0, None, pk.KV_F32)  # nothing to do
    assert pk.kv_get_device_error(c.pool) == 0
    for x in (c, d64):
        x.close()
    pk.kv_pool_destroy(bf)


# ------------------------------------------------------- a run of them together
@pytest.mark.parametrize("q_dtype", ["bf16", "f16"])
def test_serving_run(q_dtype):
    """A prompt in two chunks, then decode steps captured once and replayed, on a pool
    managed by its allocator, the rotation applied on the way."""
    require_cuda()
    B, hq, hkv, d, width, base = 3, 8, 2, 128, 32, 400
    rng = np.random.default_rng(12)
    prompts = [70, 150, 33]
    pool = pk.kv_pool_create(64, 16, hkv, d, pk.KV_I4)
    pk.kv_pool_set_i4_scales(pool, 0.5, 0.5)
    alloc = pk.kv_pool_allocator(pool)
    tables, nblocks, lens = np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int64)
    cow = np.zeros(B, np.int32), np.zeros(B, np.int32)
    table = rope_table(base, d)
    t_table = torch.from_numpy(table).cuda()
    ks, vs = [np.zeros((0, hkv, d))] * B, [np.zeros((0, hkv, d))] * B

    def new_tokens(n_new):
        T = int(sum(n_new))
        slots = np.zeros(T, np.int64)
        pk.kv_prepare_append_batch(alloc, tables, nblocks, lens, np.asarray(n_new, np.int32), slots, *cow)
        pos = np.concatenate([lens[b] + np.arange(n) for b, n in enumerate(n_new)]).astype(np.int32)
        qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to(TORCH[q_dtype])
        at = 0
        for b, n in enumerate(n_new):
            rows = qkv[at:at + n]
            k = rotate32(rows[:, hq:hq + hkv].float().numpy(), table[pos[at:at + n]], d, False)
            ks[b] = np.concatenate([ks[b], stored(k, 0.5)])
            vs[b] = np.concatenate([vs[b], stored(f64(rows[:, hq + hkv:]), 0.5)])
            at += n
        q = torch.from_numpy(rotate32(qkv[:, :hq].float().numpy(), table[pos], d, False)).to(TORCH[q_dtype])
        lens[:] += n_new
        return qkv, slots, pos, q

    def append(qkv, slots, pos, q_out):
        row = (hq + 2 * hkv) * d
        pk.kv_append_rope(pool, qkv[:, hq:], qkv[:, hq + hkv:], KV[q_dtype], slots, len(slots), row, row, pos, t_table, base, d,
                          False, qkv, q_out, hq, row)

    for part in (0.5, 1.0):  # chunked prefill
        n_new = [int(p * part) - int(lens[b]) for b, p in enumerate(prompts)]
        qkv, slots, pos, q_ref = new_tokens(n_new)
        T = len(slots)
        q = torch.empty(T, hq, d, dtype=TORCH[q_dtype], device="cuda")
        append(qkv.cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), q)
        assert torch.equal(q.cpu(), q_ref)
        cu = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        n = pk.kv_prefill_i4_workspace_size(pool, B, hq, width, max(n_new))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        out = torch.empty(T, hq, d, dtype=TORCH[q_dtype], device="cuda")
        lse = torch.empty(T, hq, device="cuda")
        pk.paged_prefill_attention_i4(pool, q, KV[q_dtype], torch.from_numpy(cu).cuda(), T, max(n_new),
                                      torch.from_numpy(tables).cuda(), width, torch.from_numpy(lens.astype(np.int32)).cuda(), B,
                                      hq, d ** -0.5, out, KV[q_dtype], lse, ws, n)
        torch.cuda.synchronize()
        for b in range(B):
            rows = slice(cu[b], cu[b + 1])
            ref = attend(f64(q_ref)[rows], ks[b], vs[b], d ** -0.5, [int(lens[b]) - n_new[b] + i + 1 for i in range(n_new[b])])
            check_attention(f64(out)[rows], f64(lse)[rows], ref, d ** -0.5, int(lens[b]), q_dtype, 2.0 ** -11, floor=2.0 ** -24)

    # decode steps: fixed buffers, the step captured once
    buf = dict(qkv=torch.empty(B, hq + 2 * hkv, d, dtype=TORCH[q_dtype], device="cuda"),
               slots=torch.empty(B, dtype=torch.int64, device="cuda"), pos=torch.empty(B, dtype=torch.int32, device="cuda"),
               tables=torch.empty(B, width, dtype=torch.int32, device="cuda"), lens=torch.empty(B, dtype=torch.int32, device="cuda"),
               q=torch.empty(B, hq, d, dtype=TORCH[q_dtype], device="cuda"), out=torch.empty(B, hq, d, dtype=TORCH[q_dtype], device="cuda"),
               lse=torch.empty(B, hq, device="cuda"))
    splits = 4
    n = pk.kv_decode_workspace_size(B, hq, hkv, d, width, splits)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        append(buf["qkv"], buf["slots"], buf["pos"], buf["q"])
        pk.paged_decode_attention_i4(pool, buf["q"], KV[q_dtype], buf["tables"], width, buf["lens"], B, hq, d ** -0.5, buf["out"],
                                     KV[q_dtype], buf["lse"], splits, ws, n)

    graph = None
    for i in range(20):
        qkv, slots, pos, q_ref = new_tokens([1] * B)
        for name, x in (("qkv", qkv), ("slots", torch.from_numpy(slots)), ("pos", torch.from_numpy(pos)),
                        ("tables", torch.from_numpy(tables)), ("lens", torch.from_numpy(lens.astype(np.int32)))):
            buf[name].copy_(x)
        if i == 0:
            step()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            ref = attend(f64(q_ref)[b:b + 1], ks[b], vs[b], d ** -0.5, [int(lens[b])])
            check_attention(f64(buf["out"])[b:b + 1], f64(buf["lse"])[b:b + 1], ref, d ** -0.5, int(lens[b]), q_dtype, 2.0 ** -11,
                            f"step {i}")
    assert pk.kv_get_device_error(pool) == 0
    pk.kv_pool_destroy(pool)
