"""kv_append_rope and kv_read_tokens on the GPU: the rotation against 64 bits,
what a 4-bit pool stores against the format's definition (equal, value by value),
everything that is not rotated bit by bit, and what is left out."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _i4 import HALF_FLOOR, HALF_STEP, KV, TORCH, f64, raw_bytes, rope_table, rotate32, stored

pytestmark = pytest.mark.gpu


def _inputs(T, hq, hkv, d, dtype, seed, max_pos=300):
    rng = np.random.default_rng(seed)
    qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to(TORCH[dtype]).cuda()
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    nb = T // 16 + 3
    slots = rng.permutation(nb * 16)[:T].astype(np.int64)
    return qkv, pos, slots, nb


def _rotated64(x, cs, rot, interleaved):
    x = f64(x)
    c, s = cs[:, None, :rot // 2].astype(np.float64), cs[:, None, rot // 2:].astype(np.float64)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y, mag = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 48), (64, 64), (64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv", [(1, 8, 1), (37, 7, 1), (700, 12, 4)])
def test_rotary_append(dtype, d, rot, interleaved, T, hq, hkv):
    require_cuda()
    qkv, pos, slots, nb = _inputs(T, hq, hkv, d, dtype, 11)
    if T > 3:
        slots[2] = -1                      # a padding token: rotated, not stored
    table = rope_table(300, rot)
    pool = pk.kv_pool_create(nb, 16, hkv, d, KV[dtype])
    e = qkv.element_size()
    before = []
    for ptr in pk.kv_pool_ptrs(pool):
        raw_bytes(ptr, nb * hkv * 16 * d * e).fill_(0x35)
        before.append(raw_bytes(ptr, nb * hkv * 16 * d * e).view(TORCH[dtype]).view(nb, hkv, 16, d))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    q_out = torch.empty(T, hq, d, dtype=TORCH[dtype], device="cuda")
    row = (hq + 2 * hkv) * d
    t_slots = torch.from_numpy(slots).cuda()
    pk.kv_append_rope(pool, k, v, KV[dtype], t_slots, T, row, row, torch.from_numpy(pos).cuda(),
                      torch.from_numpy(table).cuda(), 300, rot, interleaved, q, q_out, hq, row)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0
    cs = table[pos]
    for got, x in ((f64(q_out), q), (None, k)):
        ref, mag = _rotated64(x, cs, rot, interleaved)
        if got is None:
            ok = slots >= 0
            got = f64(before[0])[slots[ok] // 16, :, slots[ok] % 16]
            ref, mag = ref[ok], mag[ok]
        # two products and a sum in fp32 (three roundings of the magnitudes), one of the type
        tol = mag * 3 * 2.0 ** -24 * (1 + HALF_STEP[dtype]) + HALF_STEP[dtype] * np.abs(ref) + HALF_FLOOR[dtype]
        tol[..., rot:] = 0                 # moved bit by bit
        assert np.all(np.abs(got - ref) <= tol)
    ok = slots >= 0
    assert torch.equal(before[1][torch.from_numpy(slots[ok] // 16).cuda(), :, torch.from_numpy(slots[ok] % 16).cuda()],
                       v[torch.from_numpy(ok).cuda()])
    used = np.zeros((nb, 16), bool)
    used[slots[ok] // 16, slots[ok] % 16] = True
    for x in before:                       # the other slots as they were
        rest = x.transpose(1, 2)[torch.from_numpy(~used).cuda()].contiguous().view(torch.uint8)
        assert torch.all(rest == 0x35)
    # the way back
    ko, vo = (torch.zeros(T, hkv, d, dtype=TORCH[dtype], device="cuda").fill_(3) for _ in "kv")
    pk.kv_read_tokens(pool, t_slots, T, ko, vo, KV[dtype])
    assert torch.equal(vo[torch.from_numpy(ok).cuda()], v[torch.from_numpy(ok).cuda()])
    assert torch.all(vo[torch.from_numpy(~ok).cuda()] == 3) and torch.all(ko[torch.from_numpy(~ok).cuda()] == 3)
    pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_in_place_equals_out_of_place(interleaved):
    require_cuda()
    qkv, pos, slots, nb = _inputs(65, 8, 2, 128, "bf16", 3)
    table, t_pos, t_slots = torch.from_numpy(rope_table(300, 64)).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    pool = pk.kv_pool_create(nb, 16, 2, 128, pk.KV_BF16)
    row = 12 * 128
    q = qkv[:, :8]
    out = torch.empty(65, 8, 128, dtype=torch.bfloat16, device="cuda")
    args = (pool, qkv[:, 8:10], qkv[:, 10:], pk.KV_BF16, t_slots, 65, row, row, t_pos, table, 300, 64, interleaved)
    pk.kv_append_rope(*args, q, out, 8, row)
    kv = qkv[:, 8:].clone()
    pk.kv_append_rope(*args, q, q, 8, row)
    torch.cuda.synchronize()
    assert torch.equal(out, q) and torch.equal(kv, qkv[:, 8:])
    pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("pool_type", ["bf16", "i4"])
def test_bad_slots_and_positions_are_left_out_and_flagged(pool_type):
    require_cuda()
    T, hq, hkv, d = 5, 4, 2, 128
    qkv, pos, slots, nb = _inputs(T, hq, hkv, d, "bf16", 4)
    pos[1], pos[3] = -1, 300
    slots[2] = nb * 16
    pool = pk.kv_pool_create(nb, 16, hkv, d, pk.KV_BF16 if pool_type == "bf16" else pk.KV_I4)
    if pool_type == "bf16":
        views = [raw_bytes(ptr, nb * hkv * 16 * d * 2) for ptr in pk.kv_pool_ptrs(pool)]
    else:  # K and V tiles alternate in one array
        views = [raw_bytes(pk.kv_pool_ptrs(pool)[0], nb * hkv * 18 * d)]
    for x in views:
        x.fill_(0x35)
    q_out = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda").fill_(9)
    row = (hq + 2 * hkv) * d
    pk.kv_append_rope(pool, qkv[:, hq:], qkv[:, hq + hkv:], pk.KV_BF16, torch.from_numpy(slots).cuda(), T, row, row,
                      torch.from_numpy(pos).cuda(), torch.from_numpy(rope_table(300, 128)).cuda(), 300, 128, False,
                      qkv, q_out, hq, row)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0x2 | 0x20
    assert torch.all(q_out[[1, 3]] == 9) and not torch.any(q_out[[0, 2, 4]] == 9)
    touched = sum(int((x != 0x35).sum()) for x in views)
    two_tokens = 2 * 2 * hkv * (d * 2 if pool_type == "bf16" else d * 9 // 16)
    assert two_tokens * 0.9 < touched <= two_tokens  # tokens 0 and 4 only (a byte may happen to be 0x35)
    pk.kv_pool_destroy(pool)


def _hard_rows(T, hkv, d, dtype, rng):
    """Rows full of what quantising gets wrong: ties, zeros, tiny and huge values."""
    x = rng.standard_normal((T, hkv, d)).astype(np.float32)
    x[0] = 0
    if T > 8:
        x[1] = np.arange(hkv * d).reshape(hkv, d) % 29 / 4 - 3.5      # quotients on borders
        x[2] = np.round(x[2] * 8) / 8
        x[3] = x[3] * 1e-4                                          # scales below e4m3's normal range
        x[4] = x[4] * 1e-7                                          # scales that round to zero
        x[5] = x[5] * 2000                                          # past the largest value
        x[6] = np.sign(x[6]) * 7 * 2.0 ** rng.integers(-12, 12, (hkv, d))
        x[7] = np.repeat(rng.integers(1, 113, (hkv, d // 16)) * 0.4375, 16, 1)  # maxima between two scales
    return torch.from_numpy(x).to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("T,hkv", [(1, 1), (33, 3), (900, 8)])
def test_i4_store_is_what_the_format_defines(dtype, d, T, hkv):
    require_cuda()
    rng = np.random.default_rng(d + T)
    k, v = _hard_rows(T, hkv, d, dtype, rng), _hard_rows(T, hkv, d, dtype, rng)
    nb = T // 16 + 2
    slots = torch.from_numpy(rng.permutation(nb * 16)[:T].astype(np.int64)).cuda()
    pool = pk.kv_pool_create(nb, 16, hkv, d, pk.KV_I4)
    pk.kv_pool_set_i4_scales(pool, 0.25, 2.0)
    pk.kv_append_rope(pool, k.cuda(), v.cuda(), KV[dtype], slots, T)
    ref_k, ref_v = stored(f64(k), 0.25), stored(f64(v), 2.0)
    for out in ("f32", "bf16", "f16"):
        ko, vo = (torch.empty(T, hkv, d, dtype=TORCH[out], device="cuda") for _ in "kv")
        pk.kv_read_tokens(pool, slots, T, ko, vo, KV[out])
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(pool) == 0
        np.testing.assert_array_equal(f64(ko), ref_k)
        np.testing.assert_array_equal(f64(vo), ref_v)
    pk.kv_pool_destroy(pool)


def test_i4_nan_and_infinity():
    require_cuda()
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((4, 2, 128)).astype(np.float32))
    x[0, 0, 3] = float("nan")
    x[1, 1, 20], x[1, 1, 40] = float("inf"), -float("inf")
    pool = pk.kv_pool_create(1, 16, 2, 128, pk.KV_I4)
    slots = torch.arange(4).cuda()
    pk.kv_append_rope(pool, x.cuda(), x.cuda(), pk.KV_F32, slots, 4)
    ko, vo = (torch.empty(4, 2, 128, device="cuda") for _ in "kv")
    pk.kv_read_tokens(pool, slots, 4, ko, vo, pk.KV_F32)
    ref = stored(f64(x))
    assert np.isnan(ref).sum() == 16 and np.abs(ref[1, 1]).max() == 3136
    np.testing.assert_array_equal(f64(ko), ref)
    np.testing.assert_array_equal(f64(vo), ref)
    pk.kv_pool_destroy(pool)


@pytest.mark.parametrize("dtype,d,rot,interleaved", [("bf16", 128, 128, False), ("f16", 64, 32, True), ("f32", 128, 48, False)])
def test_i4_stores_the_rotated_key(dtype, d, rot, interleaved):
    require_cuda()
    T, hq, hkv = 203, 6, 3
    qkv, pos, slots, nb = _inputs(T, hq, hkv, d, dtype, 21)
    table = rope_table(300, rot)
    pool = pk.kv_pool_create(nb, 16, hkv, d, pk.KV_I4)
    q_out = torch.empty(T, hq, d, dtype=TORCH[dtype], device="cuda")
    row = (hq + 2 * hkv) * d
    t_slots = torch.from_numpy(slots).cuda()
    pk.kv_append_rope(pool, qkv[:, hq:], qkv[:, hq + hkv:], KV[dtype], t_slots, T, row, row, torch.from_numpy(pos).cuda(),
                      torch.from_numpy(table).cuda(), 300, rot, interleaved, qkv, q_out, hq, row)
    ko, vo = (torch.empty(T, hkv, d, device="cuda") for _ in "kv")
    pk.kv_read_tokens(pool, t_slots, T, ko, vo, pk.KV_F32)
    k32 = qkv[:, hq:hq + hkv].float().cpu().numpy()
    np.testing.assert_array_equal(f64(ko), stored(rotate32(k32, table[pos], rot, interleaved)))
    np.testing.assert_array_equal(f64(vo), stored(f64(qkv[:, hq + hkv:])))
    # the same rotation as a 16/32-bit pool's append gives q
    ref = torch.from_numpy(rotate32(qkv[:, :hq].float().cpu().numpy(), table[pos], rot, interleaved)).to(TORCH[dtype])
    bad = (q_out.cpu() != ref).nonzero()
    assert not len(bad), (len(bad), bad[:4], q_out.cpu()[tuple(bad[0])], ref[tuple(bad[0])])
    pk.kv_pool_destroy(pool)


def test_two_tokens_of_a_pair_stored_apart():
    """Neighbouring tokens share words of the V tile: writing one keeps the other."""
    require_cuda()
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((16, 2, 128)).astype(np.float32)).cuda()
    pool = pk.kv_pool_create(1, 16, 2, 128, pk.KV_I4)
    for t in rng.permutation(16):
        pk.kv_append_rope(pool, x[t:t + 1], x[t:t + 1], pk.KV_F32, torch.tensor([int(t)]).cuda(), 1)
    ko, vo = (torch.empty(16, 2, 128, device="cuda") for _ in "kv")
    pk.kv_read_tokens(pool, torch.arange(16).cuda(), 16, ko, vo, pk.KV_F32)
    np.testing.assert_array_equal(f64(ko), stored(f64(x)))
    np.testing.assert_array_equal(f64(vo), stored(f64(x)))
    pk.kv_pool_destroy(pool)


def test_i4_blocks_copy_and_swap():
    require_cuda()
    rng = np.random.default_rng(6)
    T, hkv, d = 48, 2, 64
    x = torch.from_numpy(rng.standard_normal((T, hkv, d)).astype(np.float32)).cuda()
    pool = pk.kv_pool_create(8, 16, hkv, d, pk.KV_I4)
    pk.kv_append_rope(pool, x, -x, pk.KV_F32, torch.arange(T).cuda(), T)
    pk.kv_copy_blocks(pool, torch.tensor([1], dtype=torch.int32).cuda(), torch.tensor([5], dtype=torch.int32).cuda(), 1)
    n = pk.kv_swap_bytes(pool, 2)
    assert n == 2 * 2 * hkv * 9 * d
    buf = torch.empty(n, dtype=torch.uint8).pin_memory()
    pk.kv_swap_out(pool, torch.tensor([0, 2], dtype=torch.int32).cuda(), 2, buf)
    pk.kv_swap_in(pool, torch.tensor([6, 7], dtype=torch.int32).cuda(), 2, buf)
    want = torch.cat([torch.arange(16, 32), torch.arange(0, 16), torch.arange(32, 48)])
    got = torch.arange(5 * 16, 8 * 16)
    a = [torch.empty(48, hkv, d, device="cuda") for _ in range(4)]
    pk.kv_read_tokens(pool, want.cuda(), 48, a[0], a[1], pk.KV_F32)
    pk.kv_read_tokens(pool, got.cuda(), 48, a[2], a[3], pk.KV_F32)
    torch.cuda.synchronize()
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3]) and torch.equal(a[0], -a[1])
    # copy on write of a shared block
    ids = np.zeros(1, np.int32)
    pk.kv_alloc_blocks(pool, ids)
    pk.kv_share_blocks(pool, ids)
    bid, copied = pk.kv_cow_if_shared(pool, int(ids[0]))
    assert copied and bid != ids[0]
    pk.kv_read_tokens(pool, torch.arange(16).cuda() + 16 * bid, 16, a[2], a[3], pk.KV_F32)
    pk.kv_read_tokens(pool, torch.arange(16).cuda() + 16 * int(ids[0]), 16, a[0], a[1], pk.KV_F32)
    torch.cuda.synchronize()
    assert torch.equal(a[0][:16], a[2][:16])
    pk.kv_pool_destroy(pool)


def test_refusals():
    require_cuda()
    t = torch.zeros(1 << 16, dtype=torch.float32, device="cuda")
    idx = torch.zeros(64, dtype=torch.int64, device="cuda")
    bf = pk.kv_pool_create(4, 16, 2, 128, pk.KV_BF16)
    i4 = pk.kv_pool_create(4, 16, 2, 128, pk.KV_I4)

    def refused(status, f, *a, **k):
        with pytest.raises(pk.KVError) as e:
            f(*a, **k)
        assert e.value.status == status, (e.value.status, a, k)

    ok = dict(positions=idx, cos_sin=t, max_position=8, rot_dim=32)
    refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_F16, idx, 1, **ok)       # not the pool's type
    refused(-3, pk.kv_append_rope, i4, t, t, pk.KV_I4, idx, 1, **ok)
    refused(-3, pk.kv_append_rope, i4, t, t, 9, idx, 1, **ok)
    refused(-1, pk.kv_append_rope, bf, None, t, pk.KV_BF16, idx, 1, **ok)
    refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_BF16, None, 1, **ok)
    refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_BF16, idx, -1, **ok)
    for bad in (dict(rot_dim=8), dict(rot_dim=144), dict(rot_dim=-16), dict(max_position=0), dict(positions=None),
                dict(cos_sin=None), dict(k_stride=128), dict(v_stride=257), dict(k_stride=-256),
                dict(q=t), dict(q=t, q_out=t), dict(q=t, q_out=t, num_q_heads=4, q_stride=100),
                dict(q=t, q_out=t, num_q_heads=4, q_stride=1024, q_out_stride=512)):
        refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_BF16, idx, 1, **{**ok, **bad})
    refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_BF16, idx, 1, q=t, q_out=t, num_q_heads=4)  # q without a rotation
    refused(-1, pk.kv_append_rope, bf, t.data_ptr() + 8, t, pk.KV_BF16, idx, 1, **ok)          # alignment
    refused(-1, pk.kv_append_rope, bf, t, t, pk.KV_BF16, idx, 1, **{**ok, "cos_sin": t.data_ptr() + 4})
    refused(-1, pk.kv_read_tokens, bf, idx, 1, t, t, pk.KV_F32)
    refused(-3, pk.kv_read_tokens, i4, idx, 1, t, t, pk.KV_I4)
    refused(-1, pk.kv_read_tokens, i4, idx, 1, None, t, pk.KV_F32)
    refused(-1, pk.kv_read_tokens, i4, idx, -1, t, t, pk.KV_F32)
    refused(-3, pk.kv_pool_set_i4_scales, bf, 1.0, 1.0)
    for bad in (0.0, -1.0, 3.0, float("nan"), float("inf"), 2.0 ** 40, 2.0 ** -40):
        refused(-1, pk.kv_pool_set_i4_scales, i4, bad, 1.0)
        refused(-1, pk.kv_pool_set_i4_scales, i4, 1.0, bad)
    refused(-3, pk.kv_append, i4, t, t, idx, 1)
    i32 = torch.zeros(64, dtype=torch.int32, device="cuda")
    refused(-3, pk.paged_decode_attention, i4, t, i32, 1, i32, 1, 4, 1.0, t, pk.KV_F32)
    refused(-3, pk.paged_decode_attention_noalloc, i4, t, i32, 1, i32, 1, 4, 1.0, t, pk.KV_F32)
    refused(-3, pk.paged_append_and_decode, i4, t, t, t, idx, i32, 1, i32, 1, 4, 1.0, t, pk.KV_F32)
    refused(-3, pk.paged_prefill_attention, i4, t, i32, 1, 1, i32, 1, i32, 1, 4, 1.0, t, pk.KV_F32)
    with pytest.raises(pk.KVError):
        pk.kv_contig_create(1, 16, 2, 128, pk.KV_I4)
    pk.kv_append_rope(bf, None, None, pk.KV_BF16, None, 0)  # nothing to do
    pk.kv_read_tokens(i4, None, 0, None, None, pk.KV_F32)
    assert pk.kv_get_device_error(bf) == 0 and pk.kv_get_device_error(i4) == 0
    pk.kv_pool_destroy(bf)
    pk.kv_pool_destroy(i4)


def test_append_and_read_captured_in_a_graph():
    require_cuda()
    qkv, pos, slots, nb = _inputs(64, 8, 2, 128, "bf16", 8)
    table, t_pos, t_slots = torch.from_numpy(rope_table(300, 128)).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    pool = pk.kv_pool_create(nb, 16, 2, 128, pk.KV_I4)
    q_out = torch.empty(64, 8, 128, dtype=torch.bfloat16, device="cuda")
    ko, vo = (torch.empty(64, 2, 128, device="cuda") for _ in "kv")
    row = 12 * 128

    def step():
        pk.kv_append_rope(pool, qkv[:, 8:], qkv[:, 10:], pk.KV_BF16, t_slots, 64, row, row, t_pos, table, 300, 128, False,
                          qkv, q_out, 8, row)
        pk.kv_read_tokens(pool, t_slots, 64, ko, vo, pk.KV_F32)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    new = torch.randn_like(qkv.float()).to(torch.bfloat16)
    qkv.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(ko), stored(rotate32(qkv[:, 8:10].float().cpu().numpy(), table.cpu().numpy()[pos], 128, False)))
    np.testing.assert_array_equal(f64(vo), stored(f64(qkv[:, 10:])))
    pk.kv_pool_destroy(pool)


def test_rotated_queries_reach_an_overlapping_decode():
    """With launch overlap on, a 16-bit decode reads its queries before the previous
    kernel has ended; it must see the ones this call wrote all the same."""
    require_cuda()
    B, hq, hkv, d, L = 64, 32, 8, 128, 900
    rng = np.random.default_rng(3)
    width = -(-(L + 1) // 16)
    pool = pk.kv_pool_create(B * width, 16, hkv, d, pk.KV_BF16)
    table, tables = torch.from_numpy(rope_table(L + 1, d)).cuda(), torch.arange(B * width, dtype=torch.int32).view(B, width).cuda()
    rows = torch.randn(B * L, hkv, d, device="cuda").to(torch.bfloat16)
    j = torch.arange(L)
    slots = (tables.cpu().long()[:, j // 16] * 16 + j % 16).reshape(-1).cuda()
    pk.kv_append_rope(pool, rows, rows, pk.KV_BF16, slots, B * L)
    lens = torch.full((B,), L + 1, dtype=torch.int32, device="cuda")
    new = (tables.long()[:, L // 16] * 16 + L % 16).contiguous()
    pos = torch.full((B,), L, dtype=torch.int32, device="cuda")
    n = pk.kv_decode_workspace_size(B, hq, hkv, d, width, 2)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    qkvs = [torch.from_numpy(rng.standard_normal((B, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(8)]
    row = (hq + 2 * hkv) * d

    def steps(overlap):
        pk.kv_pool_set_launch_overlap(pool, overlap)
        q = torch.zeros(B, hq, d, dtype=torch.bfloat16, device="cuda")
        outs = [torch.empty(B, hq, d, device="cuda") for _ in qkvs]
        for qkv, out in zip(qkvs, outs):  # one query buffer, rewritten by each step
            pk.kv_append_rope(pool, qkv[:, hq:], qkv[:, hq + hkv:], pk.KV_BF16, new, B, row, row, pos, table, L + 1, d, False, qkv, q,
                              hq, row)
            pk.paged_decode_attention(pool, q, tables, width, lens, B, hq, d ** -0.5, out, pk.KV_F32, None, 2, ws, n)
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(pool) == 0
        return outs

    plain = steps(False)
    for _ in range(5):
        for a, b in zip(plain, steps(True)):
            assert torch.equal(a, b)
    pk.kv_pool_destroy(pool)


def test_on_a_stream_of_its_own():
    require_cuda()
    qkv, pos, slots, nb = _inputs(65, 8, 2, 128, "f16", 13)
    pool = pk.kv_pool_create(nb, 16, 2, 128, pk.KV_I4)
    t_slots = torch.from_numpy(slots).cuda()
    k, v = qkv[:, 8:10].contiguous(), qkv[:, 10:].contiguous()
    ko, vo = (torch.empty(65, 2, 128, device="cuda") for _ in "kv")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pk.kv_append_rope(pool, k, v, pk.KV_F16, t_slots, 65, stream=s)          # given
    with torch.cuda.stream(s):
        pk.kv_read_tokens(pool, t_slots, 65, ko, vo, pk.KV_F32)              # current
    s.synchronize()
    np.testing.assert_array_equal(f64(ko), stored(f64(k)))
    np.testing.assert_array_equal(f64(vo), stored(f64(v)))
    pk.kv_pool_destroy(pool)
