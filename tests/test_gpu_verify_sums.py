"""Draws of verification next to the borders between tokens, after rejections."""
import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


@pytest.fixture
def pool():
    require_cuda()
    p = pk.kv_pool_create(1, 16, 1, 64, pk.KV_F32)
    yield p
    pk.kv_pool_destroy(p)


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


HEAVY, LIGHT = 64, 65536


def two_rejections(seed):
    """p, q of 131072 tokens in fp32 (whole numbers of 2^-45, so as integers too) whose second residual is half on 64
    tokens and half on 65536 behind them; the last two tokens, with p = 0, are the drafts."""
    rng = np.random.default_rng(seed)
    vocab, s = 131072, 2.0 ** -11
    q, p = np.zeros(vocab, np.float32), np.zeros(vocab, np.float32)
    n = HEAVY + LIGHT
    q[:n] = rng.uniform(2.0 ** -18, 3 * 2.0 ** -18, n)
    q[:n] *= 0.5 / q[:n].sum(dtype=np.float64)
    rest = np.where(np.arange(n) < HEAVY, s / 4 / HEAVY, s / 4 / LIGHT) * rng.uniform(0.5, 1.5, n)
    p[:n] = (1 + s) * q[:n].astype(np.float64) + rest
    q[-2:] = 2.0 ** -10
    unit = 2.0 ** 45
    pi, qi = (x.astype(np.float64) * unit for x in (p, q))
    assert (pi == np.rint(pi)).all() and (qi == np.rint(qi)).all()
    return p, q, [int(x) for x in pi], [int(x) for x in qi]


def test_borders_after_two_rejections(pool):
    """W_2 = max(p - (1 + S_1) q, 0), S_1 = sum max(p - q, 0): exact in whole numbers of 2^-90 here.

    The kernel holds W_2 in whole numbers of 2^-45.  Rounded, 65600 weights err by at most half of one each and as often
    up as down: their sum by 75 (one standard deviation), of 2^33 that S_2 has.  Cut off, all would err by half of
    one in one direction, and the border between the 64 and the 65536 would lie 16000 below its place.  Numbers are drawn
    from 2000 to 30000 off the border on both sides: 25 standard deviations and more."""
    for seed in range(3):
        p, q, pi, qi = two_rejections(seed)
        vocab = len(p)
        s1 = sum(max(a - b, 0) for a, b in zip(pi, qi))
        w = [max(((a - b) << 45) - s1 * b, 0) for a, b in zip(pi, qi)]
        total, border = sum(w), sum(w[:HEAVY])
        assert 2 ** 32 < total >> 45 < 2 ** 34 and abs(border / total - 0.5) < 0.1
        u = [np.float32((border + off * 2 ** 45) / total) for off in
             (-30000, -14000, -8000, -5000, -3000, 3000, 5000, 8000, 14000, 30000)]
        want = []
        for x in u:
            # the first token whose running sum passes x * total, with x's exact value
            num, den = float(x).as_integer_ratio()
            point, run, at = num * total // den, 0, 0
            assert abs(point - border) > 2000 * 2 ** 45
            while run + w[at] <= point:
                run += w[at]
                at += 1
            want.append(at)
        b = len(u)
        rows = lambda x: torch.from_numpy(x).cuda().repeat(3 * b, 1)
        tokens = np.tile([0, vocab - 1, vocab - 2], b)
        count, path, out = ints(np.full(b, 7)), ints(np.full((b, 1), 7)), ints(np.full((b, 2), 7))
        pk.kv_verify_tree(pool, rows(p), rows(q), pk.KV_F32, vocab, ints(np.arange(0, 3 * b + 1, 3)), 3 * b, 3,
                          ints(np.tile([-1, 0, 0], b)), ints(tokens), torch.full((3 * b,), 0.5, device="cuda"),
                          torch.from_numpy(np.array(u)).cuda(), b, 1, count, path, out)
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(pool) == 0
        assert (count == 0).all() and (path == -1).all() and (out[:, 1] == -1).all()
        assert out[:, 0].tolist() == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("row", [(0.3, 0.1, 0.05, 0.05), (0.5, 0.25, 0.125, 0.125), (0.8, 0.1, 0.3, 0.3),
                                 (0.9975, 0.002, 0.0005, 0.0), (0.6, 0.2, 0.1, 0.0)])
def test_chosen_drafts_of_rows_of_any_sum(pool, dtype, row):
    """Without q a row counts as summing to one: after the draft of token 0 was rejected that of token 1 is
    accepted below p(1) / (1 - p(0)), then that of token 2 below p(2) / (1 - p(0) - p(1)), whatever the row sums to; the
    draw divides by what is left.  Numbers lie 2^-10 off each border, the fp64 tests 2^-50."""
    p = torch.zeros(1, 40, dtype=dtype)
    p[0, :4] = torch.tensor(row)
    p0, p1, p2, p3 = p[0, :4].double().tolist()
    one = 1 - 2.0 ** -24
    up = lambda x: min(one, x * (1 + 2.0 ** -10))
    second, third = p1 / (1 - p0), p2 / (1 - p0 - p1) if p0 + p1 < 1 else 2.0
    cases = [([p0 * (1 - 2.0 ** -10), one, one], 0.5, [0]), ([one, second * (1 - 2.0 ** -10), one], 0.5, [1])]
    if second < 1:
        cases.append(([one, up(second), min(one, third * (1 - 2.0 ** -10))], 0.5, [2]))
        if third < 1:
            left = p3 if p3 else p0 + p1 + p2   # nothing left: the whole row
            cases += [([one, up(second), up(third)], u, []) for u in (0.0, 0.25, 0.75, one)]
    b = len(cases)
    accept = np.array([[0.5, *c[0]] for c in cases], np.float32)
    count, path, out = ints(np.full(b, 7)), ints(np.full((b, 1), 7)), ints(np.full((b, 2), 7))
    pk.kv_verify_tree(pool, p.cuda().repeat(4 * b, 1), None, {4: pk.KV_F32, 2: pk.KV_BF16}[p.element_size()]
                      if dtype != torch.float16 else pk.KV_F16, 40, ints(np.arange(0, 4 * b + 1, 4)), 4 * b, 4,
                      ints(np.tile([-1, 0, 0, 0], b)), ints(np.tile([0, 0, 1, 2], b)), torch.from_numpy(accept).cuda().flatten(),
                      torch.tensor([c[1] for c in cases], dtype=torch.float32, device="cuda"), b, 1, count, path, out)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0
    assert path[:, 0].tolist() == [c[2][0] + 1 if c[2] else -1 for c in cases]
    for i, (_, u, way) in enumerate(cases):
        if way:
            assert out[i, 0] == way[0]
        elif p3:
            assert out[i, 0] == 3
        else:
            sums = np.cumsum([p0, p1, p2])
            assert out[i, 0] == int(np.searchsorted(sums, float(np.float32(u)) * sums[-1], side="right"))


def test_products_next_to_the_probability(pool):
    """u q(x) < p(x) decides exactly, where u q rounded to fp32 equals p too, down to numbers whose products lose
    bits below fp32's smallest: the expected side is that of whole numbers."""
    rng = np.random.default_rng(0)
    us, qs, ps = [], [], []
    for low in (-1, -60, -100, -120, -124, -125, -126, -127, -130, -140):
        for _ in range(60):
            u = np.float32(1 - 2.0 ** -24 * rng.integers(1, 2 ** int(rng.integers(1, 12))))
            q = np.float32(np.ldexp(1 + rng.random(), low - 1))
            exact = u.astype(np.float64) * q.astype(np.float64)
            near = exact.astype(np.float32)   # rounded to nearest
            for p in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))):
                us.append(u), qs.append(q), ps.append(p)
    # the product is below p by 2^-46 of it, which is below 2^-149
    us.append(np.float32(1 - 2.0 ** -23)), qs.append(np.float32(2.0 ** -126 * (1 + 2.0 ** -23))), ps.append(np.float32(2.0 ** -126))
    b = len(us)
    want = [float(u) * float(q) < float(p) for u, q, p in zip(us, qs, ps)]   # 48 bits: exact
    assert want[-1] and 0 < sum(want) < b
    assert sum(np.float32(u * q) == p for u, q, p in zip(us, qs, ps)) > 500
    p, q = torch.zeros(2 * b, 8), torch.zeros(2 * b, 8)
    p[:, 5], q[:, 5] = torch.from_numpy(np.repeat(ps, 2)), torch.from_numpy(np.repeat(qs, 2))
    p[:, 0] = 0.5
    count, path, out = ints(np.full(b, 7)), ints(np.full((b, 1), 7)), ints(np.full((b, 2), 7))
    pk.kv_verify_tree(pool, p.cuda(), q.cuda(), pk.KV_F32, 8, ints(np.arange(0, 2 * b + 1, 2)), 2 * b, 2, None,
                      ints(np.tile([0, 5], b)), torch.from_numpy(np.repeat(us, 2)).cuda(), torch.full((b,), 0.5, device="cuda"),
                      b, 1, count, path, out)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0
    assert count.bool().tolist() == want


@pytest.mark.parametrize("vocab,step", [(1000, -45), (1 << 17, -45), ((1 << 17) + 1, -44), (1 << 18, -44), ((1 << 18) + 1, -43),
                                        (1 << 19, -43), ((1 << 19) + 1, -42), (1 << 20, -42)])
def test_steps_of_a_draw(pool, vocab, step):
    """Entries of half a step count as nothing, those just above as one step."""
    p = torch.zeros(4, vocab)
    half = 2.0 ** (step - 1)
    p[0, :] = half                                  # nothing
    p[1, :], p[1, 77] = half, half * (1 + 2.0 ** -20)   # one step
    p[2, 3], p[2, 5], p[2, 900] = 2.0 ** step, half, 3 * half   # one, nothing, two (a tie, to even)
    p[3, 3], p[3, 900] = 2.0 ** step, 3 * half
    count, out = ints(np.full(4, 7)), ints(np.full((4, 1), 7))
    pk.kv_verify_tree(pool, p.cuda(), None, pk.KV_F32, vocab, ints(np.arange(5)), 4, 1, None, ints(np.zeros(4)),
                      torch.zeros(4, device="cuda"), torch.tensor([0.5, 0.9, 0.34, 0.33], device="cuda"), 4, 0, count, None, out)
    torch.cuda.synchronize()
    assert pk.kv_get_device_error(pool) == 0
    assert (count == 0).all() and out[:, 0].tolist() == [-1, 77, 900, 3]
