"""How tree attention holds its softmax weights: small ones under a large one, and each for itself."""
import math

import numpy as np
import pytest
import torch

from _gpu import require_cuda
from _tree import DT, HALF, TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


@pytest.mark.parametrize("dtype,out_dtype", [("f16", "f32"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("nodes", [3, 12, 30, 60])
@pytest.mark.parametrize("sink", [0, 5000])
@pytest.mark.parametrize("gap", [12, 14, 15, 16, 17, 18])
def test_small_weights_under_a_sink(dtype, out_dtype, nodes, sink, gap):
    """One key with a value of zero, n others `gap` (natural log) below it with values 1 and 0.75:
    out = value n w / (1 + n w), w = exp(-gap).

    Relative error.  The others' scores are 0, the sink's q.k is exact: its scaled score and the distance
    to the reference are off by 3 2^-24 gap, the exponential by 2^-22.  A weight in parts is off by 2^-22 of
    itself and, in fp16, by 2^-34 of the largest weight at most: 2^-34 / w.  The n equal products are added 16 at a
    time, one addition a part, each cut off by 2^-23 of the sum so far: 3 n / 16 2^-23 (fp32 pools: n 2^-24 is
    less than twice that).  The sum of weights: each tile's adds 2^-24 of it, n / 128 tiles.  Joining pieces and the
    division: 2^-21."""
    n = 8192
    case = TreeCase(dtype, 64, 1, 4, [n], [nodes], kind="star", seed=1)
    try:
        k, v = torch.zeros_like(case.k[0]), torch.ones_like(case.v[0])
        k[sink, :, 0] = gap
        v[:, :, 32:] = 0.75
        v[sink] = 0
        case.k[0], case.v[0], case.q = k, v, torch.zeros_like(case.q)
        case.q[:, :, 0] = 8.0   # times the scale of 1/8
        case.write(0)
        a = case.args(out_dtype)
        case.call(a)
        torch.cuda.synchronize()
        w = math.exp(-gap)
        got = a["out"].double().cpu().numpy()
        for node in range(nodes):
            others = n - 1 + (1 if node == 0 else 2)   # the node and the one above it
            want = others * w / (1 + others * w) * np.repeat([1.0, 0.75], 32)
            tol = 3 * gap * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -22 + 3 * n / 16 * 2.0 ** -23 + n / 128 * 2.0 ** -24 + 2.0 ** -21
            if dtype == "f16":
                tol += 2.0 ** -34 / w
            if out_dtype == "f16":
                tol += HALF["f16"]
                # an output below 2^-14 is a multiple of 2^-24
                tol += 2.0 ** -25 / want.min()
            assert (np.abs(got[node] - want) <= tol * want).all(), (node, got[node][0, [0, 63]], want[[0, 63]], tol)
    finally:
        case.close()


# Keys that are one in a dimension of their own, so that a query's entries are its scores (a product and
# zeros, exact), and values that let an output show single weights.
def one_hot_case(dtype, d, g, nodes, keys, cached, width, seed, small):
    """`keys` rows per dimension at places of `pos`; `small`: the second of a pair, by the
    first.  A table of 33 blocks or more lets a sequence be cut."""
    case = TreeCase(dtype, d, 2, g, [cached], [nodes], kind="star", seed=seed, width=width)
    rng = np.random.default_rng(seed)
    pos = rng.permutation(cached)[:keys * d].reshape(keys, d)
    k, v = torch.zeros_like(case.k[0]), torch.zeros_like(case.v[0])
    for j in range(keys):
        for i in range(d):
            k[int(pos[j, i]), :, i] = 8.0 * (small if j else 1.0)
    q = (torch.from_numpy(rng.uniform(-2.0, 1.5, (nodes, case.hq, d))) * (math.sqrt(d) / 8)).to(DT[dtype])
    case.k[0], case.q = k, q
    return case, k, v, pos


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [4, 13, 30, 70])
@pytest.mark.parametrize("cached,width", [(140, 0), (140, 33), (1500, 0)])
def test_every_weight_for_itself(dtype, d, nodes, cached, width):
    """Value i is one in dimension i alone, so out[i] is key i's share; out[i] / out[0] = exp(s_i - s_0) whatever
    the sum of weights is.

    Each of the two is off by: its distance to the reference, rounded below 2^4 log2 units, 2^-21 ln 2; the scaled
    scores, 3 2^-24 of |s_i - s_0| (their common part is the reference's, which cancels); the exponential,
    2^-22; the weight's parts, 2^-24 (three of bf16), 2^-22 (two of fp16); up to three parts added, 2^-23 each;
    the joining of pieces, 2^-22 and a product, copies of a row the same, and the division's product: 2^-20.
    Two parts of bf16 would be off by up to 2^-16, one of fp16 by 2^-11."""
    case, k, v, pos = one_hot_case(dtype, d, 4, nodes, 1, cached, width, seed=nodes, small=1.0)
    try:
        for i in range(d):
            v[int(pos[0, i]), :, i] = 1.0
        case.v[0] = v
        case.write(0)
        a = case.args("f32")
        case.call(a)
        torch.cuda.synchronize()
        got = a["out"].double().cpu().numpy()[:nodes]
        s = case.q.double().numpy() * 8.0 * case.scale
        want = np.exp(s - s[:, :, :1])
        err = np.abs(got / got[:, :, :1] - want) / want
        parts = {"bf16": 2.0 ** -24, "f16": 2.0 ** -22, "f32": 0.0}[dtype]
        tol = 2 * (2.0 ** -21 * math.log(2) + 2.0 ** -22 + parts + 3 * 2.0 ** -23 + 2.0 ** -20) + 3 * 2.0 ** -24 * np.abs(s - s[:, :, :1])
        assert (err <= tol).all(), (err.max(), tol.min())
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes", [4, 13, 30, 70])
@pytest.mark.parametrize("cached,width", [(300, 0), (300, 33), (1500, 0)])
def test_differences_of_weights(dtype, d, nodes, cached, width):
    """16-bit output: two keys a dimension, 1 / 128 apart in score, with values one and minus one, so that what the
    output's rounding loses is small beside the weights: out[i] = (w - w') / sum.

    Of (w + w') / sum: 2^-16 (two parts of bf16) or 2^-22 (of fp16) and the terms of the test above, 2^-18 in all; of
    out: the sum of n weights n 2^-24, and the rounding of the output.  One part of bf16 would be off by 2^-9, of fp16 by 2^-12."""
    small = 1 - 2.0 ** -7
    case, k, v, pos = one_hot_case(dtype, d, 4, nodes, 2, cached, width, seed=nodes, small=small)
    try:
        for i in range(d):
            v[int(pos[0, i]), :, i], v[int(pos[1, i]), :, i] = 1.0, -1.0
        case.v[0] = v
        case.write(0)
        a = case.args(dtype)
        case.call(a)
        torch.cuda.synchronize()
        got = a["out"].double().cpu().numpy()[:nodes]
        s = case.q.double().numpy() * 8.0 * case.scale
        w, w2 = np.exp(s), np.exp(s * small)
        own = np.full((nodes, 1), 2.0)   # scores of zero: the node and the one above it, the other keys
        own[0] = 1.0
        total = (w + w2).sum(2) + own + cached - 2 * d
        want = (w - w2) / total[:, :, None]
        parts = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22}[dtype]
        tol = (w + w2) / total[:, :, None] * (parts + 2.0 ** -18) + np.abs(want) * (HALF[dtype] + cached * 2.0 ** -24)
        if dtype == "f16":
            tol += 2.0 ** -25   # outputs below 2^-14
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("first,last,step,gap", [(2840, 4096, 2, 4), (2840, 4096, 2, 6), (8192, 16384, 8, 4), (8192, 16384, 8, 8),
                                                 (16384, 32768, 16, 8), (16384, 32768, 16, 16)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("nodes", [4, 30, 60])
def test_scores_beyond_the_steps_of_their_maximum(dtype, first, last, step, gap, sign, nodes):
    """Scores of 2^24 and more (log2 units): fp32 holds their maximum, and what is added to it or taken
    from it, in steps of 1 to 16 units.  All keys of a row have one score, of exact products in fp32, but one of the
    second tile's, `gap` above: out = 128 w / (1 + (n - 1) w), w = exp(-gap), for the 128 keys with a value of one.

    A row's keys share their reference, however it is rounded; their distances to it are exact but for one
    rounding, 2^-20 of the weight; the exponential, the parts (and 2^-34 of the largest weight in fp16), the sums of up
    to n = 400 keys and the joining of pieces: 2^-22, 2^-16 of bf16, n 2^-23, 2^-20.  gap times the scale is off by
    2^-23 of itself."""
    cached, g = 300, 4
    case = TreeCase(dtype, 64, 1, g, [cached], [nodes], kind="star", seed=1, width=33)
    try:
        k, v = torch.zeros_like(case.k[0]), torch.zeros_like(case.v[0])
        k[:, :, 0], k[200, :, 1] = 32768.0 * sign, gap
        v[:128] = 1.0
        q0 = np.random.default_rng(nodes).choice(np.arange(first, last, step), (nodes, g))
        q = torch.zeros_like(case.q)
        q[:, :, 0], q[:, :, 1] = torch.from_numpy(q0 // 8 * 8 if dtype != "bf16" else 1 << np.log2(q0).astype(int)), 8.0
        case.k[0], case.v[0], case.q = k, v, q
        case.write(0)
        a = case.args("f32")
        case.call(a)
        torch.cuda.synchronize()
        got, w = a["out"].double().cpu().numpy()[:nodes], math.exp(-gap)
        for i in range(nodes):
            n = cached + (1 if i == 0 else 2)
            want = 128 * w / (1 + (n - 1) * w)
            tol = 2.0 ** -20 + 2.0 ** -22 + 2.0 ** -16 + n * 2.0 ** -23 + 2.0 ** -20 + gap * 2.0 ** -23 + 2.0 ** -34 / w
            assert (np.abs(got[i] - want) <= tol * want).all(), (i, q[i, :, 0], got[i][:, 0], want)
    finally:
        case.close()
