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
