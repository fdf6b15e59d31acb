"""Tree attention: what NaN and infinities in attended keys do, however small their weights."""
import math

import numpy as np
import pytest
import torch

from _gpu import require_cuda
from _tree import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("place", [5, 700, "node"])
@pytest.mark.parametrize("width,nodes", [(0, 4), (80, 4), (80, 40)])
def test_a_value_whose_weight_underflows(dtype, bad, place, width, nodes):
    """Key `place` has a score 400 below the first one's: its weight is zero in fp32.  Its value is NaN or infinite
    in three dimensions: a row that attends it is NaN or infinite there, and nowhere else."""
    case = TreeCase(dtype, 64, 2, 4, [900 if width else 400], [nodes], kind="star", seed=1, width=width)
    if place == 700 and not width:
        place = 300
    at = case.lens[0] - nodes + 2 if place == "node" else place   # node 2 sees itself and node 0
    try:
        k = torch.zeros_like(case.k[0])
        k[0, :, 0], k[at, :, 0] = 20.0, -30.0
        case.k[0], case.q = k, torch.zeros_like(case.q)
        case.q[:, :, 0] = 64.0     # scores of 160 and -240
        case.v[0][at, :, [3, 30, 63]] = bad
        case.write(0)
        a = case.args("f32")
        case.call(a)
        torch.cuda.synchronize()
        out = a["out"].cpu().numpy()
        for i in range(nodes):
            if place != "node" or i == 2:
                assert not np.isfinite(out[i][:, [3, 30, 63]]).any(), i
                assert np.isfinite(np.delete(out[i], [3, 30, 63], axis=1)).all(), i
            else:
                assert np.isfinite(out[i]).all(), i
    finally:
        case.close()
