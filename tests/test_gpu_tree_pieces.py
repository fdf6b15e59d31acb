"""Tree attention where a CTA works on piece after piece, its buffers filled anew for each."""
import numpy as np
import pytest
import torch

from _gpu import require_cuda
from _tree import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,g", [(8, 4), (16, 4), (4, 8), (30, 2), (32, 4)])
@pytest.mark.parametrize("width", [0, 40])
def test_the_queries_of_every_piece(dtype, out_dtype, d, nodes, g, width):
    """170 sequences of a key tile or two, 4 kv heads: four or five pairs to a CTA, with four, two and
    one copies of a row.  A piece's copies meet in the buffer that the queries of the piece after the
    next are copied into; each piece has queries of its own, so one that finds another's is off by
    the size of an output."""
    rng = np.random.default_rng(nodes * g)
    case = TreeCase(dtype, d, 4, g, rng.integers(0, 200, 170), rng.integers(1, nodes + 1, 170), width=width, seed=nodes)
    try:
        a = case.args(out_dtype, max_q_len=nodes)
        case.call(a)
        case.check(a)
        first, lse = a["out"].clone(), a["lse"].clone()
        for _ in range(10):
            a["out"].fill_(777)
            case.call(a)
            assert torch.equal(first, a["out"]) and torch.equal(lse, a["lse"])
    finally:
        case.close()
