"""Verification of drafted tokens against the walk in 64 bits, and the draws against their law."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _tree import DT, KV, random_parents, verify_reference

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


class VerifyCase:
    def __init__(self, vocab, nodes, kind="tree", dtype="f32", drawn=True, seed=0, peak=4.0, noise=1.0, max_path=None,
                 p_pad=0, q_pad=0, shift=0):
        rng = np.random.default_rng(seed)
        self.vocab, self.nodes, self.dtype, self.drawn = vocab, list(nodes), dtype, drawn
        self.batch = len(nodes)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.total = int(self.cu[-1])
        self.trees = [random_parents(rng, t, kind) for t in nodes]
        self.parents = np.array(sum(self.trees, []), np.int32)
        g = torch.Generator().manual_seed(seed)
        z = peak * torch.randn(max(1, self.total), vocab, generator=g)
        self.p = torch.softmax(z, -1).to(DT[dtype])
        self.q = torch.softmax(z + noise * torch.randn(z.shape, generator=g), -1).to(DT[dtype])
        self.tokens = np.zeros(self.total, np.int32)
        for b in range(self.batch):
            for i in range(1, nodes[b]):
                r = int(self.cu[b]) + max(0, self.trees[b][i])
                w = self.q[r].double().numpy()
                # (two of five drafts from the target's likely ones, so that paths are long too)
                if drawn:
                    self.tokens[self.cu[b] + i] = rng.choice(vocab, p=w / w.sum())
                else:
                    self.tokens[self.cu[b] + i] = np.argsort(-w)[rng.integers(0, min(vocab, 3))]
        self.accept_u = rng.random(max(1, self.total), np.float32)
        self.sample_u = rng.random(max(1, self.batch), np.float32)
        self.max_path = max([1] + list(nodes)) if max_path is None else max_path
        self.p_stride, self.q_stride, self.shift = vocab + p_pad, vocab + q_pad, shift

    def rows(self, x, stride):
        """Device rows of that stride, starting `shift` elements behind an aligned address; NaN between them."""
        buf = torch.full((x.shape[0] * stride + self.shift,), math.nan, dtype=x.dtype, device="cuda")
        buf[self.shift:].view(x.shape[0], stride)[:, :self.vocab] = x.cuda()
        return buf[self.shift:]

    def args(self):
        def dev(x):
            return torch.from_numpy(np.ascontiguousarray(x)).cuda()
        b = self.batch
        return dict(p=self.rows(self.p, self.p_stride), q=self.rows(self.q, self.q_stride) if self.drawn else None,
                    cu=dev(self.cu), parents=dev(self.parents), tokens=dev(self.tokens), au=dev(self.accept_u),
                    su=dev(self.sample_u), count=torch.full((b + 2,), 77, dtype=torch.int32, device="cuda"),
                    path=torch.full((b + 2, max(1, self.max_path)), 77, dtype=torch.int32, device="cuda"),
                    out=torch.full((b + 2, self.max_path + 1), 77, dtype=torch.int32, device="cuda"))

    def call(self, pool, a, stream=None):
        pk.kv_verify_tree(pool, a["p"], a["q"], KV[self.dtype], self.vocab, a["cu"], self.total, max([0] + self.nodes),
                          a["parents"], a["tokens"], a["au"], a["su"], self.batch, self.max_path, a["count"],
                          a["path"] if self.max_path else None, a["out"], target_stride=self.p_stride,
                          draft_stride=self.q_stride, stream=stream)

    def check(self, pool, a, err=0):
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(pool) == err
        count, path, out = verify_reference(
            self.p.double().numpy(), self.q.double().numpy() if self.drawn else None, self.cu, self.parents, self.tokens,
            self.accept_u, self.sample_u, self.max_path, self.vocab)
        b = self.batch
        assert a["count"][:b].tolist() == count.tolist()
        if self.max_path:
            assert a["path"][:b].cpu().numpy().tolist() == path.tolist()
        assert a["out"][:b].cpu().numpy().tolist() == out.tolist()
        for x in ("count", "path", "out"):  # rows behind the batch
            assert (a[x][b:] == 77).all()
        return count


def run(pool, case, err=0):
    a = case.args()
    case.call(pool, a)
    return case.check(pool, a, err)


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 64, 511, 512, 513, 1000, 4096, 8191, 32000, 50001])
@pytest.mark.parametrize("drawn", [True, False])
def test_vocabularies(pool, vocab, drawn):
    run(pool, VerifyCase(vocab, [1, 4, 0, 9, 2], drawn=drawn, seed=vocab))


def test_largest_vocabulary(pool):
    run(pool, VerifyCase(1 << 20, [3, 5], seed=1))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["chain", "star", "tree", "forest"])
@pytest.mark.parametrize("drawn", [True, False])
def test_types_and_trees(pool, dtype, kind, drawn):
    counts = [run(pool, VerifyCase(1500, [6, 12, 20, 7, 33], kind=kind, dtype=dtype, drawn=drawn, seed=s, peak=6.0, noise=0.5))
              for s in range(4)]
    assert max(c.max() for c in counts) > 0


@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 64, 65, 128, 255, 256])
def test_tree_sizes(pool, nodes):
    for kind in ("chain", "tree", "star"):
        run(pool, VerifyCase(300, [nodes, 3], kind=kind, seed=nodes, noise=0.3, max_path=min(nodes, 255)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 3), (8, 0), (8, 8)])
def test_strides_and_alignment(pool, dtype, pad, shift):
    run(pool, VerifyCase(5000, [5, 9, 2], dtype=dtype, p_pad=pad, q_pad=2 * pad, shift=shift, seed=pad))


@pytest.mark.parametrize("batch", [1, 7, 100, 1500])
def test_batches(pool, batch):
    nodes = np.random.default_rng(batch).integers(0, 5, batch).tolist()
    run(pool, VerifyCase(200, nodes, seed=batch))


@pytest.mark.parametrize("max_path", [0, 1, 2])
def test_paths_end_at_the_limit(pool, max_path):
    run(pool, VerifyCase(50, [9, 7, 1], kind="chain", noise=0.1, max_path=max_path, seed=6))


def test_many_rejections(pool):
    # drafts that the target likes little, twenty of one node: the residual is taken twenty times
    for seed in range(3):
        run(pool, VerifyCase(700, [21, 21], kind="star", noise=3.0, peak=2.0, seed=seed))


def test_same_draft_twice(pool):
    case = VerifyCase(40, [6, 6], kind="star", drawn=False, seed=2)
    case.tokens[1:6] = [3, 3, 5, 3, 5]
    case.accept_u[:] = 0.999
    run(pool, case)


def test_equal_distributions(pool):
    # p = q: every draft that is drawn is accepted; one that is not in q leaves nothing behind it
    case = VerifyCase(64, [4, 4, 4], kind="chain", seed=3)
    case.q = case.p.clone()
    counts = run(pool, case)
    assert counts.tolist() == [3, 3, 3]
    case = VerifyCase(8, [3], kind="star", seed=3)
    case.p[0] = torch.tensor([0.5, 0.5, 0, 0, 0, 0, 0, 0])
    case.q = case.p.clone()
    case.tokens[1:] = [4, 0]     # has no probability; what is left for node 2 is nothing
    assert run(pool, case).tolist() == [0]


def test_greedy_rows(pool):
    # one at the target's token: drafts that name it are accepted, the next token is it
    case = VerifyCase(1000, [4, 4, 4], kind="chain", drawn=False, seed=8)
    best = np.random.default_rng(1).integers(0, 1000, 12)
    case.p.zero_()
    case.p[torch.arange(12), torch.from_numpy(best)] = 1.0
    case.tokens[1:4] = best[0:3]           # all three
    case.tokens[5:8] = [best[4], 7, 8]     # one
    case.tokens[9:12] = [(best[8] + 1) % 1000, 1, 2]
    assert run(pool, case).tolist() == [3, 1, 0]


def test_borders_of_the_draw(pool):
    # probabilities of whole 2^-24ths: the running sums are known, the numbers hit them exactly
    vocab = 600
    case = VerifyCase(vocab, [1] * 64, seed=0)
    case.p.zero_()
    case.p[:, [3, 5, 511, 512, 599]] = torch.tensor([0.125, 0.25, 0.25, 0.25, 0.125])
    u = np.array([0, 0.125, 0.375, 0.625, 0.875, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, math.inf, 1e-30, 1e-45], np.float32)
    u = np.concatenate([u, np.nextafter(u[1:5], 0, dtype=np.float32), np.nextafter(u[1:5], 1, dtype=np.float32)])
    case.sample_u[:len(u)] = u
    a = case.args()
    case.call(pool, a)
    torch.cuda.synchronize()
    got = a["out"][:len(u), 0].tolist()
    assert got == [3, 5, 511, 512, 599, 599, 599, 599, 3, 3, 599, 3, 3] + [3, 5, 511, 512] + [5, 511, 512, 599]


def test_entries_that_are_no_probabilities(pool):
    case = VerifyCase(100, [1, 1, 1, 3], kind="chain", seed=5)
    case.p[0, :50] = math.nan
    case.p[0, 50:60] = -1.0
    case.p[1] = 0
    case.p[2] = math.inf      # ones
    case.p[3] = math.nan      # nothing: no draft is accepted, no token drawn
    a = case.args()
    case.call(pool, a)
    count = case.check(pool, a)
    assert count.tolist() == [0, 0, 0, 0]
    assert a["out"][1, 0] == -1 and a["out"][3, 0] == -1


def test_drafts_that_are_none(pool):
    case = VerifyCase(100, [5, 5], kind="star", noise=0.1, seed=4)
    case.tokens[1:3] = [-1, -7]
    run(pool, case)
    case.tokens[7] = 100
    run(pool, case, err=0x40)
    case.tokens[7] = 2 ** 31 - 1
    run(pool, case, err=0x40)


def test_parents_out_of_order(pool):
    case = VerifyCase(100, [5, 3], kind="chain", noise=0.0, seed=4)
    case.parents[2] = 2
    case.parents[6] = -9
    assert run(pool, case, err=0x40).tolist() == [1, 0]


def test_chains_without_parents(pool):
    case = VerifyCase(300, [5, 0, 8], kind="chain", noise=0.2, seed=4)
    a = case.args()
    a["parents"] = None
    case.call(pool, a)
    case.check(pool, a)


def test_rows_out_of_range(pool):
    case = VerifyCase(100, [4, 4, 4], kind="chain", noise=0.0, seed=4)
    for cu in ([0, 4, 8, 13], [0, 4, 3, 12], [-1, 4, 8, 12], [0, 4, 12, 12]):
        a = case.args()
        a["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        case.call(pool, a)
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(pool) == 0x1
        for b in range(3):
            n = cu[b + 1] - cu[b]
            if n < 0 or n > 4 or cu[b] < 0 or cu[b + 1] > 12 or n == 0:
                assert a["count"][b] == 0 and (a["out"][b] == -1).all() and (a["path"][b] == -1).all()
            elif n == 4 and cu[b] == 4 * b:
                assert a["count"][b] == 3


def test_emitted_tokens_follow_the_target(pool):
    """The first emitted token of a two-level tree has the target's distribution whatever the draft proposes.

    n independent steps, 12 tokens: a count of probability p is off by at most 5 sqrt(n p (1 - p)) but in
    6e-7 of cases (a normal bound, 12 of them)."""
    n, vocab = 20000, 12
    g = np.random.default_rng(0)
    p = g.dirichlet(np.ones(vocab)).astype(np.float32)
    q = g.dirichlet(np.ones(vocab)).astype(np.float32)
    for drawn in (True, False):
        case = VerifyCase(vocab, [1], seed=0)
        case.drawn = drawn
        case.nodes, case.batch, case.max_path = [4] * n, n, 3
        case.cu, case.total = np.arange(0, 4 * n + 1, 4, dtype=np.int32), 4 * n
        case.parents = np.tile(np.array([-1, 0, 0, 0], np.int32), n)
        case.p, case.q = torch.from_numpy(np.tile(p, (4 * n, 1))), torch.from_numpy(np.tile(q, (4 * n, 1)))
        case.tokens = g.choice(vocab, 4 * n, p=q.astype(np.float64) / q.sum(dtype=np.float64)).astype(np.int32)
        if not drawn:
            case.tokens = np.tile(np.array([0, 7, 2, 9], np.int32), n)
        case.accept_u, case.sample_u = g.random(4 * n, np.float32), g.random(n, np.float32)
        a = case.args()
        case.call(pool, a)
        torch.cuda.synchronize()
        seen = np.bincount(a["out"][:n, 0].cpu().numpy(), minlength=vocab)
        assert (np.abs(seen - n * p) <= 5 * np.sqrt(n * p * (1 - p))).all(), (seen, n * p)


def test_captured_and_replayed(pool):
    case = VerifyCase(3000, [6, 9, 1, 12], seed=11)
    a = case.args()
    case.call(pool, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.call(pool, a)
    for seed in range(3):
        r = np.random.default_rng(seed)
        case.accept_u, case.sample_u = r.random(case.total, np.float32), r.random(4, np.float32)
        a["au"].copy_(torch.from_numpy(case.accept_u))
        a["su"].copy_(torch.from_numpy(case.sample_u))
        graph.replay()
        case.check(pool, a)


def test_two_streams_at_once(pool):
    one, two = VerifyCase(20000, [6] * 8, seed=1), VerifyCase(9000, [9] * 8, seed=2)
    a, b = one.args(), two.args()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        one.call(pool, a, stream=s)
        two.call(pool, b, stream=t)
    torch.cuda.synchronize()
    one.check(pool, a)
    two.check(pool, b)


def test_offsets_past_32_bits(pool):
    # rows so far apart that the last one begins past 2^31 elements
    case = VerifyCase(1000, [4, 4], kind="chain", noise=0.2, seed=9)
    stride = (1 << 31) // 7 + 5000
    buf = torch.zeros(8 * stride, dtype=torch.bfloat16, device="cuda")
    case.dtype = "bf16"
    case.p, case.q = case.p.bfloat16(), case.q.bfloat16()
    buf.view(8, stride)[:, :1000] = case.p.cuda()
    a = case.args()
    a["p"], case.p_stride = buf, stride
    case.call(pool, a)
    case.check(pool, a)


def test_refusals(pool):
    case = VerifyCase(100, [4], seed=1)
    a = case.args()

    def refused(status, **change):
        x = dict(pool=pool, p=a["p"], q=a["q"], dt=pk.KV_F32, vocab=100, cu=a["cu"], total=4, n=4, tokens=a["tokens"],
                 au=a["au"], su=a["su"], batch=1, m=4, count=a["count"], path=a["path"], out=a["out"], ps=0, qs=0)
        x.update(change)
        with pytest.raises(pk.KVError) as e:
            pk.kv_verify_tree(x["pool"], x["p"], x["q"], x["dt"], x["vocab"], x["cu"], x["total"], x["n"], a["parents"],
                              x["tokens"], x["au"], x["su"], x["batch"], x["m"], x["count"], x["path"], x["out"],
                              target_stride=x["ps"], draft_stride=x["qs"])
        assert e.value.status == status, change
    for change in (dict(pool=None), dict(p=None), dict(cu=None), dict(tokens=None), dict(au=None), dict(su=None),
                   dict(count=None), dict(path=None), dict(out=None), dict(vocab=0), dict(total=-1), dict(n=-1),
                   dict(batch=-1), dict(m=-1), dict(ps=99), dict(qs=99), dict(ps=-1), dict(qs=-1),
                   dict(p=a["p"].data_ptr() + 2)):
        refused(-1, **change)
    for change in (dict(dt=pk.KV_I4), dict(dt=9), dict(vocab=(1 << 20) + 1), dict(n=257), dict(m=256)):
        refused(-3, **change)
    torch.cuda.synchronize()
    assert (a["count"] == 77).all() and (a["path"] == 77).all() and (a["out"] == 77).all()
