"""Keeping the accepted nodes in the cache, and whole steps over drafted tokens."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda
from _tree import DT, HALF, KV, TreeCase, random_parents, verify_reference, views

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    require_cuda()


class KeepCase:
    """Pools of random rows, sequences with trees at their ends, rising paths."""

    def __init__(self, dtype, d, hkv, cached, nodes, counts, layers=2, max_path=None, seed=0, spare=2):
        rng = np.random.default_rng(seed)
        self.dtype, self.d, self.hkv, self.nodes, self.layers = dtype, d, hkv, list(nodes), layers
        self.lens = [c + t for c, t in zip(cached, nodes)]
        self.batch = len(nodes)
        need = [-(-n // 16) for n in self.lens]
        self.width = max(1, max(need))
        self.blocks = sum(need) + spare
        ids = rng.permutation(self.blocks)
        self.tables = np.full((self.batch, self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        self.paths = [sorted(rng.choice(np.arange(1, t), c, replace=False).tolist()) if c else []
                      for t, c in zip(nodes, counts)]
        self.max_path = max([1] + list(counts)) if max_path is None else max_path
        self.pools = [pk.kv_pool_create(self.blocks, 16, hkv, d, KV[dtype]) for _ in range(layers)]
        g = torch.Generator().manual_seed(seed)
        bits = torch.int32 if dtype == "f32" else torch.int16
        self.before = []
        for p in self.pools:
            kv = []
            for x in views(p, self.blocks, hkv, d, dtype):
                r = torch.randint(-2 ** 15, 2 ** 15, x.shape, generator=g).to(bits)  # any bits, NaN too
                x.view(bits).copy_(r)
                kv.append(r)
            self.before.append(kv)

    def args(self):
        def ints(x):
            return torch.tensor(x, dtype=torch.int32).cuda()
        cu = np.concatenate([[0], np.cumsum(self.nodes)])
        path = [p + [-1] * (self.max_path - len(p)) for p in self.paths]
        return dict(cu=ints(cu.tolist()), path=ints(path), count=ints([len(p) for p in self.paths]),
                    tables=torch.from_numpy(self.tables).cuda(), lens=ints(self.lens),
                    new=torch.full((self.batch + 2,), 77, dtype=torch.int32, device="cuda"))

    def call(self, a, pools=None, stream=None):
        pk.kv_keep_path(pools or self.pools, a["cu"], max([1] + self.nodes), a["path"], self.max_path, a["count"],
                        a["tables"], self.width, a["lens"], self.batch, a["new"], stream=stream)

    def expect(self, skip=(), rows=()):
        """The pools' bits; `skip`: sequences left alone, `rows`: (sequence, index in its path) left out."""
        out = [[x.clone() for x in kv] for kv in self.before]
        for b, path in enumerate(self.paths):
            if b in skip:
                continue
            first = self.lens[b] - self.nodes[b]
            for i, node in enumerate(path):
                if (b, i) in rows:
                    continue
                s, d = first + node, first + i + 1
                for old, new in zip(self.before, out):
                    for x, y in zip(old, new):
                        y[self.tables[b, d // 16], :, d % 16] = x[self.tables[b, s // 16], :, s % 16]
        return out

    def check(self, a, err=0, skip=(), rows=(), expected=None):
        torch.cuda.synchronize()
        for p in self.pools:
            assert pk.kv_get_device_error(p) == err
        expected = expected or self.expect(skip, rows)
        for p, kv in zip(self.pools, expected):
            for x, y in zip(views(p, self.blocks, self.hkv, self.d, self.dtype), kv):
                assert torch.equal(x.view(y.dtype).cpu(), y)
        lens = [n if b in skip or t == 0 else n - t + 1 + len(path)
                for b, (n, t, path) in enumerate(zip(self.lens, self.nodes, self.paths))]
        assert a["new"].tolist() == lens + [77, 77]

    def close(self):
        for p in self.pools:
            pk.kv_pool_destroy(p)


def run(case, **kw):
    try:
        a = case.args()
        case.call(a)
        case.check(a, **kw)
    finally:
        case.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_types_and_heads(dtype, d, hkv):
    run(KeepCase(dtype, d, hkv, [20, 0, 15, 100], [9, 5, 1, 30], [4, 2, 0, 7], seed=d + hkv))


@pytest.mark.parametrize("nodes,count", [(1, 0), (2, 1), (17, 16), (20, 9), (64, 8), (64, 63), (255, 17), (256, 255), (256, 128)])
def test_path_lengths(nodes, count):
    run(KeepCase("bf16", 64, 2, [7, 33], [nodes, 3], [count, 2], seed=nodes + count))


@pytest.mark.parametrize("layers", [1, 3, 127, 128, 129, 260])
def test_layers(layers):
    run(KeepCase("f16", 64, 1, [5, 30], [6, 8], [3, 2], layers=layers))


@pytest.mark.parametrize("batch", [1, 50, 700])
def test_batches(batch):
    rng = np.random.default_rng(batch)
    nodes = rng.integers(0, 12, batch).tolist()
    run(KeepCase("bf16", 64, 1, rng.integers(0, 70, batch).tolist(), nodes, [int(rng.integers(0, max(1, t))) for t in nodes]))


def test_paths_that_do_not_rise():
    case = KeepCase("bf16", 64, 2, [20, 20, 20, 20, 20], [8] * 5, [3, 3, 3, 3, 3], seed=1)
    try:
        a = case.args()
        for b, path in ((0, [2, 2, 5]), (1, [4, 3, 6]), (2, [0, 1, 2]), (3, [1, 2, 8])):
            a["path"][b, :3] = torch.tensor(path, dtype=torch.int32)
        case.call(a)
        case.check(a, err=0x40, skip=(0, 1, 2, 3))
    finally:
        case.close()


def test_sizes_out_of_range():
    case = KeepCase("bf16", 64, 2, [20, 20, 20], [8] * 3, [3, 3, 3], seed=1)
    try:
        a = case.args()
        a["count"][0] = 9
        a["count"][1] = -1
        case.call(a)
        case.check(a, err=0x40, skip=(0, 1))
        for x in case.pools:
            assert pk.kv_get_device_error(x) == 0
    finally:
        case.close()
    case = KeepCase("bf16", 64, 2, [20, 20, 20], [8] * 3, [3, 3, 3], seed=1)
    try:
        a = case.args()
        a["lens"][0] = 5
        a["lens"][1] = 16 * case.width + 1
        case.lens[0], case.lens[1] = 5, 16 * case.width + 1
        case.call(a)
        case.check(a, err=0x1, skip=(0, 1))
    finally:
        case.close()


def test_blocks_out_of_range():
    case = KeepCase("f32", 64, 2, [10, 20], [24, 8], [3, 3], seed=1)
    case.paths[0] = [3, 9, 20]    # tokens 13, 19 and 30 to places 11, 12 and 13
    try:
        a = case.args()
        a["tables"][0, 1] = case.blocks  # tokens 16 .. 31: two of the sources
        case.call(a)
        case.check(a, err=0x1, rows=((0, 1), (0, 2)))
    finally:
        case.close()


def test_captured_and_replayed():
    case = KeepCase("bf16", 128, 2, [20, 40], [16, 16], [3, 3], seed=1)
    case.paths = [[1, 8, 12], [5, 9, 10]]  # a second pass finds what the first found
    try:
        a = case.args()
        case.call(a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            case.call(a)
        a["new"].fill_(77)
        graph.replay()
        case.check(a)
    finally:
        case.close()


def test_a_decode_that_overlaps_reads_the_new_lengths():
    case = KeepCase("bf16", 128, 2, [700, 40, 300], [16, 9, 30], [3, 0, 7], layers=1, seed=4)
    pool = case.pools[0]
    try:
        for x in views(pool, case.blocks, 2, 128, "bf16"):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(5)).bfloat16())
        a = case.args()
        q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
        n = pk.kv_decode_workspace_size(3, 8, 2, 128, case.width, 1)
        ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
        outs = [torch.zeros(3, 8, 128, device="cuda") for _ in range(2)]

        def decode(lens, out):
            pk.paged_decode_attention(pool, q, a["tables"], case.width, lens, 3, 8, 1 / math.sqrt(128), out, pk.KV_F32, None, 1,
                                      ws, n)
        case.call(a)
        torch.cuda.synchronize()
        lens = a["new"][:3].clone()
        decode(lens, outs[0])
        torch.cuda.synchronize()
        a["count"].zero_()  # nothing moves again; the lengths shrink to the roots
        case.paths = [[], [], []]
        roots = torch.tensor([701, 41, 301], dtype=torch.int32, device="cuda")
        decode(roots, outs[0])
        torch.cuda.synchronize()
        pk.kv_pool_set_launch_overlap(pool, True)
        for _ in range(20):
            a["new"].fill_(1)
            case.call(a)
            decode(a["new"], outs[1])
            torch.cuda.synchronize()
            assert torch.equal(outs[0], outs[1])
    finally:
        case.close()


def test_offsets_past_32_bits():
    blocks = 140000
    case = KeepCase("bf16", 128, 8, [40], [9], [3], layers=1, seed=2)
    pool = pk.kv_pool_create(blocks, 16, 8, 128, pk.KV_BF16)
    try:
        far = blocks - case.blocks
        for x, y in zip(views(pool, blocks, 8, 128, "bf16"), case.before[0]):
            x[far:].view(torch.int16).copy_(y)
        a = case.args()
        a["tables"] = torch.where(a["tables"] >= 0, a["tables"] + far, a["tables"])
        case.call(a, pools=[pool])
        torch.cuda.synchronize()
        for x, y in zip(views(pool, blocks, 8, 128, "bf16"), case.expect()[0]):
            assert torch.equal(x[far:].view(torch.int16).cpu(), y)
    finally:
        case.close()
        pk.kv_pool_destroy(pool)


def test_refusals():
    case = KeepCase("bf16", 64, 2, [20], [8], [3], layers=2)
    other = [pk.kv_pool_create(case.blocks, 16, 2, 64, pk.KV_F16), pk.kv_pool_create(case.blocks + 1, 16, 2, 64, pk.KV_BF16),
             pk.kv_pool_create(case.blocks, 16, 1, 64, pk.KV_BF16), pk.kv_pool_create(case.blocks, 16, 2, 128, pk.KV_BF16)]
    i4 = pk.kv_pool_create(case.blocks, 16, 2, 64, pk.KV_I4)
    try:
        a = case.args()

        def refused(status, **change):
            x = dict(pools=case.pools, cu=a["cu"], n=8, path=a["path"], m=case.max_path, count=a["count"], tables=a["tables"],
                     width=case.width, lens=a["lens"], batch=1, new=a["new"])
            x.update(change)
            with pytest.raises(pk.KVError) as e:
                pk.kv_keep_path(x["pools"], x["cu"], x["n"], x["path"], x["m"], x["count"], x["tables"], x["width"],
                                x["lens"], x["batch"], x["new"])
            assert e.value.status == status, change
        for change in ([dict(pools=[case.pools[0], o]) for o in other] +
                       [dict(pools=[]), dict(pools=[case.pools[0]] * 2), dict(pools=[None]), dict(cu=None), dict(path=None),
                        dict(count=None), dict(tables=None), dict(lens=None), dict(new=None), dict(n=-1), dict(m=-1),
                        dict(width=-1), dict(batch=-1), dict(new=a["lens"])]):
            refused(-1, **change)
        for change in (dict(pools=[i4]), dict(n=257), dict(m=256), dict(width=1 << 27), dict(batch=1 << 24)):
            refused(-3, **change)
        torch.cuda.synchronize()
        assert (a["new"] == 77).all()
    finally:
        case.close()
        for p in other + [i4]:
            pk.kv_pool_destroy(p)


# ------------------------------------------------------------ whole steps
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 128)])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_over_drafted_tokens(dtype, d, captured):
    """Append a tree, attend, verify, keep, and go on: what every step leaves in the caches is what a cache
    holds that was given the accepted tokens alone, and a decode over it sees exactly those."""
    hkv, g, layers, vocab, batch, T, steps = 2, 4, 2, 90, 3, 12, 4
    hq, width, blocks = hkv * g, 8, 40
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(7)
    pools = [pk.kv_pool_create(blocks, 16, hkv, d, KV[dtype]) for _ in range(layers)]
    try:
        tables = rng.permutation(blocks)[:batch * width].reshape(batch, width).astype(np.int32)
        t_tables = torch.from_numpy(tables).cuda()
        kept = [0, 5, 33]                       # tokens in the caches
        rows = [[[torch.randn(n, hkv, d, generator=gen).to(DT[dtype]) for n in kept] for _ in "kv"] for _ in pools]

        def slots(b, first, n):
            j = np.arange(first, first + n)
            return tables[b, j // 16].astype(np.int64) * 16 + j % 16
        for p, (k, v) in zip(pools, rows):
            for b, n in enumerate(kept):
                if n:
                    pk.kv_append(p, k[b].cuda(), v[b].cuda(), torch.from_numpy(slots(b, 0, n)).cuda(), n)
        cu = torch.arange(0, batch * T + 1, T, dtype=torch.int32, device="cuda")
        dev = dict(k=[torch.zeros(batch * T, hkv, d, dtype=DT[dtype], device="cuda") for _ in pools],
                   v=[torch.zeros(batch * T, hkv, d, dtype=DT[dtype], device="cuda") for _ in pools],
                   q=[torch.zeros(batch * T, hq, d, dtype=DT[dtype], device="cuda") for _ in pools],
                   out=[torch.zeros(batch * T, hq, d, dtype=torch.float32, device="cuda") for _ in pools],
                   slots=torch.zeros(batch * T, dtype=torch.int64, device="cuda"),
                   parents=torch.zeros(batch * T, dtype=torch.int32, device="cuda"),
                   tokens=torch.zeros(batch * T, dtype=torch.int32, device="cuda"),
                   p=torch.zeros(batch * T, vocab, device="cuda"), dq=torch.zeros(batch * T, vocab, device="cuda"),
                   au=torch.zeros(batch * T, device="cuda"), su=torch.zeros(batch, device="cuda"),
                   lens=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                   new=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                   count=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                   path=torch.zeros(batch, T, dtype=torch.int32, device="cuda"),
                   emitted=torch.zeros(batch, T + 1, dtype=torch.int32, device="cuda"))
        n_ws = pk.kv_tree_workspace_size(pools[0], batch, hq, width, T)
        ws = torch.empty(n_ws, dtype=torch.uint8, device="cuda")

        def step():
            for i, p in enumerate(pools):
                pk.kv_append(p, dev["k"][i], dev["v"][i], dev["slots"], batch * T)
                pk.paged_tree_attention(p, dev["q"][i], cu, batch * T, T, dev["parents"], t_tables, width, dev["lens"],
                                        batch, hq, 1 / math.sqrt(d), dev["out"][i], pk.KV_F32, None, ws, n_ws)
            pk.kv_verify_tree(pools[0], dev["p"], dev["dq"], pk.KV_F32, vocab, cu, batch * T, T, dev["parents"],
                              dev["tokens"], dev["au"], dev["su"], batch, T, dev["count"], dev["path"], dev["emitted"])
            pk.kv_keep_path(pools, cu, T, dev["path"], T, dev["count"], t_tables, width, dev["lens"], batch, dev["new"])
        graph = None
        moved = 0
        for s in range(steps):
            trees = [random_parents(rng, T, "tree") for _ in range(batch)]
            z = 5 * torch.randn(batch * T, vocab, generator=gen)
            p = torch.softmax(z, -1)
            q = torch.softmax(z + 0.3 * torch.randn(z.shape, generator=gen), -1)
            tokens = np.array([rng.choice(vocab, p=q[b * T + max(0, trees[b][i])].double().numpy() /
                                          q[b * T + max(0, trees[b][i])].double().numpy().sum())
                               for b in range(batch) for i in range(T)], np.int32)
            new_rows = [[torch.randn(batch * T, h, d, generator=gen).to(DT[dtype]) for h in (hkv, hkv, hq)] for _ in pools]
            au, su = rng.random(batch * T, np.float32), rng.random(batch, np.float32)
            for i in range(layers):
                for name, x in zip("kvq", new_rows[i]):
                    dev[name][i].copy_(x)
            dev["slots"].copy_(torch.from_numpy(np.concatenate([slots(b, kept[b], T) for b in range(batch)])))
            dev["parents"].copy_(torch.tensor(sum(trees, []), dtype=torch.int32))
            dev["tokens"].copy_(torch.from_numpy(tokens))
            dev["p"].copy_(p)
            dev["dq"].copy_(q)
            dev["au"].copy_(torch.from_numpy(au))
            dev["su"].copy_(torch.from_numpy(su))
            dev["lens"].copy_(torch.tensor([n + T for n in kept], dtype=torch.int32))
            torch.cuda.synchronize()
            if captured and s == 1:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            if graph:
                graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            for x in pools:
                assert pk.kv_get_device_error(x) == 0
            count, path, emitted = verify_reference(p.double().numpy(), q.double().numpy(), cu.tolist(),
                                                    sum(trees, []), tokens, au, su, T, vocab)
            assert dev["count"].tolist() == count.tolist() and dev["emitted"].cpu().numpy().tolist() == emitted.tolist()
            for b in range(batch):
                stay = [0] + [int(x) for x in path[b] if x >= 0]
                moved += sum(x != i for i, x in enumerate(stay))
                for i in range(layers):
                    for j in range(2):
                        rows[i][j][b] = torch.cat([rows[i][j][b], new_rows[i][j][b * T:b * T + T][stay]])
                kept[b] += len(stay)
            assert dev["new"].tolist() == kept
            assert max(kept) + T <= 16 * width
            for i, x in enumerate(pools):
                for view, mine in zip(views(x, blocks, hkv, d, dtype), rows[i]):
                    for b in range(batch):
                        at = torch.from_numpy(slots(b, 0, kept[b])).cuda()
                        assert torch.equal(view[at // 16, :, at % 16].cpu(), mine[b])
        assert moved > 0
        # a decode step over what was kept
        q = torch.randn(batch, hq, d, generator=gen).to(DT[dtype])
        out = torch.zeros(batch, hq, d, device="cuda")
        n = pk.kv_decode_workspace_size(batch, hq, hkv, d, width, 1)
        pk.paged_decode_attention(pools[0], q.cuda(), t_tables, width, dev["new"], batch, hq, 1 / math.sqrt(d), out,
                                  pk.KV_F32, None, 1, torch.empty(max(16, n), dtype=torch.uint8, device="cuda"), n)
        torch.cuda.synchronize()
        for b in range(batch):
            k, v = (rows[0][j][b].double() for j in range(2))
            for h in range(hq):
                w = torch.softmax(k[:, h // g] @ q[b, h].double() / math.sqrt(d), 0)
                # (the decode's own tolerance)
                assert (out[b, h].double().cpu() - w @ v[:, h // g]).abs().max() <= 2e-3 * v.abs().max()
    finally:
        for p in pools:
            pk.kv_pool_destroy(p)
