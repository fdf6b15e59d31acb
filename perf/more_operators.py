"""Cases that measure a step over drafted tokens: attention of a tree of drafts
over the cache, the verification of the drafts against the target's
probabilities, and the move that leaves only the accepted ones in the cache.

With ``own`` false ``run`` computes an operator from elementary torch
operations; with ``own`` true it makes the library's calls.

A sequence's tree has T nodes, the last T tokens of its cache.  Node 0 is the
token that the step before emitted, the others are drafts, and a node's parent
comes before it.  A node attends every token before the tree, its ancestors and
itself.  Verification walks from node 0: a child whose token x was drawn from
the draft's q is accepted if u q(x) < p(x), p the target's probabilities after
the node; a rejected one leaves p = max(p - q, 0), normalised, to the next child
and, after the last, to the draw of the next token.  Without q the drafts were
chosen, not drawn: q is one at the draft itself.
"""
import math
import random

import torch

own = False

BLOCK = 16  # tokens per block
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a nearly idle server of a small model: two short sequences, a few drafts each
        dict(name="tree 2 short", op="tree", dtype="f16", out="f32", batch=2, cached_lo=40, cached_hi=400,
             nodes_lo=4, nodes_hi=8, hq=8, hkv=8, d=64),
        # trees of 64 nodes over ordinary contexts
        dict(name="tree 16 x 64 nodes", op="tree", dtype="bf16", out="bf16", batch=16, cached_lo=1000,
             cached_hi=8000, nodes_lo=64, nodes_hi=64, hq=32, hkv=8, d=128),
        # few very long contexts, eight query heads per kv head
        dict(name="tree 4 long", op="tree", dtype="bf16", out="bf16", batch=4, cached_lo=32768, cached_hi=131072,
             nodes_lo=26, nodes_hi=26, hq=32, hkv=4, d=128),
        # a full batch of chats whose trees were cut to what each draft was sure of
        dict(name="tree 64 ragged", op="tree", dtype="f16", out="f16", batch=64, cached_lo=512, cached_hi=4096,
             nodes_lo=1, nodes_hi=17, hq=32, hkv=8, d=128),
        # a small fp32 model, odd sizes, a sequence that starts here
        dict(name="tree fp32 odd", op="tree", dtype="f32", out="f32", batch=5, cached_lo=0, cached_hi=1531,
             nodes_lo=3, nodes_hi=33, hq=12, hkv=4, d=64),
        # one sequence, four drafts in a row
        dict(name="verify one chain", op="verify", dtype="f32", batch=1, nodes=5, chain=True, drawn=True,
             vocab=32000),
        # a full batch, five drafts in a row each, a large vocabulary
        dict(name="verify 64 chains", op="verify", dtype="f32", batch=64, nodes=6, chain=True, drawn=True,
             vocab=128000),
        # trees of 64 nodes
        dict(name="verify 16 trees", op="verify", dtype="f32", batch=16, nodes=64, chain=False, drawn=True,
             vocab=128000),
        # trees of each draft's likeliest tokens (no q), 16-bit probabilities, an odd vocabulary
        dict(name="verify chosen odd", op="verify", dtype="bf16", batch=33, nodes=26, chain=False, drawn=False,
             vocab=50001),
        # a full batch, every layer's cache of an ordinary model
        dict(name="keep 64 x 24 layers", op="keep", dtype="bf16", layers=24, batch=64, nodes=32, depth=6,
             cached=40, hkv=8, d=128),
        # three sequences, two layers of a small fp32 model
        dict(name="keep 3 x 2 fp32", op="keep", dtype="f32", layers=2, batch=3, nodes=9, depth=4, cached=101,
             hkv=3, d=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "verify", "keep"))
    dtype = rng.choice(("bf16", "f16", "bf16", "f16", "f32"))
    if op == "verify":
        vocab = _log(rng, 1000, 160000)
        nodes = _log(rng, 1, 96)
        # at most the rows of the listed trees
        batch = _log(rng, 1, max(1, min(256, 16 * 64 * 128000 // (vocab * nodes))))
        return dict(op=op, dtype=dtype, batch=batch, nodes=nodes, chain=rng.random() < 0.4,
                    drawn=rng.random() < 0.7, vocab=vocab)
    hkv = rng.choice((1, 2, 3, 4, 8))
    d = rng.choice((64, 128))
    if op == "keep":
        depth = rng.randint(1, 16)
        layers, batch = _log(rng, 1, 24), _log(rng, 1, 128)
        # at most the listed pools
        most = 24 * 64 * 8 * 128 * 2 * 80 // (layers * batch * hkv * d * (4 if dtype == "f32" else 2))
        nodes = _log(rng, depth + 1, 96)
        return dict(op=op, dtype=dtype, layers=layers, batch=batch, nodes=nodes, depth=depth,
                    cached=_log(rng, 1, max(1, min(4096, most - nodes))), hkv=hkv, d=d)
    g = rng.randint(1, 8)
    batch = _log(rng, 1, 64)
    nodes = _log(rng, 1, 192)
    # at most the listed long contexts, in bytes and in products; fp32 without the tensor cores a tenth of them
    most = min(286000 * 4 * 128 // (batch * hkv * d), 286000 * 26 * 32 * 128 // (batch * nodes * g * hkv * d))
    most = max(1, min(131072, most // 2 if dtype != "f32" else most // 20))
    cached = _log(rng, min(16, most), most)
    return dict(op=op, dtype=dtype, out=rng.choice((dtype, "f32")), batch=batch, cached_lo=_log(rng, 1, cached) - 1,
                cached_hi=cached, nodes_lo=_log(rng, 1, nodes), nodes_hi=nodes, hq=g * hkv, hkv=hkv, d=d)


def _spread(batch, lo, hi):
    """`batch` numbers from lo to hi, evenly spaced (over their logarithm for long spans)."""
    if batch == 1:
        return [hi]
    if lo > 0 and hi > 3 * lo and hi > 8192:
        return [int(round(lo * (hi / lo) ** (i / (batch - 1)))) for i in range(batch)]
    return [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]


def _sizes(case):
    """(tokens in the cache, nodes of its tree) of each sequence."""
    cached = _spread(case["batch"], case["cached_lo"], case["cached_hi"])
    nodes = _spread(case["batch"], case["nodes_lo"], case["nodes_hi"])[::-1]
    return [(c + t, t) for c, t in zip(cached, nodes)]


def _accepted(case):
    """(accepted drafts, those of them that are in their place already) of each sequence."""
    return [(m, m // 3) for m in _spread(case["batch"], 0, min(case["depth"], (case["nodes"] - 1) // 2))]


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    e = _size(case["dtype"])
    if case["op"] == "keep":
        row = 2 * case["hkv"] * case["d"] * e * case["layers"]
        moved = sum(m - s for m, s in _accepted(case))
        return {"bytes": 2 * moved * row + case["batch"] * (4 * case["depth"] + 16), "flops": 0}
    if case["op"] == "verify":
        # the row that the next token is drawn from, p and q; p and q of each draft on the way
        rows = case["batch"] * case["vocab"] * (2 if case["drawn"] else 1)
        return {"bytes": rows * e + case["batch"] * case["nodes"] * 12, "flops": 2 * rows}
    oe = _size(case["out"])
    sizes = _sizes(case)
    rows = sum(t for _, t in sizes)
    keys = sum(n for n, _ in sizes)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    # a node sees what is cached and its ancestors, about log2 of the tree
    pairs = sum(t * (n - t) + sum(i.bit_length() for i in range(1, t + 1)) for n, t in sizes)
    return {"bytes": 2 * keys * hkv * d * e + rows * (hq * (d * (e + oe) + 4) + 4) + keys // 4,
            "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _parents(rng, nodes, chain=False):
    """A tree in the order in which drafting adds nodes: parents by index, -1 for node 0."""
    if chain:
        return list(range(-1, nodes - 1))
    return [-1] + [rng.randint((i - 1) // 4, (i - 1) // 2) for i in range(1, nodes)]


def _rows(g, n, heads, d, dtype, size, channels=False):
    """n rows of activations: normal values; keys have channels of unlike sizes."""
    x = torch.randn(n, heads, d, generator=g, device="cuda", dtype=torch.float32) * size
    if channels:
        x *= torch.exp(0.7 * torch.randn(1, heads, d, generator=g, device="cuda"))
    return x.to(dtype)


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _offsets(counts):
    return [sum(counts[:i]) for i in range(len(counts) + 1)]


def _table(g, need):
    """Shuffled blocks: the tables of sequences that need these many, and the pool's size."""
    width, blocks = max(1, max(need)), sum(need) + 2
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    tables = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    return tables, blocks


def _slots(tables, b, first, count):
    j = torch.arange(first, first + count, device="cuda")
    return tables[b, j // BLOCK].long() * BLOCK + j % BLOCK


def _tree_inputs(case, seed):
    """Rows of a cache of ragged sequences in shuffled blocks, the trees at their ends, the queries."""
    g, rng = _gen(seed), random.Random(seed)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    sizes = _sizes(case)
    rng.shuffle(sizes)
    tables, blocks = _table(g, [-(-n // BLOCK) for n, _ in sizes])
    slots = torch.cat([_slots(tables, b, 0, n) for b, (n, _) in enumerate(sizes)])
    total, rows = sum(n for n, _ in sizes), sum(t for _, t in sizes)
    k = _rows(g, total, hkv, d, dt, 1.0, True)
    v = _rows(g, total, hkv, d, dt, 0.4)
    q = _rows(g, rows, hq, d, dt, 1.0)
    parents = [_parents(rng, t) for _, t in sizes]
    return dict(lens=[n for n, _ in sizes], nodes=[t for _, t in sizes], tables=tables, blocks=blocks, slots=slots,
                k=k, v=v, q=q, trees=parents, parents=_ints(sum(parents, [])),
                cu=_ints(_offsets([t for _, t in sizes])), seq_lens=_ints([n for n, _ in sizes]))


def _verify_inputs(case, seed):
    """Probabilities of a peaked vocabulary, the draft's a noisy copy of the target's, and the drafts."""
    g, rng = _gen(seed), random.Random(seed)
    batch, nodes, vocab, dt = case["batch"], case["nodes"], case["vocab"], DTYPES[case["dtype"]]
    trees = [_parents(rng, nodes, case["chain"]) for _ in range(batch)]
    rows = batch * nodes
    p = torch.empty(rows, vocab, dtype=dt, device="cuda")
    q = torch.empty(rows, vocab, dtype=dt, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for at in range(0, rows, step):
        z = 6.0 * torch.randn(min(step, rows - at), vocab, generator=g, device="cuda")
        p[at:at + step] = torch.softmax(z, -1)
        z += torch.randn(z.shape, generator=g, device="cuda")
        q[at:at + step] = torch.softmax(z, -1)
        del z
    parents = _ints(trees)  # [batch][nodes]
    row = (torch.arange(batch, device="cuda")[:, None] * nodes + parents.clamp(min=0)).flatten()
    tokens = torch.empty(rows, dtype=torch.int64, device="cuda")
    if case["drawn"]:
        for at in range(0, rows, step):
            tokens[at:at + step] = torch.multinomial(q[row[at:at + step]].float(), 1, generator=g)[:, 0]
    else:
        # the k-th child of a node is the draft's k-th likeliest token
        rank = _ints([[t[:i].count(t[i]) for i in range(nodes)] for t in trees]).flatten().long()
        best = torch.topk(q, min(vocab, 16), dim=-1).indices
        tokens[:] = best[row, rank.clamp(max=best.shape[1] - 1)]
    s = dict(p=p, parents=parents.flatten().contiguous(), tokens=tokens.int(), trees=trees,
             accept_u=torch.rand(rows, generator=g, device="cuda"),
             sample_u=torch.rand(batch, generator=g, device="cuda"), cu=_ints(list(range(0, rows + 1, nodes))))
    if case["drawn"]:
        s["q"] = q
    # what a way down may hold: every draft of a chain; a tree's parents have at most half their child's index
    s["max_path"] = max(1, nodes - 1 if case["chain"] else nodes.bit_length())
    s["children"] = max([1] + [t.count(i) for t in trees for i in set(t) if i >= 0])
    return s


def _keep_inputs(case, seed):
    """Pools of every layer, the accepted nodes of each sequence.

    The first third of a path lies where it belongs; the others come from behind
    the places that are filled, so that a second pass finds what the first found.
    """
    g, rng = _gen(seed), random.Random(seed)
    t = case["nodes"]
    lens = [max(0, case["cached"] - 7 * b % 25) + t for b in range(case["batch"])]
    rng.shuffle(lens)
    tables, blocks = _table(g, [-(-n // BLOCK) for n in lens])
    done = _accepted(case)
    rng.shuffle(done)
    paths = [list(range(1, s + 1)) + sorted(rng.sample(range(m + 1, t), m - s)) for m, s in done]
    path = [p + [-1] * (case["depth"] - len(p)) for p in paths]
    shape = (blocks, case["hkv"], BLOCK, case["d"])
    fill = [[_rows(g, blocks, case["hkv"] * BLOCK, case["d"], DTYPES[case["dtype"]], 1.0).view(shape) for _ in "kv"]
            for _ in range(case["layers"])]
    return dict(lens=lens, paths=paths, tables=tables, blocks=blocks, pools=fill, path=_ints(path),
                count=_ints([m for m, _ in done]), cu=_ints(list(range(0, t * len(lens) + 1, t))),
                seq_lens=_ints(lens))


# ------------------------------------------------------------ plain forms
def _ancestors(parents):
    """[T][T] truth values: node j is node i or above it; steps up the tree, doubled until they pass its root."""
    t = len(parents)
    seen = torch.eye(t, device="cuda") + (parents[:, None] == torch.arange(t, device="cuda")).float()
    for _ in range(t.bit_length()):
        seen = (seen @ seen > 0).float()
    return seen > 0


def _run_tree(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out, lse = [], []
    at = 0
    for b, (n, t) in enumerate(zip(s["lens"], s["nodes"])):
        j = torch.arange(n, device="cuda")
        blk, off = s["tables"][b][j // BLOCK].long(), j % BLOCK
        k, v = (s[x][blk, :, off].float().transpose(0, 1) for x in ("pool_k", "pool_v"))  # [Hkv][n][D]
        q = s["q"][at:at + t].float().view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
        x = (q @ k.transpose(1, 2) * s["scale"]).view(hkv, hq // hkv, t, n)
        x[..., n - t:].masked_fill_(~_ancestors(s["parents"][at:at + t]), -math.inf)
        m = x.amax(-1, keepdim=True)
        x = x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        o = (x.view(hkv, -1, n) @ v).view(hkv, hq // hkv, t, d) / l
        out.append(o.permute(2, 0, 1, 3).reshape(t, hq, d))
        lse.append((m + torch.log(l)).permute(2, 0, 1, 3).reshape(t, hq))
        at += t
    return {"out": torch.cat(out).to(DTYPES[c["out"]]), "lse": torch.cat(lse)}


def _run_verify(s):
    """All sequences at once, a level of the trees at a time; sums in 64 bits (a draw lies between two of them)."""
    c = s["case"]
    batch, nodes, depth = c["batch"], c["nodes"], s["max_path"]
    parents, tokens = s["parents"].view(batch, nodes), s["tokens"].view(batch, nodes).long()
    u = s["accept_u"].view(batch, nodes).double()
    seq = torch.arange(batch, device="cuda")
    node = torch.zeros(batch, dtype=torch.long, device="cuda")
    count = torch.zeros_like(node)
    path = torch.full((batch, depth), -1, dtype=torch.long, device="cuda")
    ended = torch.zeros(batch, dtype=torch.bool, device="cuda")
    drawn_from = None
    for level in range(depth + 1):
        p0 = s["p"][seq * nodes + node].double()
        p = p0
        taken = torch.full_like(node, -1)
        if level < depth:
            q = s["q"][seq * nodes + node].double() if c["drawn"] else None
            is_child = parents == node[:, None]
            rank = is_child.cumsum(1)
            for k in range(1, s["children"] + 1):
                here = is_child & (rank == k)
                child = here.int().argmax(1)
                live = here.any(1) & (taken < 0)
                x = tokens[seq, child]
                px = p[seq, x]
                ok = u[seq, child] * (q[seq, x] if c["drawn"] else 1.0) < px
                taken = torch.where(live & ok, child, taken)
                if c["drawn"]:
                    left = (p - q).clamp(min=0)
                else:
                    left = p.scatter(1, x[:, None], 0.0)
                total = left.sum(1, keepdim=True) if c["drawn"] else 1 - px[:, None]
                left = torch.where(total > 0, left / total.clamp(min=1e-300), torch.zeros_like(left))
                p = torch.where((live & ~ok)[:, None], left, p)
        # nothing left: the draw is from p itself
        p = torch.where(p.sum(1, keepdim=True) > 0, p, p0)
        drawn_from = p if drawn_from is None else torch.where(ended[:, None], drawn_from, p)
        ended = ended | (taken < 0)
        if level < depth:
            path[:, level] = torch.where(ended, path[:, level], taken)
            count = torch.where(ended, count, count + 1)
            node = torch.where(ended, node, taken)
    sums = drawn_from.cumsum(1)
    point = s["sample_u"].double()[:, None] * sums[:, -1:]
    token = (sums > point).int().argmax(1)
    emitted = torch.cat([torch.where(path >= 0, tokens.gather(1, path.clamp(min=0)), path), path[:, :1] * 0 - 1], 1)
    emitted[seq, count] = token
    return {"accepted": count.int(), "path": path.int(), "tokens": emitted.int()}


def _run_keep(s):
    m = s["count"]
    depth = s["path"].shape[1]
    i = torch.arange(depth, device="cuda")
    live = i[None] < m[:, None]
    first = (s["seq_lens"] - (s["cu"][1:] - s["cu"][:-1])).long()[:, None]
    src = (first + torch.where(live, s["path"], 0)).clamp(max=s["tables"].shape[1] * BLOCK - 1)
    dst = first + torch.where(live, i[None] + 1, 0)  # places that nothing is moved to keep the root
    dst = dst.clamp(max=s["tables"].shape[1] * BLOCK - 1)
    sb, so = s["tables"].gather(1, src // BLOCK).long(), src % BLOCK
    db, do = s["tables"].gather(1, dst // BLOCK).long(), dst % BLOCK
    out = {}
    for layer, pools in enumerate(s["pools"]):
        for name, x in zip("kv", pools):
            x[db, :, do] = x[sb, :, so]
            out[f"{name}{layer}"] = x
    out["seq_lens"] = first[:, 0].int() + 1 + m
    return out


# ------------------------------------------------------ the library's calls
class _Pool:
    """A library pool, destroyed with its last reference."""

    def __init__(self, blocks, hkv, d, dtype):
        import paged_kv_cache_196_gb300 as pk
        self.pk = pk
        self.handle = pk.kv_pool_create(blocks, BLOCK, hkv, d, _own_dtype(pk, dtype))

    def __del__(self):
        self.pk.kv_pool_destroy(self.handle)

    def views(self, shape, dtype):
        """Torch tensors over the pool's K and V arrays."""
        class Raw:
            pass
        out = []
        for ptr in self.pk.kv_pool_ptrs(self.handle):
            raw = Raw()
            raw.pool = self  # the tensors keep the pool
            raw.__cuda_array_interface__ = dict(shape=shape, typestr="<f4" if dtype == torch.float32 else "<i2",
                                                data=(ptr, False), version=3, strides=None)
            out.append(torch.as_tensor(raw, device="cuda").view(dtype))
        return out


def _own_dtype(pk, name):
    return {"f32": pk.KV_F32, "bf16": pk.KV_BF16, "f16": pk.KV_F16}[name]


def _own_tree(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    pk.paged_tree_attention(s["pool"].handle, s["q"], s["cu"], s["q"].shape[0], max(s["nodes"]), s["parents"],
                            s["tables"], s["tables"].shape[1], s["seq_lens"], c["batch"], c["hq"], s["scale"],
                            s["out"], s["out_dt"], s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    pk.kv_verify_tree(s["pool"].handle, s["p"], s.get("q"), s["dt"], c["vocab"], s["cu"], s["p"].shape[0], c["nodes"],
                      s["parents"], s["tokens"], s["accept_u"], s["sample_u"], c["batch"], s["max_path"],
                      s["count"], s["path"], s["emitted"])
    return {"accepted": s["count"], "path": s["path"], "tokens": s["emitted"]}


def _own_keep(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    pk.kv_keep_path(s["handles"], s["cu"], c["nodes"], s["path"], c["depth"], s["count"], s["tables"],
                    s["tables"].shape[1], s["seq_lens"], c["batch"], s["new_lens"])
    out = {f"{name}{layer}": x for layer, pools in enumerate(s["pools"]) for name, x in zip("kv", pools)}
    out["seq_lens"] = s["new_lens"]
    return out


def _prepare_tree(case, seed):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    s = _tree_inputs(case, seed)
    k, v, slots = s.pop("k"), s.pop("v"), s.pop("slots")
    s["case"], s["scale"] = case, 1 / math.sqrt(d)
    if not own:
        for name, rows in (("pool_k", k), ("pool_v", v)):
            s[name] = torch.zeros(s["blocks"], hkv, BLOCK, d, dtype=dt, device="cuda")
            s[name][slots // BLOCK, :, slots % BLOCK] = rows
        return s
    import paged_kv_cache_196_gb300 as pk
    s["pool"] = _Pool(s["blocks"], hkv, d, case["dtype"])
    s["out_dt"] = _own_dtype(pk, case["out"])
    pk.kv_append(s["pool"].handle, k, v, slots, len(slots))
    s["out"] = torch.empty(s["q"].shape[0], hq, d, dtype=DTYPES[case["out"]], device="cuda")
    s["lse"] = torch.empty(s["q"].shape[0], hq, dtype=torch.float32, device="cuda")
    s["ws_bytes"] = pk.kv_tree_workspace_size(s["pool"].handle, case["batch"], hq, s["tables"].shape[1],
                                              max(s["nodes"]))
    s["ws"] = torch.empty(max(s["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()  # the rows appended here are dropped
    return s


def prepare(case, seed):
    if case["op"] == "tree":
        return _prepare_tree(case, seed)
    s = _verify_inputs(case, seed) if case["op"] == "verify" else _keep_inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import paged_kv_cache_196_gb300 as pk
    if case["op"] == "verify":
        # the pool of the step: its device and its error word
        s["pool"], s["dt"] = _Pool(1, 1, 64, "f32"), _own_dtype(pk, case["dtype"])
        s["count"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
        s["path"] = torch.empty(case["batch"], s["max_path"], dtype=torch.int32, device="cuda")
        s["emitted"] = torch.empty(case["batch"], s["max_path"] + 1, dtype=torch.int32, device="cuda")
        return s
    shape = (s["blocks"], case["hkv"], BLOCK, case["d"])
    s["own_pools"] = [_Pool(s["blocks"], case["hkv"], case["d"], case["dtype"]) for _ in s["pools"]]
    views = [p.views(shape, DTYPES[case["dtype"]]) for p in s["own_pools"]]
    for mine, given in zip(views, s["pools"]):
        for x, y in zip(mine, given):
            x.copy_(y)
    s["pools"], s["handles"] = views, [p.handle for p in s["own_pools"]]
    s["new_lens"] = torch.empty(case["batch"], dtype=torch.int32, device="cuda")
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "verify": _own_verify, "keep": _own_keep}[op](state)
    return {"tree": _run_tree, "verify": _run_verify, "keep": _run_keep}[op](state)


# ------------------------------------------------------------ in 64 bits
def _exact_tree(case, seed):
    s = _tree_inputs(case, seed)
    hq, d = case["hq"], case["d"]
    g = hq // case["hkv"]
    rows = s["q"].shape[0]
    out = torch.empty(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(rows, hq, dtype=torch.float64, device="cuda")
    at = row = 0
    for n, t, tree in zip(s["lens"], s["nodes"], s["trees"]):
        seen = torch.ones(t, n, dtype=torch.bool)
        seen[:, n - t:] = False
        for i in range(t):
            j = i
            while j >= 0:
                seen[i, n - t + j] = True
                j = tree[j]
        seen = seen.cuda()
        for h in range(hq):
            x = s["q"][row:row + t, h].double() @ s["k"][at:at + n, h // g].double().T / math.sqrt(d)
            x = torch.where(seen, x, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[row:row + t, h] = z
            out[row:row + t, h] = torch.exp(x - z[:, None]) @ s["v"][at:at + n, h // g].double()
        at += n
        row += t
    return {"out": out, "lse": lse}


def _exact_verify(case, seed):
    s = _verify_inputs(case, seed)
    nodes, depth = case["nodes"], s["max_path"]
    tokens, accept_u, sample_u = s["tokens"].tolist(), s["accept_u"].tolist(), s["sample_u"].tolist()
    counts, paths, emitted = [], [], []
    for b, tree in enumerate(s["trees"]):
        at, way = 0, []
        while True:
            row = s["p"][b * nodes + at].double()
            left = row.clone()
            step = None
            for child in [i for i in range(at + 1, nodes) if tree[i] == at]:
                if len(way) == depth:
                    break
                x = tokens[b * nodes + child]
                q = s["q"][b * nodes + at].double() if case["drawn"] else None
                if accept_u[b * nodes + child] * (q[x].item() if case["drawn"] else 1.0) < left[x].item():
                    step = child
                    break
                if case["drawn"]:
                    left = torch.relu(left - q)
                    mass = left.sum().item()
                else:
                    mass = 1 - left[x].item()
                    left[x] = 0
                left = left / mass if mass > 0 else torch.zeros_like(left)
            if step is None:
                break
            way.append(step)
            at = step
        if left.sum().item() <= 0:
            left = row
        sums = torch.cumsum(left, 0)
        point = torch.full((1,), sample_u[b] * sums[-1].item(), dtype=torch.float64, device="cuda")
        token = int(torch.searchsorted(sums, point, right=True).item())
        counts.append(len(way))
        paths.append(way + [-1] * (depth - len(way)))
        words = [tokens[b * nodes + i] for i in way] + [token]
        emitted.append(words + [-1] * (depth + 1 - len(words)))
    return {"accepted": _ints(counts), "path": _ints(paths), "tokens": _ints(emitted)}


def _exact_keep(case, seed):
    s = _keep_inputs(case, seed)
    first = [n - case["nodes"] for n in s["lens"]]
    tables = s["tables"].tolist()
    out = {}

    def place(b, j):
        return tables[b][j // BLOCK], j % BLOCK

    moves = [(place(b, first[b] + src), place(b, first[b] + i + 1)) for b, way in enumerate(s["paths"])
             for i, src in enumerate(way) if src != i + 1]
    for layer, pools in enumerate(s["pools"]):
        for name, x in zip("kv", pools):
            y = x.clone()
            if moves:
                sb, so, db, do = (_ints([m[i][j] for m in moves], torch.int64) for i in (0, 1) for j in (0, 1))
                y[db, :, do] = x[sb, :, so]
            out[f"{name}{layer}"] = y
    out["seq_lens"] = _ints([f + 1 + len(way) for f, way in zip(first, s["paths"])])
    return out


def exact(case, seed):
    return {"tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](case, seed)
