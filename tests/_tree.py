"""What the tests of drafted tokens share: caches with trees at their ends, 64-bit
references, and how far a kernel may be off.

Error of an attention output, derived from the arithmetic and not from runs.  Products
of 16-bit values are exact in fp32, those of fp32 values off by 2^-24; a sum of D of them in
fp32 in any order by (D + 1) 2^-24 of the sum of magnitudes A.  Scaling a score and taking
its distance to the reference adds roundings of 2^-24 of the score's and the distance's size (in
log2 units: times log2 e, and back).  So a score is off by
  ds = scale A (D + 2) 2^-24 + 4 |s|max 2^-24,
with |s|max <= scale A, a weight by the factor exp(ds) and the exponential's own 2^-22, and,
where it is held in two parts of a 16-bit type of half step h, by h^2 (in three, by h^3).  Sums over n keys, in
any order and piecewise: n 2^-24 of the sum of magnitudes, numerator and denominator; the
merge of up to n pieces scales each once more (2^-22).  With |o| <= V = max |v|:
  |error of o| <= V (2 ds + 2 (2^-21 + h^2 or h^3) + 2 n 2^-24) + half step of the output * |o|
  |error of lse| <= ds + 2^-21 + n 2^-24 + 4 |lse| 2^-24.
(h^2 once for the numerator; twice leaves room for second order terms.)
"""
import math

import numpy as np
import torch

import paged_kv_cache_196_gb300 as pk

KV = {"f32": pk.KV_F32, "bf16": pk.KV_BF16, "f16": pk.KV_F16}
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def random_parents(rng, nodes, kind):
    """Parents of a tree by index: a chain, a star, a random tree, or a forest (-1 beside the root)."""
    if nodes == 0:
        return []
    if kind == "chain":
        return list(range(-1, nodes - 1))
    if kind == "star":
        return [-1] + [0] * (nodes - 1)
    if kind == "forest":
        return [-1] + [int(rng.integers(-1, i)) for i in range(1, nodes)]
    return [-1] + [int(rng.integers(0, i)) for i in range(1, nodes)]


def ancestors(parents):
    """Sets of each node and the nodes above it."""
    out = []
    for i in range(len(parents)):
        s, j = set(), i
        while j >= 0:
            s.add(j)
            j = parents[j]
        out.append(s)
    return out


class TreeCase:
    """A pool of shuffled blocks, filled row by row; what no token owns is NaN."""

    def __init__(self, dtype, d, hkv, g, cached, nodes, kind="tree", seed=0, spare=3, width=0, q_size=1.0, garbage=None):
        self.dtype, self.d, self.hkv, self.g, self.hq = dtype, d, hkv, g, hkv * g
        self.cached, self.nodes = list(cached), list(nodes)
        self.lens = [c + t for c, t in zip(cached, nodes)]
        self.batch = len(self.lens)
        self.scale = 1 / math.sqrt(d)
        rng = np.random.default_rng(seed)
        self.parents = [random_parents(rng, t, kind) for t in nodes]
        need = [-(-n // 16) for n in self.lens]
        self.width = max(1, max(need), width)
        self.blocks = sum(need) + spare
        ids = rng.permutation(self.blocks)
        self.tables = np.full((self.batch, self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        t = torch.Generator().manual_seed(seed)

        def rows(n, heads, size):
            return (torch.randn(n, heads, d, generator=t) * size).to(DT[dtype])
        self.k = [rows(n, hkv, 1.0) for n in self.lens]
        self.v = [rows(n, hkv, 1.0) for n in self.lens]
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.total = int(self.cu[-1])
        self.q = rows(self.total, self.hq, q_size)
        self.pool = pk.kv_pool_create(self.blocks, 16, hkv, d, KV[dtype])
        self.k_view, self.v_view = views(self.pool, self.blocks, hkv, d, dtype)
        self.k_view.fill_(math.nan if garbage is None else garbage)
        self.v_view.fill_(math.nan if garbage is None else garbage)
        for b, n in enumerate(self.lens):
            if n:
                self.write(b)

    def widen(self, width):
        """Tables of that many columns."""
        self.tables = np.concatenate([self.tables, np.full((self.batch, width - self.width), -1, np.int32)], 1)
        self.width = width

    def slots(self, b, n=None):
        j = np.arange(self.lens[b] if n is None else n)
        return self.tables[b, j // 16].astype(np.int64) * 16 + j % 16

    def write(self, b):
        s = torch.from_numpy(self.slots(b)).cuda()
        self.k_view[s // 16, :, s % 16] = self.k[b].cuda()
        self.v_view[s // 16, :, s % 16] = self.v[b].cuda()

    def flat_parents(self):
        return torch.tensor(sum(self.parents, []), dtype=torch.int32)

    def args(self, out_dtype=None, chain=False, rows=0, max_q_len=None):
        """Device buffers of a call; `rows` more rows of q and out behind the last tree."""
        out_dtype = out_dtype or self.dtype
        total = self.total + rows
        a = dict(out_dtype=out_dtype, total=total, max_q_len=max_q_len or max(1, max(self.nodes)))
        a["q"] = torch.zeros(max(1, total), self.hq, self.d, dtype=DT[self.dtype])
        a["q"][:self.total] = self.q
        a["q"] = a["q"].cuda()
        a["cu"] = torch.from_numpy(self.cu).cuda()
        parents = torch.zeros(max(1, total), dtype=torch.int32)
        parents[:self.total] = self.flat_parents()
        a["parents"] = None if chain else parents.cuda()
        a["tables"] = torch.from_numpy(self.tables).cuda()
        a["lens"] = torch.tensor(self.lens, dtype=torch.int32).cuda()
        a["out"] = torch.full((max(1, total), self.hq, self.d), 777.0, dtype=DT[out_dtype], device="cuda")
        a["lse"] = torch.full((max(1, total), self.hq), 777.0, device="cuda")
        n = pk.kv_tree_workspace_size(self.pool, self.batch, self.hq, self.width, a["max_q_len"])
        a["ws_bytes"] = n
        a["ws"] = torch.full((max(4, n // 4),), math.nan, device="cuda")
        return a

    def call(self, a, stream=None, lse=True):
        pk.paged_tree_attention(self.pool, a["q"], a["cu"], a["total"], a["max_q_len"], a["parents"], a["tables"],
                                self.width, a["lens"], self.batch, self.hq, self.scale, a["out"], KV[a["out_dtype"]],
                                a["lse"] if lse else None, a["ws"], a["ws_bytes"], stream=stream)

    def reference(self, gone=(), out_dtype=None):
        """out, lse in 64 bits and the bounds of their errors; `gone`: (sequence, block index) pairs whose
        keys are left out."""
        out = np.zeros((self.total, self.hq, self.d))
        lse = np.full((self.total, self.hq), -np.inf)
        out_tol, lse_tol = np.zeros(out.shape), np.zeros(lse.shape)
        h = 0.0 if self.dtype == "f32" else HALF[self.dtype]
        parts = h ** (3 if (self.dtype, out_dtype) == ("bf16", "f32") else 2)
        for b, (n, t) in enumerate(zip(self.lens, self.nodes)):
            if not t:
                continue
            r0 = int(self.cu[b])
            q = self.q[r0:r0 + t].double().numpy()
            k, v = self.k[b].double().numpy(), self.v[b].double().numpy()
            seen = np.zeros((t, n), bool)
            for i, s in enumerate(ancestors(self.parents[b])):
                seen[i, :n - t] = True
                for j in s:
                    seen[i, n - t + j] = True
            for bb, block in gone:
                if bb == b:
                    seen[:, 16 * block:16 * block + 16] = False
            for hq in range(self.hq):
                kh, vh = k[:, hq // self.g], v[:, hq // self.g]
                with np.errstate(invalid="ignore"):
                    s = q[:, hq] @ kh.T * self.scale
                s = np.where(seen, s, -np.inf)
                m = s.max(1, keepdims=True)
                m[m == -np.inf] = 0
                with np.errstate(invalid="ignore"):
                    w = np.exp(s - m)
                l = w.sum(1, keepdims=True)
                for i in range(t):
                    if not l[i, 0] == 0:
                        lse[r0 + i, hq] = m[i, 0] + math.log(l[i, 0]) if l[i, 0] == l[i, 0] else math.nan
                        keys = np.flatnonzero(seen[i])
                        out[r0 + i, hq] = (w[i, keys] / l[i, 0]) @ vh[keys]
                with np.errstate(invalid="ignore"):
                    a = np.where(seen, np.abs(q[:, hq]) @ np.abs(kh).T * self.scale, 0).max(1)
                ds = a * (self.d + 6) * 2.0 ** -24
                big = np.abs(np.where(seen[:, :, None], vh[None], 0)).max((1, 2)) if n else np.zeros(t)
                out_tol[r0:r0 + t, hq] = (big * (2 * ds + 2 * (2.0 ** -21 + parts) + 2 * n * 2.0 ** -24))[:, None]
                lse_tol[r0:r0 + t, hq] = ds + 2.0 ** -21 + n * 2.0 ** -24 + 4 * 2.0 ** -24 * np.abs(
                    np.where(np.isfinite(lse[r0:r0 + t, hq]), lse[r0:r0 + t, hq], 0))
        return out, lse, out_tol, lse_tol

    def check(self, a, gone=(), err=0, rows=None):
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(self.pool) == err
        out, lse, out_tol, lse_tol = self.reference(gone, a["out_dtype"])
        got, got_lse = a["out"].double().cpu().numpy()[:self.total], a["lse"].double().cpu().numpy()[:self.total]
        keep = np.ones(self.total, bool) if rows is None else rows
        with np.errstate(invalid="ignore"):
            bound = out_tol + HALF[a["out_dtype"]] * np.abs(out)
            bad = (np.abs(got - out) > bound) | ~np.isfinite(got)
            bad_lse = ~((got_lse == lse) | (np.abs(got_lse - lse) <= lse_tol))
        bad[~keep] = bad_lse[~keep] = False
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], out[bad][:5], bound[bad][:5])
        assert not bad_lse.any(), (np.argwhere(bad_lse)[:5], got_lse[bad_lse][:5], lse[bad_lse][:5])
        if a["total"] > self.total:  # rows of no tree
            assert (a["out"][self.total:] == 777).all() and (a["lse"][self.total:] == 777).all()

    def close(self):
        pk.kv_pool_destroy(self.pool)


class _Raw:
    pass


def views(pool, blocks, hkv, d, dtype):
    """Torch tensors over a pool's K and V."""
    out = []
    for ptr in pk.kv_pool_ptrs(pool):
        raw = _Raw()
        raw.__cuda_array_interface__ = dict(shape=(blocks, hkv, 16, d), typestr="<f4" if dtype == "f32" else "<i2",
                                            data=(ptr, False), version=3, strides=None)
        out.append(torch.as_tensor(raw, device="cuda").view(DT[dtype]))
    return out


# ------------------------------------------------------------ verification
def verify_reference(p, q, cu, parents, tokens, accept_u, sample_u, max_path, vocab):
    """The walk in 64 bits with Python's exact integers where a border decides: p, q as lists of float64 arrays."""
    counts, paths, emitted = [], [], []

    def clean(x):
        with np.errstate(invalid="ignore"):
            return np.where(x > 0, np.minimum(x, 1.0), 0.0)
    for b in range(len(cu) - 1):
        q0, t = int(cu[b]), int(cu[b + 1] - cu[b])
        at, way = 0, []
        word = -1
        while t:
            row = clean(p[q0 + at])
            left, mass = row.copy(), 1.0
            step = None
            if len(way) < max_path:
                for c in range(at + 1, t):
                    up, x = int(parents[q0 + c]), int(tokens[q0 + c])
                    if up != at or x < 0 or x >= vocab or mass <= 0:
                        continue
                    qx = clean(q[q0 + at])[x] if q is not None else 1.0
                    if float(accept_u[q0 + c]) * qx * mass < left[x]:
                        step = c
                        break
                    if q is not None:
                        left = np.maximum(left - mass * clean(q[q0 + at]), 0)
                        mass = math.fsum(left)
                    else:
                        mass -= left[x]
                        left[x] = 0
            if step is None:
                break
            way.append(step)
            at = step
        if t:
            if math.fsum(left) <= 0:
                left = row
            total = math.fsum(left)
            if total > 0:
                u = min(max(float(sample_u[b]), 0.0), 1 - 2.0 ** -24)
                sums = np.cumsum(left)
                word = int(np.searchsorted(sums, u * sums[-1], side="right"))
        counts.append(len(way))
        paths.append(way + [-1] * (max_path - len(way)))
        w = [int(tokens[q0 + i]) for i in way] + [word]
        emitted.append(w + [-1] * (max_path + 1 - len(w)))
    return np.array(counts), np.array(paths).reshape(len(counts), max_path), np.array(emitted)
