"""Plain numpy forms of the rotary append and the 4-bit cache, and the device
objects their tests share.  Rotation: the formula in fp32 operations, as the
library documents it.  Everything else: 64 bits."""
import math

import numpy as np
import torch

import paged_kv_cache_196_gb300 as pk
from _gpu import require_cuda

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KV = {"f32": pk.KV_F32, "bf16": pk.KV_BF16, "f16": pk.KV_F16}
HALF_STEP = {x: torch.finfo(t).eps / 2 for x, t in TORCH.items()}  # of a rounding, relative
# Half the spacing of a type's subnormals: a value below its smallest normal number
# (fp16: 2^-14, spacing 2^-24) is rounded by up to that, however small it is.
HALF_FLOOR = {x: torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2 for x, t in TORCH.items()}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()


def rope_table(max_pos, rot, base=10000.0):
    """[max_pos][rot / 2 cos, rot / 2 sin], fp32 of 64-bit angles."""
    a = np.arange(max_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate32(x, cs, rot, interleaved):
    """x [T][H][D] fp32, cs [T][rot]: two products and a sum, each rounded to fp32."""
    x = x.astype(np.float32).copy()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if interleaved:
        i1, i2 = slice(0, rot, 2), slice(1, rot, 2)
    else:
        i1, i2 = slice(0, rot // 2), slice(rot // 2, rot)
    x1, x2 = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1] = x1 * c - x2 * s
    x[..., i2] = x2 * c + x1 * s
    return x


# every finite e4m3 value >= 0 in order: code e m -> value
E4M3 = np.array([(m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
                 for e in range(16) for m in range(8)][:127])


def e4m3_round(x):
    """x >= 0 (64-bit) to the nearest e4m3, ties to the even code, at most 448."""
    x = np.minimum(x, E4M3[-1])
    hi = np.searchsorted(E4M3, x).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - E4M3[lo], E4M3[hi] - x
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (E4M3[hi] == x)
    return np.where(up, E4M3[hi], E4M3[lo])


def stored(x, g=1.0):
    """What a 4-bit pool of scale g keeps of x [..., D]."""
    x = np.asarray(x, np.float64) / g
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.abs(b).max(-1, keepdims=True)  # NaN propagates
        s = np.where(np.isnan(m), np.nan, e4m3_round(np.where(np.isnan(m), 0, m) / 7))
        c = np.clip(np.rint(np.clip(b, -1e30, 1e30) / np.where(s == 0, 1, s)), -7, 7)
        c = np.where(s == 0, 0, c)
        out = np.where(np.isnan(s), np.nan, c * s * g)
    return out.reshape(x.shape)


def attend(q, k, v, scale, seen):
    """q [T][Hq][D], k, v [n][Hkv][D] (64-bit), row i sees keys < seen[i].

    Returns o, lse, and per (row, head) the mean |v| under the weights [T][Hq][D]
    the largest sum |q||k| of a seen key [T][Hq] and the largest |v|, for error bounds."""
    T, hq, d = q.shape
    g = hq // k.shape[1]
    o, av = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    lse, mag = np.full((T, hq), -np.inf), np.zeros((T, hq))
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        for i in range(T):
            n = seen[i]
            if n == 0:
                continue
            s = scale * (kh[:n] @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            lse[i, h] = m + math.log(w.sum())
            w /= w.sum()
            o[i, h], av[i, h] = w @ vh[:n], w @ np.abs(vh[:n])
            mag[i, h] = (np.abs(kh[:n]) @ np.abs(q[i, h])).max()
    return o, lse, av, mag, np.abs(v).max(initial=0.0)


def check_attention(out, lse, ref, scale, n_keys, out_type, weight_step, what="", floor=2.0 ** -31):
    """Bounds: a score is an fp32 sum of exact products (D + 8 roundings of at most
    2^-23 of sum |q||k|, the tensor core truncating); a weight's relative error is twice
    that times the softmax scale (numerator and denominator), 2^-21 for the
    exponential, and weight_step for its rounding; o sums n / 16 tiles in fp32; out
    is rounded once to its type.  floor: the smallest weights are fp16 subnormals,
    whose half spacing is 2^-25 however small they are, where the largest weight is at
    least 2^6 (the 4-bit decode's; its second part is rounded alike): 2^-31 of it per key."""
    o, ref_lse, av, mag, vmax = ref
    d = o.shape[-1]
    ds = abs(scale) * mag * (d + 8) * 2.0 ** -23
    rel = weight_step + 2 * ds + 2.0 ** -20 + (n_keys / 16 + 32) * 2.0 ** -22
    tol = av * rel[..., None] + HALF_STEP[out_type] * np.abs(o) * (1 + rel[..., None]) + floor * n_keys * vmax + HALF_FLOOR[out_type]
    assert np.all(np.isfinite(out)), what
    bad = np.abs(out - o) > tol
    assert not bad.any(), f"{what}: {np.abs(out - o)[bad].max():.3e} over {tol[bad].min():.3e} at {np.argwhere(bad)[0]}"
    if lse is not None:
        fin = np.isfinite(ref_lse)
        assert np.all(np.isneginf(lse[~fin])), what
        tol = ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(ref_lse, where=fin, out=np.zeros_like(ref_lse))
        assert np.all(np.abs(lse[fin] - ref_lse[fin]) <= tol[fin]), f"{what}: lse"


class Cache:
    """Ragged sequences in a 4-bit pool with shuffled blocks, the rows appended by
    the library; kv, vv: what the pool stands for (64-bit, per sequence)."""

    def __init__(self, lens, hkv, d, dtype="bf16", seed=1, k_scale=0.5, v_scale=0.25, extra=3, poison=True,
                 num_blocks=None):
        require_cuda()
        rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.d, self.dtype = np.asarray(lens, np.int32), hkv, d, dtype
        need = [-(-int(n) // 16) for n in lens]
        self.nb = num_blocks or sum(need) + extra
        self.width = max(1, max(need))
        order = rng.permutation(self.nb)[:sum(need)] if num_blocks is None else self.nb - 1 - rng.permutation(sum(need))
        self.tables = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        self.pool = pk.kv_pool_create(self.nb, 16, hkv, d, pk.KV_I4)
        pk.kv_pool_set_i4_scales(self.pool, k_scale, v_scale)
        if poison:  # every byte 0xff: codes of 7, scales that are NaN
            raw_bytes(pk.kv_pool_ptrs(self.pool)[0], self.nb * hkv * 18 * d).fill_(255)
        rows = [torch.from_numpy(rng.standard_normal((max(int(n), 1), hkv, d)).astype(np.float32))[:int(n)] for n in lens]
        self.k = [(x * torch.from_numpy(np.exp(0.5 * rng.standard_normal((1, hkv, d))).astype(np.float32))).to(TORCH[dtype])
                  for x in rows]
        self.v = [torch.from_numpy(rng.standard_normal((int(n), hkv, d)).astype(np.float32) * 0.7).to(TORCH[dtype]) for n in lens]
        self.slots = [self.tables[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16 for b, n in enumerate(lens)]
        total = int(self.lens.sum())
        if total:
            pk.kv_append_rope(self.pool, torch.cat(self.k).cuda(), torch.cat(self.v).cuda(), KV[dtype],
                              torch.from_numpy(np.concatenate(self.slots)).cuda(), total)
            torch.cuda.synchronize()
        self.kv = [stored(f64(x), k_scale) for x in self.k]
        self.vv = [stored(f64(x), v_scale) for x in self.v]
        self.t_tables, self.t_lens = torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda()

    def queries(self, rows, hq, dtype, seed=5):
        rng = np.random.default_rng(seed)
        return torch.from_numpy(rng.standard_normal((rows, hq, self.d)).astype(np.float32)).to(TORCH[dtype]).cuda()

    def decode(self, q, q_dtype, out_type, splits=0, tables=None, lens=None, scale=None, order=None, expect=0, stream=None):
        B, hq, d = q.shape
        out = torch.empty(B, hq, d, dtype=TORCH[out_type], device="cuda").fill_(7)
        lse = torch.empty(B, hq, dtype=torch.float32, device="cuda")
        ws_bytes = pk.kv_decode_workspace_size(B, hq, self.hkv, d, self.width, splits)
        ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device="cuda")
        pk.paged_decode_attention_i4(self.pool, q, KV[q_dtype], self.t_tables if tables is None else tables, self.width,
                                     self.t_lens if lens is None else lens, B, hq, scale or d ** -0.5, out, KV[out_type],
                                     lse, splits, ws, ws_bytes, seq_order=order, stream=stream)
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(self.pool) == expect
        return out, lse

    def prefill(self, q, q_dtype, out_type, cu, max_q, tables=None, lens=None, expect=0):
        rows, hq, d = q.shape
        out = torch.empty(rows, hq, d, dtype=TORCH[out_type], device="cuda").fill_(7)
        lse = torch.empty(rows, hq, dtype=torch.float32, device="cuda").fill_(7)
        B = len(cu) - 1
        n = pk.kv_prefill_i4_workspace_size(self.pool, B, hq, self.width, max_q)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        pk.paged_prefill_attention_i4(self.pool, q, KV[q_dtype], torch.from_numpy(np.asarray(cu, np.int32)).cuda(), rows,
                                      max_q, self.t_tables if tables is None else tables, self.width,
                                      self.t_lens if lens is None else lens, B, hq, d ** -0.5, out, KV[out_type], lse, ws, n)
        torch.cuda.synchronize()
        assert pk.kv_get_device_error(self.pool) == expect
        return out, lse

    def close(self):
        pk.kv_pool_destroy(self.pool)


class _Raw:
    pass


def raw_bytes(ptr, n):
    r = _Raw()
    r.__cuda_array_interface__ = {"shape": (n,), "typestr": "|u1", "data": (ptr, False), "version": 3, "strides": None}
    return torch.as_tensor(r, device="cuda")
