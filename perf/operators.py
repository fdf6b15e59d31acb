"""Cases that measure the rotary append and the 4-bit cache: the append with
its position rotation, the quantising append with the read of what it stored,
decode attention and chunked prefill attention over a 4-bit pool.

With ``own`` false ``run`` computes an operator from elementary torch
operations; with ``own`` true it makes the library's calls.

A 4-bit pool holds, for every 16 consecutive dimensions of one (token, kv
head), sixteen integers c in -7..7 and one e4m3 scale s; the value is
c * s * g with g the pool's power-of-two scale of K or V.  s is the e4m3
nearest to max|x| / (7 g), c the integer nearest to x / (s g) (ties to even).
"""
import math

import torch

own = False

BLOCK = 16  # tokens per block
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
K_SCALE, V_SCALE = 0.5, 0.125  # a 4-bit pool's scales in these cases


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the head of every decode step: one new token of each of 64 sequences
        dict(name="rope step 64", op="rope", dtype="bf16", tokens=64, hq=32, hkv=8, d=128, rot=128,
             interleaved=False, max_pos=4096),
        # the chunk of a long-prompt prefill: 4 x 2048 tokens
        dict(name="rope chunk 8192", op="rope", dtype="bf16", tokens=8192, hq=56, hkv=8, d=128,
             rot=128, interleaved=False, max_pos=16384),
        # a small fp32 model that rotates half of each head in interleaved pairs, odd chunk
        dict(name="rope fp32 partial", op="rope", dtype="f32", tokens=1531, hq=12, hkv=4, d=64,
             rot=32, interleaved=True, max_pos=2048),
        # the same head of a step on a 4-bit pool
        dict(name="i4 append step 64", op="append", dtype="bf16", tokens=64, hq=32, hkv=8, d=128,
             rot=128, interleaved=False, max_pos=4096),
        # a prefill chunk into a 4-bit pool, read back for the next stage
        dict(name="i4 append chunk 8192", op="append", dtype="bf16", tokens=8192, hq=56, hkv=8,
             d=128, rot=128, interleaved=False, max_pos=16384),
        # odd chunk, 64-wide heads, 7 query heads per kv head, fp16
        dict(name="i4 append odd f16", op="append", dtype="f16", tokens=2049, hq=14, hkv=2, d=64,
             rot=64, interleaved=True, max_pos=131072),
        # decode of 64 chat-length sequences
        dict(name="i4 decode 64 seqs", op="decode", dtype="bf16", out="bf16", batch=64, lo=512,
             hi=4096, hq=32, hkv=8, d=128),
        # decode of few very long contexts
        dict(name="i4 decode long", op="decode", dtype="bf16", out="bf16", batch=8, lo=32768,
             hi=196608, hq=32, hkv=4, d=128),
        # a nearly idle server: 3 short sequences, one query head per kv head, fp32 output
        dict(name="i4 decode 3 short", op="decode", dtype="f16", out="f32", batch=3, lo=1, hi=190,
             hq=8, hkv=8, d=64),
        # a large prefill step: 4 chunks of 2048 after 8192 cached tokens
        dict(name="i4 prefill 4x2048", op="prefill", dtype="bf16", out="bf16", batch=4, cached_lo=8192,
             cached_hi=8192, chunk_lo=2048, chunk_hi=2048, hq=56, hkv=8, d=128),
        # chunks of mixed lengths, one of a sequence that starts here
        dict(name="i4 prefill ragged", op="prefill", dtype="f16", out="f16", batch=6, cached_lo=0,
             cached_hi=3001, chunk_lo=33, chunk_hi=700, hq=32, hkv=8, d=128),
        # five drafted tokens of each sequence, checked in one step
        dict(name="i4 prefill drafts", op="prefill", dtype="bf16", out="bf16", batch=16,
             cached_lo=1000, cached_hi=8000, chunk_lo=5, chunk_hi=5, hq=32, hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode", "prefill"))
    dtype = rng.choice(("bf16", "f16"))
    hkv = rng.choice((1, 2, 3, 4, 8))
    g = rng.randint(1, 8)
    if op in ("rope", "append"):
        if rng.random() < 0.25:
            dtype = "f32"
        d = rng.choice((64, 128))
        # at most the values of the listed chunk
        most = 8192 * 72 * 128 * 2 // ((g + 2) * hkv * d * (4 if dtype == "f32" else 2))
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(most, 16384)), hq=g * hkv, hkv=hkv,
                    d=d, rot=rng.choice((d, d // 2, 16, 48)), interleaved=rng.random() < 0.5,
                    max_pos=_log(rng, 1024, 131072))
    if op == "decode":
        d = rng.choice((64, 128))
        batch = _log(rng, 1, 256)
        # at most the cache of the listed long contexts
        hi = _log(rng, 16, min(196608, 2_500_000 * 128 // (hkv * batch * d)))
        return dict(op=op, dtype=dtype, out=rng.choice((dtype, "f32")), batch=batch,
                    lo=_log(rng, 1, hi), hi=hi, hq=g * hkv, hkv=hkv, d=d)
    batch = _log(rng, 1, 16)
    chunk = _log(rng, 1, 2048)
    most = 4 * 2048 * 9000 * 56 // (batch * chunk * g * hkv)
    cached = _log(rng, 1, max(1, min(16384, most - chunk)))
    return dict(op=op, dtype=dtype, out=dtype, batch=batch, cached_lo=_log(rng, 1, cached),
                cached_hi=cached, chunk_lo=_log(rng, 1, chunk), chunk_hi=chunk, hq=g * hkv, hkv=hkv, d=128)


def _spread(batch, lo, hi):
    """`batch` lengths from lo to hi, evenly spaced (over their logarithm for long spans)."""
    if batch == 1:
        return [hi]
    if lo > 0 and hi > 4 * lo and hi > 8192:
        return [int(round(lo * (hi / lo) ** (i / (batch - 1)))) for i in range(batch)]
    return [lo + (hi - lo) * i // (batch - 1) for i in range(batch)]


def _lengths(case):
    """(tokens in the cache, tokens of the chunk) of each sequence."""
    if case["op"] == "decode":
        return [(n, 1) for n in _spread(case["batch"], case["lo"], case["hi"])]
    cached = _spread(case["batch"], case["cached_lo"], case["cached_hi"])
    chunk = _spread(case["batch"], case["chunk_lo"], case["chunk_hi"])[::-1]
    return [(c + t, t) for c, t in zip(cached, chunk)]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    e = 4 if case["dtype"] == "f32" else 2
    row4 = 2 * hkv * d * 9 // 16  # K and V of one token in a 4-bit pool
    if case["op"] in ("rope", "append"):
        t = case["tokens"]
        b = t * (hq + 2 * hkv) * d * e + t * hq * d * e + t * (8 + 4 + 4 * case["rot"])
        f = 3 * t * (hq + hkv) * case["rot"]
        if case["op"] == "rope":
            return {"bytes": b + t * 2 * hkv * d * e, "flops": f}
        return {"bytes": b + 2 * t * row4 + t * 2 * hkv * d * 2 + 8 * t, "flops": f + 6 * t * 2 * hkv * d}
    oe = 4 if case["out"] == "f32" else 2
    lens = _lengths(case)
    rows = sum(t for _, t in lens)
    pairs = sum(t * (n - t) + t * (t + 1) // 2 if case["op"] == "prefill" else n for n, t in lens)
    return {"bytes": sum(n for n, _ in lens) * row4 + rows * hq * (d * (e + oe) + 4) + sum(n for n, _ in lens) // 4,
            "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, heads, d, dtype, size, channels=False):
    """n rows of activations: normal values; keys have channels of unlike sizes."""
    x = torch.randn(n, heads, d, generator=g, device="cuda", dtype=torch.float32) * size
    if channels:
        x *= torch.exp(0.7 * torch.randn(1, heads, d, generator=g, device="cuda"))
    return x.to(dtype)


def _table(max_pos, rot):
    """cos and sin of every position: [max_pos][rot / 2 cosines, rot / 2 sines]."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def _append_inputs(case, seed):
    g = _gen(seed)
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    # the projections leave q, k and v side by side in one row per token
    qkv = torch.cat([_rows(g, t, hq, d, dt, 1.0), _rows(g, t, hkv, d, dt, 1.0, True),
                     _rows(g, t, hkv, d, dt, 0.4)], 1)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    blocks = t // BLOCK + 3
    slots = torch.randperm(blocks * BLOCK, generator=g, device="cuda")[:t]
    pos = torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda", dtype=torch.int32)
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, table=_table(case["max_pos"], case["rot"]), blocks=blocks)


def _cache_inputs(case, seed):
    """Rows of a cache of ragged sequences in shuffled blocks, and the queries."""
    g = _gen(seed)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device="cuda").tolist()]
    need = [-(-n // BLOCK) for n, _ in lens]
    width, blocks = max(1, max(need)), sum(need) + 2
    order = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    j = [torch.arange(n, device="cuda") for n, _ in lens]
    slots = torch.cat([tables[b, x // BLOCK].long() * BLOCK + x % BLOCK for b, x in enumerate(j)])
    total = sum(n for n, _ in lens)
    rows = sum(t for _, t in lens)
    k = _rows(g, total, hkv, d, dt, 1.0, True)
    v = _rows(g, total, hkv, d, dt, 0.4)
    q = _rows(g, rows, hq, d, dt, 1.0)
    return dict(lens=[n for n, _ in lens], chunks=[t for _, t in lens], tables=tables, blocks=blocks,
                slots=slots, k=k, v=v, q=q)


# ------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][D] in fp32, its first `rot` dimensions rotated in pairs."""
    x, c, s = x.float(), cos[:, None], sin[:, None]
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2)
    else:
        x1, x2 = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    return torch.cat([y, rest], -1)


def _quantise(x, scale):
    """fp32 rows [N][H][D] -> codes -7..7 packed two to a byte, e4m3 scales."""
    g = (x / scale).unflatten(-1, (-1, 16))
    # in 64 bits: seven times a value between two scales is a common maximum
    s = (g.abs().amax(-1).double() / 7).float().clamp(max=448).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    c = torch.where(sf > 0, torch.round(g / sf), torch.zeros_like(g)).clamp(-7, 7).flatten(-2).to(torch.int32) + 8
    return (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8), s.view(torch.uint8)


def _dequantise(codes, scales, scale):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    s = scales.view(torch.float8_e4m3fn).float() * scale
    return (c.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


class _PlainCache:
    """A 4-bit cache held as packed codes and scales, a row per (slot, head)."""

    def __init__(self, slots, hkv, d):
        def zeros(n):
            return torch.zeros(slots, hkv, n, dtype=torch.uint8, device="cuda")
        self.parts = {x: (zeros(d // 2), zeros(d // 16)) for x in "kv"}

    def write(self, k, v, slots):
        for x, rows, scale in (("k", k, K_SCALE), ("v", v, V_SCALE)):
            codes, scales = _quantise(rows.float(), scale)
            self.parts[x][0][slots] = codes
            self.parts[x][1][slots] = scales

    def read(self, x, slots):
        return _dequantise(self.parts[x][0][slots], self.parts[x][1][slots], K_SCALE if x == "k" else V_SCALE)


def _run_append(s):
    c = s["case"]
    cs = s["table"][s["pos"].long()]
    cos, sin = cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:]
    q = _rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])
    if c["op"] == "rope":
        blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
        s["pool_k"][blk, :, off] = k.to(s["k"].dtype)
        s["pool_v"][blk, :, off] = s["v"]
        return {"q": q, "k": s["pool_k"], "v": s["pool_v"]}
    s["cache"].write(k, s["v"], s["slots"])
    out = s["read_dtype"]
    return {"q": q, "k": s["cache"].read("k", s["slots"]).to(out), "v": s["cache"].read("v", s["slots"]).to(out)}


def _run_decode(s):
    c = s["case"]
    b, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    width = s["tables"].shape[1] * BLOCK
    t = torch.arange(width, device="cuda")
    slots = s["tables"].clamp(min=0).long().repeat_interleave(BLOCK, 1) * BLOCK + t % BLOCK
    live = t[None] < s["seq_lens"][:, None]
    k = s["cache"].read("k", slots).transpose(1, 2)  # [B][Hkv][tokens][D]
    x = s["q"].float().view(b, hkv, hq // hkv, d) @ k.transpose(2, 3) * s["scale"]
    del k
    x = x.masked_fill(~live[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = s["cache"].read("v", slots).transpose(1, 2)
    o = p @ v / l
    return {"out": o.reshape(b, hq, d).to(DTYPES[c["out"]]), "lse": (m + torch.log(l)).reshape(b, hq)}


def _run_prefill(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    out, lse = [], []
    at = 0
    for b, (n, t) in enumerate(zip(s["lens"], s["chunks"])):
        j = torch.arange(n, device="cuda")
        slots = s["tables"][b][j // BLOCK].long() * BLOCK + j % BLOCK
        k, v = (s["cache"].read(x, slots).transpose(0, 1) for x in "kv")  # [Hkv][n][D]
        q = s["q"][at:at + t].float().view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3)
        x = q @ k[:, None].transpose(2, 3) * s["scale"]
        x = x.masked_fill(j[None] > torch.arange(n - t, n, device="cuda")[:, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        l = p.sum(-1, keepdim=True)
        out.append((p @ v[:, None] / l).permute(2, 0, 1, 3).reshape(t, hq, d))
        lse.append((m + torch.log(l)).permute(2, 0, 1, 3).reshape(t, hq))
        at += t
    return {"out": torch.cat(out).to(DTYPES[c["out"]]), "lse": torch.cat(lse)}


# ------------------------------------------------------ the library's calls
class _Pool:
    """A library pool, destroyed with its last reference."""

    def __init__(self, blocks, hkv, d, dtype):
        import paged_kv_cache_196_gb300 as pk
        self.pk = pk
        self.handle = pk.kv_pool_create(blocks, BLOCK, hkv, d, dtype)
        if dtype == pk.KV_I4:
            pk.kv_pool_set_i4_scales(self.handle, K_SCALE, V_SCALE)

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


def _own_append(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    row = s["qkv_stride"]
    pk.kv_append_rope(s["pool"].handle, s["k"], s["v"], s["dt"], s["slots"], c["tokens"], k_stride=row,
                      v_stride=row, positions=s["pos"], cos_sin=s["table"], max_position=c["max_pos"],
                      rot_dim=c["rot"], interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"],
                      num_q_heads=c["hq"], q_stride=row)
    if c["op"] == "rope":
        return {"q": s["q_out"], "k": s["pool_k"], "v": s["pool_v"]}
    pk.kv_read_tokens(s["pool"].handle, s["slots"], c["tokens"], s["k_out"], s["v_out"], s["read_dt"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_decode(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    pk.paged_decode_attention_i4(s["pool"].handle, s["q"], s["dt"], s["tables"], s["tables"].shape[1], s["seq_lens"],
                                 c["batch"], c["hq"], s["scale"], s["out"], s["out_dt"], s["lse"], s["splits"],
                                 s["ws"], s["ws_bytes"], seq_order=s["order"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prefill(s):
    import paged_kv_cache_196_gb300 as pk
    c = s["case"]
    pk.paged_prefill_attention_i4(s["pool"].handle, s["q"], s["dt"], s["cu_q"], s["q"].shape[0], max(s["chunks"]),
                                  s["tables"], s["tables"].shape[1], s["seq_lens"], c["batch"], c["hq"], s["scale"],
                                  s["out"], s["out_dt"], s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def prepare(case, seed):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
    if case["op"] in ("rope", "append"):
        s = _append_inputs(case, seed)
        s["case"], s["qkv_stride"] = case, (hq + 2 * hkv) * d
        # what a 4-bit pool stands for is exact in bf16
        s["read_dtype"] = torch.bfloat16
        shape = (s["blocks"], hkv, BLOCK, d)
        if own:
            import paged_kv_cache_196_gb300 as pk
            s["dt"], s["read_dt"] = _own_dtype(pk, case["dtype"]), pk.KV_BF16
            s["pool"] = _Pool(s["blocks"], hkv, d, s["dt"] if case["op"] == "rope" else pk.KV_I4)
            s["q_out"] = torch.empty(case["tokens"], hq, d, dtype=dt, device="cuda")
            s["k_out"], s["v_out"] = (torch.empty(case["tokens"], hkv, d, dtype=torch.bfloat16, device="cuda")
                                      for _ in "kv")
            if case["op"] == "rope":
                s["pool_k"], s["pool_v"] = s["pool"].views(shape, dt)
        elif case["op"] == "rope":
            s["pool_k"], s["pool_v"] = (torch.empty(shape, dtype=dt, device="cuda") for _ in "kv")
        else:
            s["cache"] = _PlainCache(s["blocks"] * BLOCK, hkv, d)
        if case["op"] == "rope":
            # what the pool held before
            s["pool_k"].fill_(0.5)
            s["pool_v"].fill_(-0.25)
        return s
    s = _cache_inputs(case, seed)
    k, v, slots = s.pop("k"), s.pop("v"), s.pop("slots")
    s["case"], s["scale"] = case, 1 / math.sqrt(d)
    s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(s["chunks"][:i]) for i in range(case["batch"] + 1)], dtype=torch.int32, device="cuda")
    if not own:
        s["cache"] = _PlainCache(s["blocks"] * BLOCK, hkv, d)
        for at in range(0, len(slots), 1 << 16):
            part = slice(at, at + (1 << 16))
            s["cache"].write(k[part], v[part], slots[part])
        return s
    import numpy as np

    import paged_kv_cache_196_gb300 as pk
    s["pool"] = _Pool(s["blocks"], hkv, d, pk.KV_I4)
    s["dt"], s["out_dt"] = _own_dtype(pk, case["dtype"]), _own_dtype(pk, case["out"])
    pk.kv_append_rope(s["pool"].handle, k, v, s["dt"], slots, len(slots))
    rows, width = s["q"].shape[0], s["tables"].shape[1]
    s["out"] = torch.empty(rows, hq, d, dtype=DTYPES[case["out"]], device="cuda")
    s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device="cuda")
    if case["op"] == "decode":
        lens = np.array(s["lens"], np.int32)
        order = np.zeros(len(lens), np.int32)
        pk.kv_decode_order(lens, order)
        s["order"] = torch.from_numpy(order).cuda()
        s["splits"] = pk.kv_decode_plan_i4(lens, hkv, width)
        s["ws_bytes"] = pk.kv_decode_workspace_size(case["batch"], hq, hkv, d, width, s["splits"])
    else:
        s["ws_bytes"] = pk.kv_prefill_i4_workspace_size(s["pool"].handle, case["batch"], hq, width, max(s["chunks"]))
    s["ws"] = torch.empty(max(s["ws_bytes"], 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()  # the rows appended here are dropped
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"decode": _own_decode, "prefill": _own_prefill}.get(op, _own_append)(state)
    return {"decode": _run_decode, "prefill": _run_prefill}.get(op, _run_append)(state)


# ------------------------------------------------------------ in 64 bits
def _e4m3_64(x):
    """x >= 0 in 64 bits to the nearest e4m3 (ties to even, at most 448)."""
    _, e = torch.frexp(x)  # x = m 2^e with m in [1/2, 1)
    step = (torch.clamp(e.long() - 4, min=-9) + 1023 << 52).view(torch.float64)  # 2^(e - 4)
    return torch.clamp(torch.round(x / step) * step, max=448.0)


def _stored_64(x, scale):
    """What a 4-bit pool keeps of x."""
    g = x.double().reshape(*x.shape[:-1], -1, 16) / scale
    m = g.abs().max(-1, keepdim=True).values
    s = _e4m3_64(m / torch.full_like(m, 7.0))  # a true division: by a number it is a product
    c = torch.clamp(torch.round(g / torch.where(s == 0, torch.ones_like(s), s)), -7, 7)
    return (c * s * scale).reshape(x.shape)


def _rotate_64(x, pos, table, case):
    y = x.double().clone()
    h = case["rot"] // 2
    c, s = table[pos.long(), :h].double()[:, None], table[pos.long(), h:].double()[:, None]
    if case["interleaved"]:
        first, second = slice(0, case["rot"], 2), slice(1, case["rot"], 2)
    else:
        first, second = slice(0, h), slice(h, 2 * h)
    a, b = x[..., first].double(), x[..., second].double()
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def exact(case, seed):
    if case["op"] in ("rope", "append"):
        s = _append_inputs(case, seed)
        q, k = (_rotate_64(s[x], s["pos"], s["table"], case) for x in "qk")
        v = s["v"].double()
        if case["op"] == "append":
            return {"q": q, "k": _stored_64(k, K_SCALE), "v": _stored_64(v, V_SCALE)}
        out = {"q": q}
        for name, rows, before in (("k", k, 0.5), ("v", v, -0.25)):
            pool = torch.full((s["blocks"] * BLOCK, case["hkv"], case["d"]), before, dtype=torch.float64, device="cuda")
            pool[s["slots"]] = rows
            out[name] = pool.view(s["blocks"], BLOCK, case["hkv"], case["d"]).transpose(1, 2).contiguous()
        return out
    s = _cache_inputs(case, seed)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    rows = s["q"].shape[0]
    out = torch.empty(rows, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(rows, hq, dtype=torch.float64, device="cuda")
    at = row = 0
    for n, t in zip(s["lens"], s["chunks"]):
        k, v = _stored_64(s["k"][at:at + n], K_SCALE), _stored_64(s["v"][at:at + n], V_SCALE)
        seen = torch.arange(n, device="cuda")[None] <= torch.arange(n - t, n, device="cuda")[:, None]
        for h in range(hq):
            x = s["q"][row:row + t, h].double() @ k[:, h // g].T / math.sqrt(d)
            x = torch.where(seen, x, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[row:row + t, h] = z
            out[row:row + t, h] = torch.exp(x - z[:, None]) @ v[:, h // g]
        at += n
        row += t
    return {"out": out, "lse": lse}
