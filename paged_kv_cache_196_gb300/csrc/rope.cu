// Append with the position rotation, and the read of cached tokens.
//
// Rotation.  With angle a = pos * f_j of pair j the pair (x1, x2) becomes
// (x1 cos a - x2 sin a, x2 cos a + x1 sin a); cos and sin come from the caller's
// fp32 table (angles of far positions need 64 bits, once per table instead of
// once per token).  The arithmetic is fp32 -- two products and one sum, each
// rounded, no contraction, so that every caller and every reference that follows
// the formula gets the same bits -- and the result is rounded once, to the
// output's type, or quantised unrounded (KV_I4).
//
// Work.  Memory-bound: each element is read and written once.  Eight
// consecutive dimensions (one 16-byte chunk of 16-bit elements) are a thread's
// share of a row; a row (one head of q, k or v) is D / 8 neighbouring lanes.  A
// warp takes 32 / (D / 8) rows of one token at a time, P times, all of q, of k or of v:
// the token's cos and sin are loaded once per thread, the rows' loads are all issued
// before the first use, and nothing branches within a warp.  The partner of a
// half-split pair sits a fixed number of lanes away and comes by shuffle, so that no
// element is loaded twice and q may be rotated in place.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "i4.cuh"
#include "internal.h"

namespace pkv {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;

struct RopeParams {
    const char *q, *k, *v;             // input rows, heads packed within a token
    long long q_stride, k_stride, v_stride, q_out_stride;  // bytes between tokens
    char *q_out;
    char *k_pool, *v_pool;
    const int64_t *slots;
    const int32_t *positions;
    const float *table;                // [max_position][rot / 2 cos, rot / 2 sin]
    int max_position;
    int rot;                           // rotated dimensions (0: none)
    int interleaved;
    int hq, hkv;                       // hq = 0: no q
    long long num_tokens, num_slots;
    float k_inv, v_inv;                // 1 / pool scales (KV_I4)
    int *err;
};

// Eight elements of type ET as fp32 and back.
template <int ET>
struct Octet {
    static constexpr int kWords = ET == KV_F32 ? 8 : 4;
    uint32_t w[kWords];
    KV_DEVICE void load(const char *src) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 u = p[i];
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    KV_DEVICE void store(char *dst) const {
        uint4 *p = reinterpret_cast<uint4 *>(dst);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) p[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    KV_DEVICE void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (ET == KV_F32) {
                x[2 * i] = __uint_as_float(w[2 * i]);
                x[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
            } else {
                const float2 f = ET == KV_BF16 ? bf16x2_to_float2(w[i]) : f16x2_to_float2(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        }
    }
    KV_DEVICE void set(const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (ET == KV_F32) {
                w[2 * i] = __float_as_uint(x[2 * i]);
                w[2 * i + 1] = __float_as_uint(x[2 * i + 1]);
            } else if constexpr (ET == KV_BF16) {
                w[i] = float2_to_bf16x2(x[2 * i], x[2 * i + 1]);
            } else {
                w[i] = float2_to_f16x2(x[2 * i], x[2 * i + 1]);
            }
        }
    }
};

// Quantises this lane's octet o of a K (V = false) or V row of token offset t
// (0..15) and stores it into the tile; the two lanes of a group share its scale.
// Every lane of the warp takes part in the shuffle, `live` lanes store.
template <int D, bool V>
KV_DEVICE void store_i4(char *tile, int t, int o, float (&x)[8], float inv, bool live) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= inv;  // a power of two
        m = i4::max_nan(m, fabsf(x[i]));
    }
    m = i4::max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t sb = i4::scale_byte(m);
    const uint32_t w = i4::codes8(x, i4::e4m3_to_float(sb));
    if (!live) return;
    if constexpr (V) {
        // quads 2 o and 2 o + 1
        uint16_t *c = reinterpret_cast<uint16_t *>(tile) + (t >> 1) * (D / 2) +
                      2 * ((2 * o) ^ i4::v_swizzle<D>(t >> 1)) + (t & 1);
        c[0] = (uint16_t)w;
        c[2] = (uint16_t)(w >> 16);
        if (!(o & 1)) tile[8 * D + (t >> 1) * (D / 8) + o + (t & 1)] = (char)sb;
    } else {
        reinterpret_cast<uint32_t *>(tile)[t * (D / 8) + o] = w;
        if (!(o & 1)) tile[8 * D + t * (D / 16) + (o >> 1)] = (char)sb;
    }
}

// y[i] = x[i] c[i] + z[i] s[i] for eight values: two products and their sum, each
// rounded.  The products run on pairs; the sums do not, since a packed product and a
// packed sum come back contracted to one rounding.
KV_DEVICE void rotate8(const float (&x)[8], const float (&z)[8], const float (&c)[8], const float (&s)[8],
                       float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 a = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(c[i], c[i + 1]));
        const float2 b = __fmul2_rn(make_float2(z[i], z[i + 1]), make_float2(s[i], s[i + 1]));
        y[i] = __fadd_rn(a.x, b.x);
        y[i + 1] = __fadd_rn(a.y, b.y);
    }
}

// IN: type of the rows; I4: 4-bit pool, else the pool holds type IN.  P: passes of a
// warp, 32 / (D / 8) rows each.  blockIdx.y: a warp's rows, first those of q, then of
// k, then of v; blockIdx.x: kRopeWarps tokens.  (Rows of one token in consecutive
// CTAs instead: 55.0 us for the chunk below.  k and v first: 49.6, but 56.1 into a 4-bit
// pool.)
//
// Bound by memory: a chunk of 8192 tokens (56 q, 8 kv heads of 128 dims, bf16) moves
// 306 MB in 50.1 us, 6100 GB/s (0.90 of a device copy); into a 4-bit pool 282 MB in
// 54.2 us, 5200 GB/s, the integer pipe busy for 54% of the time.  A step of 64 tokens (32 q, 8 kv heads): 2.5 and 2.9 us, a launch's
// length.
template <int D, int IN, bool I4, int P>
__global__ void __launch_bounds__(kRopeThreads) append_rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 8;         // lanes of one row
    constexpr int kAtOnce = 32 / kLanes;  // rows of one pass
    constexpr int kE = IN == KV_F32 ? 4 : 2;
    constexpr int kRowBytes = D * kE;
    const long long tok = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    if (tok >= p.num_tokens) return;
    const int lane = threadIdx.x & 31, o = lane % kLanes;
    // ---- whose rows
    const int uq = (p.hq + P * kAtOnce - 1) / (P * kAtOnce), ukv = (p.hkv + P * kAtOnce - 1) / (P * kAtOnce);
    const int unit = blockIdx.y;
    const bool is_q = unit < uq, is_v = unit >= uq + ukv;
    const int heads = is_q ? p.hq : p.hkv;
    const int h0 = (is_q ? unit : is_v ? unit - uq - ukv : unit - uq) * (P * kAtOnce) + lane / kLanes;
    const char *src = is_q ? p.q + tok * p.q_stride : is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride;
    src += (long long)h0 * kRowBytes + o * (8 * kE);
    Octet<IN> x[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
        if (h0 + u * kAtOnce < heads) {
            x[u].load(src + u * (kAtOnce * kRowBytes));
        } else {
#pragma unroll
            for (int i = 0; i < Octet<IN>::kWords; ++i) x[u].w[i] = 0;
        }
    }
    // ---- the token's place
    int pos = 0;
    if (p.rot > 0) {
        pos = __ldg(p.positions + tok);
        if (pos < 0 || pos >= p.max_position) {  // the token is left out
            if (unit == 0 && lane == 0) atomicOr(p.err, KV_DEVERR_POSITION);
            return;
        }
    }
    char *dst;
    int t = 0;  // the token's place in its block
    if (is_q) {
        dst = p.q_out + tok * p.q_out_stride + (long long)h0 * kRowBytes + o * (8 * kE);
    } else {
        const long long slot = __ldg(p.slots + tok);
        if (slot < 0 || slot >= p.num_slots) {
            if (slot >= 0 && unit == uq && lane == 0) atomicOr(p.err, KV_DEVERR_SLOT_RANGE);
            return;
        }
        t = (int)(slot & 15);
        const long long tile = (slot >> 4) * p.hkv + h0;
        dst = is_v ? p.v_pool : p.k_pool;
        if constexpr (I4)
            dst += tile * (18 * D);
        else
            dst += (tile * 16 + t) * kRowBytes + o * (8 * kE);
        if constexpr (I4) {
            if (is_v) {
#pragma unroll
                for (int u = 0; u < P; ++u) {
                    float y[8];
                    x[u].get(y);
                    store_i4<D, true>(dst + (long long)u * kAtOnce * (18 * D), t, o, y, p.v_inv, h0 + u * kAtOnce < heads);
                }
                return;
            }
        }
    }
    const long long step_dst = is_q ? (long long)kAtOnce * kRowBytes : (long long)kAtOnce * (I4 ? 18 * D : 16 * kRowBytes);
    // ---- cos and sin of this lane's pairs, the sign of the formula in sin; a lane
    // that rotates nothing takes 1 and 0
    float c[8], s[8];
    const bool rotates = !is_v && 8 * o < p.rot;
    const int half = p.rot / 2;
    const bool first = 8 * o < half;
    if (rotates) {
        const float *cs = p.table + (long long)pos * p.rot;
        if (p.interleaved) {  // pairs 4 o .. 4 o + 3
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(cs + 4 * o));
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(cs + half + 4 * o));
            c[0] = c[1] = c4.x, c[2] = c[3] = c4.y, c[4] = c[5] = c4.z, c[6] = c[7] = c4.w;
            s[0] = -s4.x, s[1] = s4.x, s[2] = -s4.y, s[3] = s4.y;
            s[4] = -s4.z, s[5] = s4.z, s[6] = -s4.w, s[7] = s4.w;
        } else {  // pairs j0 .. j0 + 7
            const int j0 = first ? 8 * o : 8 * o - half;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 c4 = __ldg(reinterpret_cast<const float4 *>(cs + j0 + i));
                const float4 s4 = __ldg(reinterpret_cast<const float4 *>(cs + half + j0 + i));
                c[i] = c4.x, c[i + 1] = c4.y, c[i + 2] = c4.z, c[i + 3] = c4.w;
                s[i] = first ? -s4.x : s4.x, s[i + 1] = first ? -s4.y : s4.y;
                s[i + 2] = first ? -s4.z : s4.z, s[i + 3] = first ? -s4.w : s4.w;
            }
        }
    }
    // the lane that holds the other halves of this lane's half-split pairs
    const int across = half / 8;
    const int partner = !rotates || p.interleaved ? lane : first ? lane + across : lane - across;
    const bool swaps = p.rot > 0 && !p.interleaved && !is_v;
#pragma unroll
    for (int u = 0; u < P; ++u) {
        const bool live = h0 + u * kAtOnce < heads;
        Octet<IN> other = x[u];
        if (swaps) {
#pragma unroll
            for (int i = 0; i < Octet<IN>::kWords; ++i) other.w[i] = __shfl_sync(0xffffffffu, x[u].w[i], partner);
        }
        float y[8];
        if (rotates) {
            float a[8], z[8];
            x[u].get(a);
            other.get(z);
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) z[i] = a[i + 1], z[i + 1] = a[i];
            }
            rotate8(a, z, c, s, y);
            if (!I4 || is_q) x[u].set(y);
        } else if (I4) {
            x[u].get(y);
        }
        if constexpr (I4) {
            if (!is_q) {  // a K row; the group's lanes exchange their maxima
                store_i4<D, false>(dst + u * step_dst, t, o, y, p.k_inv, live);
                continue;
            }
        }
        if (live) x[u].store(dst + u * step_dst);  // what is not rotated: bit by bit
    }
}

// Cached tokens as rows: token i's K and V rows [hkv][D] of type OUT from slot
// slots[i].  ET: the pool's type (KV_I4: codes).  A warp takes the rows of
// 32 / (D / 8) heads of a token at a time, an octet a lane: the inverse of the
// store's lanes, so that a row is written in one piece.  8192 tokens of 8 kv heads of 128
// dims from a 4-bit pool as bf16: 43 MB in 9.0 us, 4800 GB/s with the rows' lines still
// in L2; the conversions keep the integer pipe at 58%.
template <int D, int ET, int OUT>
__global__ void __launch_bounds__(kRopeThreads) read_tokens_kernel(const char *__restrict__ k_pool,
                                                                   const char *__restrict__ v_pool,
                                                                   const int64_t *__restrict__ slots,
                                                                   long long num_tokens, int hkv, long long num_slots,
                                                                   float k_scale, float v_scale,
                                                                   char *__restrict__ k_out,
                                                                   char *__restrict__ v_out, int *err) {
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
    constexpr int kE = OUT == KV_F32 ? 4 : 2;
    const long long tok = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    if (tok >= num_tokens) return;
    const int lane = threadIdx.x & 31, o = lane % kLanes;
    const long long slot = __ldg(slots + tok);
    if (slot < 0 || slot >= num_slots) {
        if (slot >= 0 && lane == 0) atomicOr(err, KV_DEVERR_SLOT_RANGE);
        return;
    }
    const int t = (int)(slot & 15);
#pragma unroll 4
    for (int h = lane / kLanes; h < hkv; h += kAtOnce) {
        const long long tile = (slot >> 4) * hkv + h;
        Octet<OUT> ko, vo;
        if constexpr (ET == KV_I4) {
            const char *kt = k_pool + tile * (18 * D), *vt = v_pool + tile * (18 * D);
            const uint32_t kw = __ldg(reinterpret_cast<const uint32_t *>(kt) + t * (D / 8) + o);
            const uint32_t kb = __ldg(reinterpret_cast<const uint8_t *>(kt) + 8 * D + t * (D / 16) + (o >> 1));
            // both tokens' words of quads 2 o and 2 o + 1
            const uint2 vq = __ldg(reinterpret_cast<const uint2 *>(
                reinterpret_cast<const uint32_t *>(vt) + (t >> 1) * (D / 4) + ((2 * o) ^ i4::v_swizzle<D>(t >> 1))));
            const uint32_t vw = __byte_perm(vq.x, vq.y, t & 1 ? 0x7632 : 0x5410);
            const uint32_t vb = __ldg(reinterpret_cast<const uint8_t *>(vt) + 8 * D + (t >> 1) * (D / 8) + (o & ~1) + (t & 1));
            const float ks = i4::e4m3_to_float(kb) * k_scale, vs = i4::e4m3_to_float(vb) * v_scale;
            float a[8], b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] = (float)((int)(kw >> (4 * j) & 15u) - 8) * ks;
                b[j] = (float)((int)(vw >> (4 * j) & 15u) - 8) * vs;
            }
            ko.set(a);
            vo.set(b);
        } else {
            const long long at = (tile * 16 + t) * (D * kE) + o * (8 * kE);
            ko.load(k_pool + at);
            vo.load(v_pool + at);
        }
        const long long at = (tok * hkv + h) * (long long)(D * kE) + o * (8 * kE);
        ko.store(k_out + at);
        vo.store(v_out + at);
    }
}

template <int D, int IN, bool I4>
static kv_status launch_append_rope(const RopeParams &p, cudaStream_t s) {
    constexpr int kAtOnce = 32 / (D / 8);
    // Passes per warp: one while that leaves SMs idle (a decode step), four when there
    // are warps enough, so that a token's cos and sin serve more rows.  With 32 q and 8
    // kv heads, one / four passes: 64 tokens 2.3 / 2.5 us (4-bit 2.7 / 3.5), 256 tokens
    // 3.3 / 3.1 (3.4 / 3.9), 512 tokens 4.6 / 3.7 (4.8 / 4.4), 4096 tokens 26.7 / 19.0
    // (28.5 / 20.9).  Two and eight passes cost the 8192-token chunk below 58.7 and 55.0
    // us.
    auto units = [&](int r) { return (p.hq + r - 1) / r + 2LL * ((p.hkv + r - 1) / r); };
    auto go = [&](auto fn, int r) {
        if (units(r) > 65535) return KV_ERR_UNSUPPORTED;
        const dim3 grid((unsigned)((p.num_tokens + kRopeWarps - 1) / kRopeWarps), (unsigned)units(r));
        fn<<<grid, kRopeThreads, 0, s>>>(p);
        return cuda_status(cudaGetLastError());
    };
    if (p.num_tokens * units(4 * kAtOnce) >= 16LL * sm_count())
        return go(append_rope_kernel<D, IN, I4, 4>, 4 * kAtOnce);
    return go(append_rope_kernel<D, IN, I4, 1>, kAtOnce);
}

template <int D, int ET, int OUT>
static void launch_read(kv_pool_t p, const int64_t *slots, long long n, void *k_out, void *v_out, cudaStream_t s) {
    read_tokens_kernel<D, ET, OUT><<<(unsigned)((n + kRopeWarps - 1) / kRopeWarps), kRopeThreads, 0, s>>>(
        (const char *)p->k, (const char *)p->v, slots, n, p->num_kv_heads, (long long)p->num_blocks * 16, p->k_scale,
        p->v_scale, (char *)k_out, (char *)v_out, p->err);
}

}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_append_rope(kv_pool_t p, const void *k_new, const void *v_new, kv_dtype in_dtype, int64_t k_stride,
                         int64_t v_stride, const int64_t *slot_mapping, const int32_t *positions,
                         const float *cos_sin, int max_position, int rot_dim, int interleaved, const void *q,
                         void *q_out, int64_t q_stride, int64_t q_out_stride, int num_q_heads, int num_tokens,
                         void *stream) {
    if (!p || num_tokens < 0 || rot_dim < 0 || k_stride < 0 || v_stride < 0 || q_stride < 0 || q_out_stride < 0 ||
        (interleaved != 0 && interleaved != 1))
        return KV_ERR_ARG;
    if (in_dtype != KV_F32 && in_dtype != KV_BF16 && in_dtype != KV_F16) return KV_ERR_UNSUPPORTED;
    if (p->dtype != KV_I4 && in_dtype != p->dtype) return KV_ERR_ARG;
    const int d = p->head_dim, e = dtype_bytes(in_dtype);
    if (rot_dim > d || rot_dim % 16) return KV_ERR_ARG;
    if (rot_dim > 0 && max_position <= 0) return KV_ERR_ARG;
    if (q && (rot_dim == 0 || !q_out || num_q_heads <= 0)) return KV_ERR_ARG;
    const int64_t kv_row = (int64_t)p->num_kv_heads * d, q_row = q ? (int64_t)num_q_heads * d : 0;
    if (k_stride == 0) k_stride = kv_row;
    if (v_stride == 0) v_stride = kv_row;
    if (q_stride == 0) q_stride = q_row;
    if (q_out_stride == 0) q_out_stride = q == q_out ? q_stride : q_row;
    if (k_stride < kv_row || v_stride < kv_row || q_stride < q_row || q_out_stride < q_row) return KV_ERR_ARG;
    if (q && q == q_out && q_stride != q_out_stride) return KV_ERR_ARG;
    // rows move in 16-byte chunks
    if ((k_stride * e) % 16 || (v_stride * e) % 16 || (q_stride * e) % 16 || (q_out_stride * e) % 16) return KV_ERR_ARG;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
                           reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q ? q_out : nullptr) |
                           reinterpret_cast<uintptr_t>(rot_dim > 0 ? cos_sin : nullptr);
    if (bits & 15) return KV_ERR_ARG;
    if (kv_status st = require_device(p->device)) return st;
    if (num_tokens == 0) return KV_OK;
    if (!k_new || !v_new || !slot_mapping || (rot_dim > 0 && (!positions || !cos_sin))) return KV_ERR_ARG;
    RopeParams r{};
    r.q = static_cast<const char *>(q);
    r.k = static_cast<const char *>(k_new);
    r.v = static_cast<const char *>(v_new);
    r.q_stride = q_stride * e;
    r.k_stride = k_stride * e;
    r.v_stride = v_stride * e;
    r.q_out_stride = q_out_stride * e;
    r.q_out = static_cast<char *>(q_out);
    r.k_pool = static_cast<char *>(p->k);
    r.v_pool = static_cast<char *>(p->v);
    r.slots = slot_mapping;
    r.positions = positions;
    r.table = cos_sin;
    r.max_position = max_position;
    r.rot = rot_dim;
    r.interleaved = interleaved;
    r.hq = q ? num_q_heads : 0;
    r.hkv = p->num_kv_heads;
    r.num_tokens = num_tokens;
    r.num_slots = (long long)p->num_blocks * p->block_size;
    r.k_inv = 1.f / p->k_scale;
    r.v_inv = 1.f / p->v_scale;
    r.err = p->err;
    const cudaStream_t s = as_stream(stream);
    auto by_type = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        const bool i4 = p->dtype == KV_I4;
        if (in_dtype == KV_F32)
            return i4 ? launch_append_rope<D, KV_F32, true>(r, s) : launch_append_rope<D, KV_F32, false>(r, s);
        if (in_dtype == KV_BF16)
            return i4 ? launch_append_rope<D, KV_BF16, true>(r, s) : launch_append_rope<D, KV_BF16, false>(r, s);
        return i4 ? launch_append_rope<D, KV_F16, true>(r, s) : launch_append_rope<D, KV_F16, false>(r, s);
    };
    const kv_status st =
        d == 128 ? by_type(std::integral_constant<int, 128>{}) : by_type(std::integral_constant<int, 64>{});
    // A decode launched to overlap the kernel before it reads q early; q is what was
    // just written.  Anything but a kernel between the two ends the overlap.
    if (st == KV_OK && q && p->launch_overlap) return cuda_status(cudaMemsetAsync(p->err + 1, 0, sizeof(int), s));
    return st;
}

kv_status kv_read_tokens(kv_pool_t p, const int64_t *slots, int num_tokens, void *k_out, void *v_out,
                         kv_dtype out_dtype, void *stream) {
    if (!p || num_tokens < 0) return KV_ERR_ARG;
    if (out_dtype != KV_F32 && out_dtype != KV_BF16 && out_dtype != KV_F16) return KV_ERR_UNSUPPORTED;
    if (p->dtype != KV_I4 && out_dtype != p->dtype) return KV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15) return KV_ERR_ARG;
    if (kv_status st = require_device(p->device)) return st;
    if (num_tokens == 0) return KV_OK;
    if (!slots || !k_out || !v_out) return KV_ERR_ARG;
    const cudaStream_t s = as_stream(stream);
    auto by_type = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (p->dtype == KV_I4) {
            if (out_dtype == KV_F32) launch_read<D, KV_I4, KV_F32>(p, slots, num_tokens, k_out, v_out, s);
            if (out_dtype == KV_BF16) launch_read<D, KV_I4, KV_BF16>(p, slots, num_tokens, k_out, v_out, s);
            if (out_dtype == KV_F16) launch_read<D, KV_I4, KV_F16>(p, slots, num_tokens, k_out, v_out, s);
        } else if (p->dtype == KV_F32) {
            launch_read<D, KV_F32, KV_F32>(p, slots, num_tokens, k_out, v_out, s);
        } else {  // rows of 16 bits are moved, whatever they mean
            launch_read<D, KV_BF16, KV_BF16>(p, slots, num_tokens, k_out, v_out, s);
        }
    };
    if (p->head_dim == 128)
        by_type(std::integral_constant<int, 128>{});
    else
        by_type(std::integral_constant<int, 64>{});
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
