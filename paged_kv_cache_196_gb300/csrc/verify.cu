// Verification of drafted tokens, and the move that leaves the accepted ones in the cache.
//
// Verification.  p is the target's distribution after a node, q the one that the node's
// children were drawn from.  A child with token x is accepted if u q(x) < p(x); after a
// rejection the next child, and in the end the draw of the next token, meet the residual
// max(p - q, 0) / sum.  Without the division: with W_0 = p, S_0 = 1,
//   W_{k+1} = max(W_k - S_k q, 0),  S_{k+1} = sum W_{k+1},  accept iff u q(x) S_k < W_k(x);
// nothing that went to zero returns, so W_k = max(p - (S_0 + .. + S_{k-1}) q, 0) at once,
// and the draw is the first index whose running sum of W_k passes u S_k.  Drafts that were
// chosen (q null) count as drawn from a q that is one at x: W loses its entry at x, and S that
// entry (from 1, what a row of probabilities sums to: the row itself is read for the draw alone).
//
// A draw from 10^5 tokens lies next to a border between two of them: sums that depend on
// their order would return another token now and then.  So weights are integers, p and q
// rounded to steps of 2^-E with E = 45, less for more than 2^17 tokens (42 for 2^20): no sum
// passes 2^62 whatever the rows hold, sums are exact in any order, and their roundings, at random,
// add up to about sqrt(vocab) 2^-47: 3e-12 for 128000 tokens.  A draw meets another token than the
// real numbers' where it lies between a border and its place here: over all borders of rows of 128000
// tokens (normal logits of deviation 6, three of them) that is a chance of 7e-7 to 3e-6, from a node's second
// rejection on, when the rounding of S_1 counts too, of 1e-6 to 5e-5.  (Products cut off instead of rounded
// 5e-5 to 5e-4; probabilities cut off would add up to 2^-30.)  Single comparisons (u q(x) against
// p(x)) are in fp64, where the product of two fp32 numbers is exact (the first test of a node looks
// in fp32 first); after a rejection, when S_k or
// S_0 + .. comes in, they are as good as fp64.
//
// A probability becomes an integer in two parts, 22 bits and E - 22: adding 2^23 to a number
// below 2^22 leaves its whole part in the mantissa, what that leaves is exact, and both parts
// sum up in 32 bits over a lane's 16 tokens: six full-rate operations where a conversion to 64
// bits takes the time of sixteen.
//
// A walk down a tree needs p(x) and q(x) of each draft, which are loaded at once for all
// nodes before it begins; only a rejection and the draw at the end read whole rows, so the
// rows of nodes that are not reached are never touched.  A sequence is worked on by a cluster
// of CTAs, each with a share of the vocabulary: a pass over a row leaves sums of chunks of
// 512 tokens in shared memory, CTAs add up their totals through distributed shared memory,
// and the draw looks into one chunk.  Every CTA walks the tree by itself, so that nothing but
// the totals is exchanged.
//
// What bounds it: chains read their last node's rows once, 64 of them over 128000 tokens (fp32, p and q)
// 65 MB and 9.8 us at the copy rate in 22 us: the start, the walk and the draw are
// latencies, and the batch is little more than one wave.  Trees read a row again for every
// rejection, one pass behind the other: 16 trees of 64 nodes 43.1 us (41.0 with products
// cut off).  With up to 15 of them, an SM to
// each CTA, a rejection costs 5 us at first and 8 to 9 from the second on; 16 share SMs, 14: 16 rejections at each of
// 16 roots 218 us.  (W_k from W_1 in k - 1 steps of 64 bits took 1050 us for them.)  The walk, 1 us, is one warp's: with all warps
// in it the fp64 unit takes several times as long.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "tree_plan.cuh"

namespace pkv {
namespace tree {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kChunk = 512;           // tokens
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxCluster = 8;
constexpr int kCtaChunks = kMaxVocab / kChunk;  // of a cluster of one

struct VerifyParams {
    const void *p, *q;  // rows of the vocabulary; q null: drafts were chosen
    int64_t p_stride, q_stride;
    int vocab, scale_exp;  // E
    const int32_t *cu_q;
    int total_q, max_q_len;
    const int32_t *parents, *tokens;
    const float *accept_u, *sample_u;
    int batch, max_path;
    int32_t *num_accepted, *path, *out_tokens;
    int *err;
};

struct VerifyShared {
    unsigned long long chunk[kCtaChunks];
    unsigned long long totals[2][kMaxCluster];  // of the cluster's CTAs, for passes in turn
    float p[kMaxNodes], q[kMaxNodes], u[kMaxNodes];  // of each node's token, in its parent's rows
    int32_t token[kMaxNodes];
    int16_t parent[kMaxNodes];                  // -1: none, or no draft
    int16_t gone[kMaxNodes];                    // rejected nodes whose tokens were chosen
    int16_t path[kMaxNodes];
    unsigned long long weight[kChunk + kChunk / 16];  // of the chunk that holds the draw, 16 and a gap
    int node, count, rejected, gone_count, end;  // where the walk stands; end: nothing is left to try
};

// A probability: not below 0 (nor NaN), not above 1.
KV_DEVICE float prob(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }

template <typename T>
KV_DEVICE float one(const void *row, int64_t i);
template <>
KV_DEVICE float one<float>(const void *row, int64_t i) {
    return __ldg(reinterpret_cast<const float *>(row) + i);
}
struct PB16 {};
struct PF16 {};
template <>
KV_DEVICE float one<PB16>(const void *row, int64_t i) {
    return bf16_to_float(__ldg(reinterpret_cast<const uint16_t *>(row) + i));
}
template <>
KV_DEVICE float one<PF16>(const void *row, int64_t i) {
    return f16x2_to_float2(__ldg(reinterpret_cast<const uint16_t *>(row) + i)).x;
}
template <typename T>
constexpr int kElem = 2;
template <>
constexpr int kElem<float> = 4;

// Which token of its chunk a lane's i-th is.
template <typename T>
KV_DEVICE int chunk_index(int i, bool wide) {
    const int lane = threadIdx.x & 31;
    constexpr int kVec = 16 / kElem<T>;
    return wide ? i / kVec * (32 * kVec) + lane * kVec + i % kVec : 32 * i + lane;
}

// A lane's 16 tokens of the chunk at `first`: in 16-byte loads where `wide`, else every 32nd.
template <typename T>
KV_DEVICE void load_chunk(const void *row, int first, int vocab, bool wide, float (&v)[16]) {
    const int lane = threadIdx.x & 31;
    if (wide) {
        if constexpr (kElem<T> == 4) {
            const float4 *src = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row) + first) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 x = __ldg(src + 32 * i);
                v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
            }
        } else {
            const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(row) + first) + lane;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 x = __ldg(src + 32 * i);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = std::is_same<T, PB16>::value ? bf16x2_to_float2(w[j]) : f16x2_to_float2(w[j]);
                    v[8 * i + 2 * j] = f.x, v[8 * i + 2 * j + 1] = f.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = first + 32 * i + lane;
            v[i] = at < vocab ? one<T>(row, at) : 0.f;
        }
    }
}

// Four tokens from `at` on: in one load where `wide`.
template <typename T>
KV_DEVICE float4 load_four(const void *row, int at, int vocab, bool wide) {
    if (wide) {
        if constexpr (kElem<T> == 4) {
            return __ldg(reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(row) + at));
        } else {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(row) + at));
            const float2 a = std::is_same<T, PB16>::value ? bf16x2_to_float2(x.x) : f16x2_to_float2(x.x);
            const float2 b = std::is_same<T, PB16>::value ? bf16x2_to_float2(x.y) : f16x2_to_float2(x.y);
            return make_float4(a.x, a.y, b.x, b.y);
        }
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at < vocab) v.x = one<T>(row, at);
    if (at + 1 < vocab) v.y = one<T>(row, at + 1);
    if (at + 2 < vocab) v.z = one<T>(row, at + 2);
    if (at + 3 < vocab) v.w = one<T>(row, at + 3);
    return v;
}

// A probability in steps of 2^-E: hi 2^(E - 22) + lo.
struct Parts {
    uint32_t hi, lo;
};
KV_DEVICE Parts parts(float x, float lo_scale) {  // x of prob(), lo_scale = 2^(E - 22)
    const float y = x * 0x1p22f;
    const float t = __fadd_rd(y, 0x1p23f);
    const float rest = y - (t - 0x1p23f);  // exact
    return Parts{__float_as_uint(t) & 0x7fffffu, __float_as_uint(__fadd_rn(rest * lo_scale, 0x1p23f)) - 0x4b000000u};
}
KV_DEVICE unsigned long long fixed(float x, int e) {
    const Parts a = parts(prob(x), __uint_as_float((uint32_t)(127 + e - 22) << 23));
    return (unsigned long long)a.hi * (1u << (e - 22)) + a.lo;  // (one multiply-add)
}

// floor(a b / 2^shift)
KV_DEVICE unsigned long long mul_shift(unsigned long long a, unsigned long long b, int shift) {
    const unsigned long long lo = a * b, hi = __umul64hi(a, b);
    if (shift >= 128) return 0;
    if (shift >= 64) return hi >> (shift - 64);
    return shift ? (lo >> shift) | (hi << (64 - shift)) : lo;
}

// S_1 + .. + S_{k-1}, as the factor of a product whose upper half is floor(2 (of it times q) / 2^E), to be
// rounded: shifted to the left as far as it goes (it is below 2^63), q the rest of the 65 - E places.  (Only a
// q of one may lose its bit there: nothing of p is left of it anyway.)
struct Taken {
    unsigned long long s;
    int q_shift, e;
    KV_DEVICE Taken(unsigned long long sum, int scale_exp) : e(scale_exp) {
        const int a = min(__clzll((long long)sum), 64 - e);
        s = sum << a;
        q_shift = 65 - e - a;
    }
    // W_k, k > 1
    KV_DEVICE unsigned long long weight(float p, float q) const {
        const unsigned long long a = fixed(p, e), b = fixed(q, e);
        const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);  // (q_shift < 32)
        const unsigned long long y = (unsigned long long)__funnelshift_l(lo, hi, q_shift) << 32 | lo << q_shift;
        const unsigned long long x = b + ((__umul64hi(s, y) + 1) >> 1);
        return a > x ? a - x : 0;
    }
};
// W_1 of a token, W_0 where k is 0.
KV_DEVICE unsigned long long first_residual(float p, float q, int k, int e) {
    const unsigned long long a = fixed(p, e), b = k ? fixed(q, e) : 0;
    return a > b ? a - b : 0;
}

KV_DEVICE unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// The cluster's barrier in two halves: arrived at when a CTA begins, waited for where it matters.
KV_DEVICE void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
KV_DEVICE void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// One pass over the node's row: sums of W_k by chunk, and of all of it over the cluster.
// `gone`: nodes whose tokens have lost their weight.  The whole cluster calls it.
template <typename T>
KV_DEVICE unsigned long long pass(const VerifyParams &a, VerifyShared &sm, const cg::cluster_group &cluster, long long row,
                                  int k, unsigned long long taken, int gone, int turn, bool first_pass) {
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = ((a.vocab + kChunk - 1) / kChunk + ctas - 1) / ctas;  // a CTA's share
    const char *p = static_cast<const char *>(a.p) + row * a.p_stride * kElem<T>;
    const char *q = static_cast<const char *>(a.q) + row * a.q_stride * kElem<T>;
    const bool p_wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0, q_wide = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
    const float lo_scale = __uint_as_float((uint32_t)(127 + a.scale_exp - 22) << 23);
    const int shift = a.scale_exp - 22;
    const Taken t(taken, a.scale_exp);
    for (int c = warp; c < chunks; c += kVerifyWarps) {
        const long long first = ((long long)rank * chunks + c) * kChunk;
        unsigned long long sum = 0;
        if (first < a.vocab) {
            const bool full = first + kChunk <= a.vocab;
            if (k <= 1) {
                float x[16], y[16];
                load_chunk<T>(p, (int)first, a.vocab, full && p_wide && (k == 0 || q_wide), x);
                if (k) load_chunk<T>(q, (int)first, a.vocab, full && p_wide && q_wide, y);
                // max(p - q, 0) part by part, where p > q (a part may be below q's; the sum is not)
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float px = prob(x[i]), qx = k ? prob(y[i]) : 0.f;
                    const Parts u = parts(px, lo_scale), v = parts(qx, lo_scale);
                    if (px > qx) hi += u.hi - v.hi, lo += u.lo - v.lo;
                }
                sum = ((unsigned long long)hi << shift) + (long long)(int32_t)lo;
            } else {
                // (a loop, since all 16 in line are more code than the rest of a pass)
                const bool wide = full && p_wide && q_wide;
                int at = (int)first + 4 * lane;
                float4 x = load_four<T>(p, at, a.vocab, wide), y = load_four<T>(q, at, a.vocab, wide);
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    const float4 x0 = x, y0 = y;
                    at += 128;
                    if (i < 3) x = load_four<T>(p, at, a.vocab, wide), y = load_four<T>(q, at, a.vocab, wide);
                    sum += t.weight(x0.x, y0.x) + t.weight(x0.y, y0.y) + t.weight(x0.z, y0.z) + t.weight(x0.w, y0.w);
                }
            }
        }
        sum = warp_sum(sum);
        if (lane == 0) sm.chunk[c] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < gone; ++i) {
                const int at = sm.token[sm.gone[i]] / kChunk - rank * chunks;
                if (at >= 0 && at < chunks) sm.chunk[at] -= fixed(sm.p[sm.gone[i]], a.scale_exp);
            }
        __syncwarp();
        unsigned long long sum = 0;
        for (int c = lane; c < chunks; c += 32) sum += sm.chunk[c];
        sum = warp_sum(sum);
        if (first_pass) cluster_wait();  // the other CTAs run: their shared memory may be written
        if (lane < ctas) *cluster.map_shared_rank(&sm.totals[turn][rank], lane) = sum;
    }
    if (first_pass && warp != 0) cluster_wait();
    cluster.sync();
    unsigned long long total = 0;
    for (int i = 0; i < ctas; ++i) total += sm.totals[turn][i];
    return total;
}

// The first token whose running sum of W_k passes `point`, counted from this CTA's share on
// (one warp; the share holds it).
template <typename T>
KV_DEVICE int find(const VerifyParams &a, VerifyShared &sm, int chunks, int rank, long long row, int k,
                   unsigned long long taken, int gone, unsigned long long point) {
    const int lane = threadIdx.x & 31;
    int c = 0;
    for (int base = 0; base < chunks; base += 32) {
        const unsigned long long mine = base + lane < chunks ? sm.chunk[base + lane] : 0;
        unsigned long long upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > point);
        if (past) {
            const int at = __ffs(past) - 1;
            point -= __shfl_sync(0xffffffffu, upto - mine, at);
            c = base + at;
            break;
        }
        point -= __shfl_sync(0xffffffffu, upto, 31);
    }
    const char *p = static_cast<const char *>(a.p) + row * a.p_stride * kElem<T>;
    const char *q = static_cast<const char *>(a.q) + row * a.q_stride * kElem<T>;
    const int first = (rank * chunks + c) * kChunk;
    const bool wide = first + kChunk <= a.vocab && (reinterpret_cast<uintptr_t>(p) & 15) == 0 &&
                      (k == 0 || (reinterpret_cast<uintptr_t>(q) & 15) == 0);
    float x[16], y[16];
    load_chunk<T>(p, first, a.vocab, wide, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = 0.f;
    if (k) load_chunk<T>(q, first, a.vocab, wide, y);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int at = chunk_index<T>(i, wide);
        sm.weight[at + at / 16] = first_residual(x[i], y[i], k, a.scale_exp);
    }
    if (k > 1) {
        const Taken t(taken, a.scale_exp);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = chunk_index<T>(i, wide);
            sm.weight[at + at / 16] = t.weight(x[i], y[i]);
        }
    }
    __syncwarp();
    for (int i = lane; i < gone; i += 32) {
        const int at = sm.token[sm.gone[i]] - first;
        if (at >= 0 && at < kChunk) sm.weight[at + at / 16] = 0;
    }
    __syncwarp();
    unsigned long long mine = 0;
    for (int i = 0; i < 16; ++i) mine += sm.weight[17 * lane + i];
    unsigned long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, upto > point);
    unsigned long long sum = upto - mine;
    int found = -1;
    for (int i = 0; i < 16 && found < 0; ++i) {
        sum += sm.weight[17 * lane + i];
        if (sum > point) found = first + 16 * lane + i;
    }
    return past ? __shfl_sync(0xffffffffu, found, __ffs(past) - 1) : -1;
}

template <typename E>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const VerifyParams a) {
    __shared__ VerifyShared sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / ctas;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool drawn = a.q != nullptr;
    cluster_arrive();

    const long long q0 = __ldg(a.cu_q + b);
    long long nodes = __ldg(a.cu_q + b + 1) - q0;
    if (nodes < 0 || nodes > a.max_q_len || q0 < 0 || q0 + nodes > a.total_q) {
        if (rank == 0 && tid == 0) atomicOr(a.err, KV_DEVERR_BLOCK_RANGE);
        nodes = 0;
    }
    const int T = (int)nodes;
    for (int i = tid; i < T; i += kVerifyThreads) {
        int up = i == 0 ? -1 : a.parents ? __ldg(a.parents + q0 + i) : i - 1;
        const int x = __ldg(a.tokens + q0 + i);
        if (i > 0) {
            if (up < -1 || up >= i || x >= a.vocab) {
                if (rank == 0) atomicOr(a.err, KV_DEVERR_TREE);
                up = -1;
            }
            if (x < 0) up = -1;
        }
        sm.parent[i] = (int16_t)up;
        sm.token[i] = x;
        if (up >= 0) {
            sm.p[i] = prob(one<E>(a.p, (q0 + up) * a.p_stride + x));
            sm.q[i] = drawn ? prob(one<E>(a.q, (q0 + up) * a.q_stride + x)) : 1.f;
            sm.u[i] = __ldg(a.accept_u + q0 + i);
        }
    }
    __syncthreads();

    const double unit = __longlong_as_double((long long)(1023 - a.scale_exp) << 52);
    const int chunks = ((a.vocab + kChunk - 1) / kChunk + ctas - 1) / ctas;
    unsigned long long total = 0;  // of the pass over W_k, once there was one: S_k
    unsigned long long taken = 0;  // S_1 + .. + S_{k-1}
    int node = 0, count = 0, turn = 0;
    int k = 0, gone = 0;           // rejections at the node
    int last = 0;                  // its child that was tried last
    double left = 1.0;             // S_k
    bool summed = false, first_pass = true;
    while (T > 0) {
        // Warp 0 of every CTA walks (64-bit floating point is slow: once is enough) until a rejection asks
        // for a pass over the row, or the walk ends.
        if (warp == 0) {
            int end = 0;
            while (true) {
                int child = T;
                if (count < a.max_path && left > 0.0)
                    for (int base = (last + 1) & ~31; base < T && child == T; base += 32) {
                        const int i = base + lane;
                        const uint32_t is = __ballot_sync(0xffffffffu, i > last && i < T && sm.parent[i] == node);
                        if (is) child = base + __ffs(is) - 1;
                    }
                if (child == T) {
                    end = 1;
                    break;
                }
                last = child;
                bool takes;
                double w = 0.0;
                if (k == 0 && gone == 0) {
                    // u q against p: a product rounded to fp32 that differs from p lies on the same side of it;
                    // one that does not is taken in 64 bits (what it lost may be below fp32's smallest number)
                    const float prod = sm.u[child] * sm.q[child];
                    takes = prod < sm.p[child] || (prod == sm.p[child] && (double)sm.u[child] * sm.q[child] < sm.p[child]);
                } else {
                    w = sm.p[child];
                    if (drawn) {
                        w = fmax(w - (1.0 + (double)taken * unit) * sm.q[child], 0.0);
                    } else {
                        for (int i = 0; i < gone; ++i)
                            if (sm.token[sm.gone[i]] == sm.token[child]) w = 0.0;
                    }
                    takes = (double)sm.u[child] * sm.q[child] * left < w;
                }
                if (takes) {
                    if (lane == 0) sm.path[count] = (int16_t)child;
                    ++count;
                    node = last = child;
                    k = gone = 0;
                    left = 1.0;
                    summed = false;
                } else if (drawn) {
                    ++k;
                    break;
                } else if (gone == 0 ? sm.p[child] > 0.f : w > 0.0) {
                    left -= gone == 0 ? (double)sm.p[child] : w;
                    __syncwarp();
                    if (lane == 0) sm.gone[gone] = (int16_t)child;
                    ++gone;
                    __syncwarp();
                }
            }
            if (lane == 0) sm.node = node, sm.count = count, sm.rejected = k, sm.gone_count = gone, sm.end = end;
        }
        __syncthreads();
        if (sm.node != node) summed = false;
        node = sm.node, count = sm.count, k = sm.rejected, gone = sm.gone_count;
        if (sm.end) break;
        // (at the node's k-th rejection the last pass was over W_{k-1}; 2^63 is never reached by rows that sum to one)
        taken = k < 2 ? 0 : min((k == 2 ? 0 : taken) + total, ~0ull >> 1);
        total = pass<E>(a, sm, cluster, q0 + node, k, taken, 0, turn, first_pass);
        turn ^= 1;
        summed = true;
        first_pass = false;
        if (warp == 0) left = (double)total * unit;
    }
    int token = -1;
    if (T > 0) {
        if (!summed) {
            total = pass<E>(a, sm, cluster, q0 + node, 0, 0, gone, turn, first_pass);
            turn ^= 1;
            first_pass = false;
        }
        if (total == 0 && (k > 0 || gone > 0)) {  // nothing is left: p itself
            k = gone = 0;
            total = pass<E>(a, sm, cluster, q0 + node, 0, 0, 0, turn, first_pass);
            turn ^= 1;
        }
        // floor(u total): u is a whole number of 2^-shift
        const float u = __ldg(a.sample_u + b);
        const uint32_t bits = __float_as_uint(u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f);
        const int e = max(1, (int)(bits >> 23));
        const unsigned long long m = (bits & 0x7fffffu) | (bits >> 23 ? 0x800000u : 0u);
        const unsigned long long point = mul_shift(total, m, 150 - e);
        unsigned long long before = 0;
        for (int i = 0; i < rank; ++i) before += sm.totals[turn ^ 1][i];
        const unsigned long long mine = sm.totals[turn ^ 1][rank];
        if (warp == 0 && point >= before && point - before < mine) {
            token = find<E>(a, sm, chunks, rank, q0 + node, k, taken, gone, point - before);
            if (lane == 0) a.out_tokens[(long long)b * (a.max_path + 1) + count] = token;
        }
    }
    if (first_pass) cluster_wait();  // (no pass: no nodes)
    if (rank == 0) {
        __syncthreads();
        if (tid == 0) a.num_accepted[b] = count;
        for (int i = tid; i <= a.max_path; i += kVerifyThreads) {
            const int at = i < count ? sm.path[i] : -1;
            if (i < a.max_path) a.path[(long long)b * a.max_path + i] = at;
            if (i != count || total == 0) a.out_tokens[(long long)b * (a.max_path + 1) + i] = at < 0 ? -1 : sm.token[at];
        }
    }
}

// ---------------------------------------------------------------- keeping a path
// The rows of path[i] move to place i + 1 behind the root.  path rises, so path[i] >= i + 1,
// and a place that is written is no later row's source: a thread that takes its 16 bytes of
// every row in order needs no second buffer.  A CTA works on one sequence of one pool; the
// pools of all layers go in one launch.  64 sequences of 24 layers, 0 to 6 accepted nodes each, 129 of whose rows of
// 2 x 8 heads x 128 bf16 values move in every layer (25 MB read and written): 6.5 us; 3.8 at the copy
// rate.  Two small pools 2.9 us, a launch.
constexpr int kKeepThreads = 256, kKeepPools = 128, kKeepAhead = 8;

struct KeepParams {
    uint4 *k[kKeepPools], *v[kKeepPools];
    int *err[kKeepPools];
    const int32_t *cu_q, *path, *num_accepted, *tables, *seq_lens;
    int32_t *new_lens;  // null in all launches of a call but the first
    int max_q_len, max_path, max_blocks, num_blocks, batch;
    int hkv, row_chunks;  // 16-byte parts of a row
};

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const __grid_constant__ KeepParams a) {
    __shared__ long long src[kMaxNodes], dst[kMaxNodes];  // rows of kv head 0; -1: not moved
    __shared__ int bad;
    const int layer = blockIdx.x / a.batch, b = blockIdx.x - layer * a.batch;
    const int tid = threadIdx.x;
    const long long t = (long long)__ldg(a.cu_q + b + 1) - __ldg(a.cu_q + b);
    const long long len = __ldg(a.seq_lens + b);
    const int count = __ldg(a.num_accepted + b);
    const bool writes_len = a.new_lens && layer == 0 && tid == 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    if (t == 0) {
        if (writes_len) a.new_lens[b] = (int32_t)len;
        return;
    }
    int wrong = 0;
    if (t < 0 || t > a.max_q_len || len < t || len > (long long)a.max_blocks * 16) {
        wrong = KV_DEVERR_BLOCK_RANGE;
    } else if (count < 0 || count > a.max_path || count >= t) {
        wrong = KV_DEVERR_TREE;
    } else {
        for (int i = tid; i < count; i += kKeepThreads) {
            const int at = __ldg(a.path + (long long)b * a.max_path + i);
            const int below = i ? __ldg(a.path + (long long)b * a.max_path + i - 1) : 0;
            if (at <= below || at >= t) bad = KV_DEVERR_TREE;
            long long from = -1, to = -1;
            if (at != i + 1 && at >= 0 && at < t) {
                const int32_t *table = a.tables + (long long)b * a.max_blocks;
                const long long s = len - t + at, d = len - t + i + 1;
                const int sb = __ldg(table + s / 16), db = __ldg(table + d / 16);
                if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                    atomicOr(a.err[layer], KV_DEVERR_BLOCK_RANGE);
                } else {
                    from = (long long)sb * a.hkv * 16 + s % 16;
                    to = (long long)db * a.hkv * 16 + d % 16;
                }
            }
            src[i] = from;
            dst[i] = to;
        }
    }
    __syncthreads();
    if (!wrong) wrong = bad;
    if (wrong) {
        if (tid == 0) atomicOr(a.err[layer], wrong);
        if (writes_len) a.new_lens[b] = (int32_t)len;
        return;
    }
    if (writes_len) a.new_lens[b] = (int32_t)(len - t + 1 + count);
    const int per_array = a.hkv * a.row_chunks;
    for (int col = tid; col < 2 * per_array; col += kKeepThreads) {
        uint4 *pool = col < per_array ? a.k[layer] : a.v[layer];
        const int at = col < per_array ? col : col - per_array;
        const int h = at / a.row_chunks, c = at - h * a.row_chunks;
        for (int i0 = 0; i0 < count; i0 += kKeepAhead) {
            uint4 x[kKeepAhead];
#pragma unroll
            for (int j = 0; j < kKeepAhead; ++j)
                if (i0 + j < count && src[i0 + j] >= 0) x[j] = pool[(src[i0 + j] + h * 16) * a.row_chunks + c];
#pragma unroll
            for (int j = 0; j < kKeepAhead; ++j)
                if (i0 + j < count && src[i0 + j] >= 0) pool[(dst[i0 + j] + h * 16) * a.row_chunks + c] = x[j];
        }
    }
}

namespace {

// CTAs of a sequence's cluster: as many as leave a chunk for each of its warps while the batch
// stays within a third more than one wave of two CTAs per SM.  Trees, which pass over rows again
// and again, gain by large clusters, chains by one wave.  In us with clusters of 1, 2, 4 and 8 (* the rule's):
//   16 trees over 128000 tokens   209, 115, 67.6, 43.2*    64 chains over 128000   38.0, 24.5, 22.2*, 27.6
//   100 trees over 50000          110, 82.0, 61.0*, 60.9   100 chains over 50000   21.4, 19.9, 23.8*, 29.8
//   200 trees over 32000          109, 63.8*, 68.7, 91.8   200 chains over 32000   21.9, 26.3*, 31.3, 49.9
//   150 trees over 32000          82.0, 54.8*, 55.7, 66.7  150 chains over 32000   16.2, 15.9*, 24.3, 38.2
int cluster_size(int vocab, int batch) {
    const int chunks = (vocab + kChunk - 1) / kChunk;
    int n = 1;
    while (n < kMaxCluster && n * kVerifyWarps < chunks && 2ll * n * batch * 3 <= 8ll * sm_count()) n *= 2;
    return n;
}

template <typename E>
kv_status launch_verify(const VerifyParams &a, cudaStream_t stream) {
    const int n = cluster_size(a.vocab, a.batch);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.batch * (unsigned)n);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, verify_kernel<E>, a));
}

}  // namespace
}  // namespace tree
}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_verify_tree(kv_pool_t p, const void *target_probs, int64_t target_stride, const void *draft_probs,
                         int64_t draft_stride, kv_dtype probs_dtype, int vocab, const int32_t *cu_q, int total_q,
                         int max_q_len, const int32_t *parents, const int32_t *tokens, const float *accept_uniform,
                         const float *sample_uniform, int batch, int max_path, int32_t *num_accepted, int32_t *path,
                         int32_t *out_tokens, void *stream) {
    if (!p || batch < 0 || total_q < 0 || max_q_len < 0 || max_path < 0 || vocab <= 0 || target_stride < 0 || draft_stride < 0)
        return KV_ERR_ARG;
    if (kv_status st = require_device(p->device)) return st;
    if ((probs_dtype != KV_F32 && probs_dtype != KV_BF16 && probs_dtype != KV_F16) || vocab > tree::kMaxVocab ||
        max_q_len > tree::kMaxNodes || max_path >= tree::kMaxNodes || batch > (1 << 27))
        return KV_ERR_UNSUPPORTED;
    if ((target_stride && target_stride < vocab) || (draft_stride && draft_stride < vocab)) return KV_ERR_ARG;
    if (batch == 0) return KV_OK;
    if (!cu_q || !num_accepted || !out_tokens || (max_path && !path)) return KV_ERR_ARG;
    if (total_q && (!target_probs || !tokens || !accept_uniform || !sample_uniform)) return KV_ERR_ARG;
    const uintptr_t align = dtype_bytes(probs_dtype) - 1;
    if ((reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs)) & align) return KV_ERR_ARG;
    tree::VerifyParams a{};
    a.p = target_probs;
    a.q = draft_probs;
    a.p_stride = target_stride ? target_stride : vocab;
    a.q_stride = draft_stride ? draft_stride : vocab;
    a.vocab = vocab;
    a.scale_exp = 45;
    while ((1ll << (62 - a.scale_exp)) < vocab) --a.scale_exp;
    a.cu_q = cu_q;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.parents = parents;
    a.tokens = tokens;
    a.accept_u = accept_uniform;
    a.sample_u = sample_uniform;
    a.batch = batch;
    a.max_path = max_path;
    a.num_accepted = num_accepted;
    a.path = path;
    a.out_tokens = out_tokens;
    a.err = p->err;
    const cudaStream_t s = as_stream(stream);
    if (probs_dtype == KV_F32) return tree::launch_verify<float>(a, s);
    return probs_dtype == KV_BF16 ? tree::launch_verify<tree::PB16>(a, s) : tree::launch_verify<tree::PF16>(a, s);
}

kv_status kv_keep_path(const kv_pool_t *pools, int num_pools, const int32_t *cu_q, int max_q_len, const int32_t *path,
                       int max_path, const int32_t *num_accepted, const int32_t *block_tables, int max_blocks,
                       const int32_t *seq_lens, int batch, int32_t *new_seq_lens, void *stream) {
    if (!pools || num_pools <= 0 || max_q_len < 0 || max_path < 0 || max_blocks < 0 || batch < 0) return KV_ERR_ARG;
    for (int i = 0; i < num_pools; ++i) {
        const kv_pool_t p = pools[i], first = pools[0];
        if (!p || p->num_blocks != first->num_blocks || p->num_kv_heads != first->num_kv_heads ||
            p->head_dim != first->head_dim || p->dtype != first->dtype || p->device != first->device)
            return KV_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (pools[j] == p) return KV_ERR_ARG;  // its rows would be moved twice
    }
    const kv_pool_t p = pools[0];
    if (kv_status st = require_device(p->device)) return st;
    if (p->dtype == KV_I4 || max_q_len > tree::kMaxNodes || max_path >= tree::kMaxNodes || max_blocks > (1 << 27) - 1 ||
        batch > INT32_MAX / tree::kKeepPools)
        return KV_ERR_UNSUPPORTED;
    if (batch == 0) return KV_OK;
    if (!cu_q || !num_accepted || !block_tables || !seq_lens || !new_seq_lens || (max_path && !path)) return KV_ERR_ARG;
    // other CTAs still read their inputs when one writes the new lengths
    auto overlaps = [&](const int32_t *x, size_t n) { return new_seq_lens < x + n && x < new_seq_lens + batch; };
    const size_t rows = (size_t)batch;
    if (overlaps(seq_lens, rows) || overlaps(num_accepted, rows) || overlaps(cu_q, rows + 1) ||
        (max_path && overlaps(path, rows * max_path)) || overlaps(block_tables, rows * max_blocks))
        return KV_ERR_ARG;
    tree::KeepParams a{};
    a.cu_q = cu_q;
    a.path = path;
    a.num_accepted = num_accepted;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.max_q_len = max_q_len;
    a.max_path = max_path;
    a.max_blocks = max_blocks;
    a.num_blocks = p->num_blocks;
    a.batch = batch;
    a.hkv = p->num_kv_heads;
    a.row_chunks = p->head_dim * dtype_bytes(p->dtype) / 16;
    for (int at = 0; at < num_pools; at += tree::kKeepPools) {
        const int n = std::min(num_pools - at, tree::kKeepPools);
        for (int i = 0; i < n; ++i) {
            a.k[i] = static_cast<uint4 *>(pools[at + i]->k);
            a.v[i] = static_cast<uint4 *>(pools[at + i]->v);
            a.err[i] = pools[at + i]->err;
        }
        a.new_lens = at == 0 ? new_seq_lens : nullptr;
        tree::keep_kernel<<<(unsigned)n * (unsigned)batch, tree::kKeepThreads, 0, as_stream(stream)>>>(a);
        if (kv_status st = cuda_status(cudaGetLastError())) return st;
    }
    // A decode launched to overlap the kernel before it reads its lengths early, and the new
    // lengths were just written.  Anything but a kernel between the two ends the overlap.
    for (int i = 0; i < num_pools; ++i)
        if (pools[i]->launch_overlap) return cuda_status(cudaMemsetAsync(p->err + 1, 0, sizeof(int), as_stream(stream)));
    return KV_OK;
}

}  // extern "C"
