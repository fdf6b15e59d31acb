// Attention of a tree of drafted tokens over a paged cache.
//
// Maths.  Sequence b holds L tokens, the last T of them the nodes of a tree, node i
// below parent[i] < i.  With S_i the L - T tokens before the tree, node i and the nodes
// above it:  o_i = sum_{j in S_i} exp(scale q_i.k_j) v_j / sum_{j in S_i} exp(scale q_i.k_j),
// in one pass over the keys with a running reference and sum per row.  A row is a
// (node, query head); the rows of a kv head and of as many nodes as fit are one matrix
// product with each tile of its keys, so a key is read once for all of them.
//
// The keys before the tree need no mask.  Those of the tree get one bit per (node, key),
// from a walk up the parents: S_i's bits are the row's mask of the last tiles.
//
// The work is spread over one wave of CTAs by tree_plan.cuh; a second kernel adds up the
// pairs that were cut: with m_s, l_s, O_s a piece's reference, sum and output,
//   o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "tree.h"
#include "tree_plan.cuh"

namespace pkv {
namespace tree {

// ---------------------------------------------------------------- fp32 arithmetic
// 32 rows of a pair against 32 keys at a time, the next 32 copied meanwhile, products by fp32
// multiply-adds: thread
// (ty, tx) holds rows 2 ty, 2 ty + 1, scores keys tx + 8 j and sums dimensions
// 4 tx + 32 i.  A warp owns eight rows, so their statistics and weights need no barrier.
// Bound by latency: two CTAs an SM of four warps each wait for shared memory and for their
// own sums.  Five ragged trees of 3 to 33 nodes over an fp32 pool (12 heads over 4, head_dim 64, to 1531
// tokens): 23.4 us where K and V take 1.3 to read; 55 for the first version, 37.7 with runs of three units
// at least.
constexpr int kSimpleRows = 32, kSimpleKeys = 32, kSimpleThreads = 128;

template <int D>
struct SimpleShared {
    float q[kSimpleRows][D + 4], k[2][kSimpleKeys][D + 4], v[2][kSimpleKeys][D + 4];
    float p[kSimpleRows][kSimpleKeys + 1];
    uint32_t anc[kSimpleRows][kMaxNodes / 32];
    PlaceScratch<kSimpleThreads> scratch;
};

// 16 bytes into shared memory, zeros if they are not there.
KV_DEVICE void copy16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kSimpleThreads) tree_simple_kernel(const TreeParams p) {
    extern __shared__ __align__(16) char raw[];
    auto &sm = *reinterpret_cast<SimpleShared<D> *>(raw);
    const int tid = threadIdx.x, ty = tid / 8, tx = tid % 8;
    const Place at = place(p.plan, blockIdx.x, sm.scratch, blockIdx.x == 0 ? p.err : nullptr);
    if (tid == 0 && p.cuts) p.cuts[blockIdx.x] = cut_of(p.plan, at, blockIdx.x, p.g);
    Pieces pieces;
    pieces.start(p.plan, at, blockIdx.x);
    Piece pc;
    while (pieces.next(p.plan, pc)) {
        const int node0 = pc.grp * p.plan.group_nodes;
        const int rows = min(p.plan.group_nodes, pc.seq.nodes - node0) * p.g;
        const int before = pc.seq.len - pc.seq.nodes;  // tokens before the tree
        const int32_t *table = p.tables + (size_t)pc.b * p.plan.max_blocks;
        __syncthreads();  // the piece before is done with what follows
        for (int i = tid; i < kSimpleRows * D / 4; i += kSimpleThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + ((size_t)(pc.seq.q0 + node0 + r / p.g) * p.hq + pc.h * p.g + r % p.g) * D + d));
            *reinterpret_cast<float4 *>(&sm.q[r][d]) = x;
        }
        if (tid < kSimpleRows) {
            for (int w = 0; w < kMaxNodes / 32; ++w) sm.anc[tid][w] = 0;
            if (tid < rows)
                walk_up(p.parents ? p.parents + pc.seq.q0 : nullptr, node0 + tid / p.g, p.err,
                        [&](int i) { sm.anc[tid][i >> 5] |= 1u << (i & 31); });
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float4 o[2][D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[0][i] = o[1][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int key1 = min(pc.t1 * kTile, pc.seq.len);
        // Keys key0 .. key0 + 31 (two blocks) into one of two buffers, zeros where there are none;
        // the bits of those that are there.
        auto fetch = [&](int key0, int buf) {
            int id[2];
            uint32_t there = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                id[i] = key0 + 16 * i < key1 ? __ldg(table + key0 / 16 + i) : -1;
                if (key0 + 16 * i >= key1) continue;
                if (id[i] < 0 || id[i] >= p.num_blocks) {
                    id[i] = -1;
                    if (tid == 0) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
                } else {
                    there |= (0xffffu >> max(0, key0 + 16 * i + 16 - key1)) << (16 * i);
                }
            }
#pragma unroll
            for (int j = 0; j < kSimpleKeys * D / 4 / kSimpleThreads; ++j) {
                const int i = tid + j * kSimpleThreads, r = i / (D / 4), d = i % (D / 4) * 4;
                const bool here = there >> r & 1;
                const size_t at0 = (((size_t)max(id[r >> 4], 0) * p.plan.hkv + pc.h) * 16 + r % 16) * D + d;
                copy16(&sm.k[buf][r][d], static_cast<const float *>(p.k) + at0, here);
                copy16(&sm.v[buf][r][d], static_cast<const float *>(p.v) + at0, here);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            return there;
        };
        uint32_t there_next = fetch(pc.t0 * kTile, 0);
        int buf = 0;
        for (int key0 = pc.t0 * kTile; key0 < key1; key0 += kSimpleKeys, buf ^= 1) {
            const uint32_t there = there_next;
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();  // this tile is there, and every thread is done with the one before
            if (key0 + kSimpleKeys < key1) there_next = fetch(key0 + kSimpleKeys, buf ^ 1);
            float s[2][4] = {};
            uint32_t seen[2];  // keys of the tile that each row attends
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&sm.q[2 * ty][d]);
                const float4 c = *reinterpret_cast<const float4 *>(&sm.q[2 * ty + 1][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 b = *reinterpret_cast<const float4 *>(&sm.k[buf][tx + 8 * j][d]);
                    s[0][j] += a.x * b.x, s[0][j] += a.y * b.y, s[0][j] += a.z * b.z, s[0][j] += a.w * b.w;
                    s[1][j] += c.x * b.x, s[1][j] += c.y * b.y, s[1][j] += c.z * b.z, s[1][j] += c.w * b.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 2 * ty + i;
                const uint32_t bits = seen[i] = key_bits(sm.anc[row], key0 - before) & there;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = bits >> (tx + 8 * j) & 1 ? s[i][j] : -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float up = fmaxf(m[i], mx * p.scale_log2);  // scale > 0
                const float ref = up == -INFINITY ? 0.f : up;
                const float alpha = ex2(m[i] - ref);
                m[i] = up;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = ex2(fmaf(s[i][j], p.scale_log2, -ref));  // one rounding, of the distance
                    sum += e;
                    sm.p[row][tx + 8 * j] = e;
                }
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                l[i] = l[i] * alpha + sum;
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    o[i][k].x *= alpha, o[i][k].y *= alpha, o[i][k].z *= alpha, o[i][k].w *= alpha;
            }
            __syncwarp();
            // What lies in a masked key reaches no row; what lies in an attended one does, though its weight may
            // be zero: a NaN or an infinity there is to show.
#pragma unroll 4
            for (int j = 0; j < kSimpleKeys; ++j) {
                const float e0 = sm.p[2 * ty][j], e1 = sm.p[2 * ty + 1][j];
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sm.v[buf][j][4 * tx + 32 * k]);
                    if (seen[0] >> j & 1)
                        o[0][k].x += e0 * v.x, o[0][k].y += e0 * v.y, o[0][k].z += e0 * v.z, o[0][k].w += e0 * v.w;
                    if (seen[1] >> j & 1)
                        o[1][k].x += e1 * v.x, o[1][k].y += e1 * v.y, o[1][k].z += e1 * v.z, o[1][k].w += e1 * v.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 2 * ty + i;
            if (row >= rows) continue;
            if (pc.slot >= 0) {
                float *part = p.partial + (size_t)pc.slot * kSimpleRows * (D + 2);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    reinterpret_cast<float4 *>(part)[(tx + 8 * k) * kSimpleRows + row] = o[i][k];
                if (tx == 0) reinterpret_cast<float2 *>(part + kSimpleRows * D)[row] = make_float2(m[i], l[i]);
                continue;
            }
            const size_t orow = (size_t)(pc.seq.q0 + node0 + row / p.g) * p.hq + pc.h * p.g + row % p.g;
            const bool seen = l[i] != 0.f;  // a row with a NaN score stays NaN
            const float inv = seen ? 1.f / l[i] : 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
                store_out4(p.out, orow * D + 4 * tx + 32 * k,
                           make_float4(o[i][k].x * inv, o[i][k].y * inv, o[i][k].z * inv, o[i][k].w * inv), p.out_type);
            if (p.lse && tx == 0)
                p.lse[orow] = seen ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
        }
    }
}

// ---------------------------------------------------------------- cut pairs
// CTA x looks at the end of run x: if it lies among the tiles of a pair, the pair is cut,
// and this CTA (with those of other y) takes one share of its rows, one share per cut.  A
// warp takes 8 rows of 16 dimensions, so that it reads lines and writes sectors whole.
// Latency again: 3 to 6 us for slots of 128 rows, 12 for 256 rows (up to 40 MB of them); all pieces
// of a pair are read at once (three, and most pairs have two), before any is used.  A launch that
// overlaps the attention's end gains nothing: its CTAs find no room beside one that takes a
// whole SM.
constexpr int kMergeThreads = 256, kMergeAhead = 3;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) tree_merge_kernel(const TreeParams p, int slot_rows) {
    const Cut cut = p.cuts[blockIdx.x + 1];
    if (cut.rows == 0) return;
    const int r0 = cut.r0, r1 = cut.r1, slot0 = cut.slot0, rows = cut.rows;
    const int shares = (r1 - r0) * (int)gridDim.y, share = (cut.r - r0 - 1) * (int)gridDim.y + (int)blockIdx.y;
    const int row0 = (int)((long long)rows * share / shares), row1 = (int)((long long)rows * (share + 1) / shares);
    const size_t step = (size_t)slot_rows * (D + 2);
    const int lane = threadIdx.x & 31;
    constexpr int kWide = D / 16;  // warps' worth of dimensions
    const int items = (row1 - row0 + 7) / 8 * kWide;
    // The place of item w's values in a slot; false if this lane has none.
    auto locate = [&](int w, int &row, int &dq, int &at_row) {
        row = row0 + w / kWide * 8 + (lane & 7);
        dq = w % kWide * 4 + (lane >> 3);
        const int node = row / p.g, x = node / p.plan.tile_nodes;
        at_row = x * 128 + row - x * p.plan.tile_nodes * p.g;
        return w < items && row < row1;
    };
    auto finish = [&](int row, int dq, float4 a, float M, float den) {
        const bool seen = den != 0.f;
        const float inv = seen ? 1.f / den : 0.f;
        const int node = row / p.g;
        const size_t orow = (size_t)(cut.q0 + cut.node0 + node) * p.hq + cut.h * p.g + row - node * p.g;
        store_out4(p.out, orow * D + 4 * dq, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv), p.out_type);
        if (p.lse && dq == 0) p.lse[orow] = seen ? (M + log2f(den)) * 0.6931471805599453f : -INFINITY;
    };
    // Pieces s0 .. s0 + kMergeAhead - 1 of the pair: their values, nothing past the last.
    auto load = [&](int s0, int dq, int at_row, bool on, float2 (&ml)[kMergeAhead], float4 (&v)[kMergeAhead]) {
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) {
            const int s = s0 + i;
            ml[i] = make_float2(-INFINITY, 0.f);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && s <= r1) {
                const float *part = p.partial + (s == r0 ? slot0 : 2 * s) * step;
                ml[i] = reinterpret_cast<const float2 *>(part + (size_t)slot_rows * D)[at_row];
                v[i] = reinterpret_cast<const float4 *>(part)[(size_t)dq * slot_rows + at_row];
            }
        }
    };
    // (a piece without a key of the row has nothing to add, whatever its reference)
    auto add = [&](const float2 (&ml)[kMergeAhead], const float4 (&v)[kMergeAhead], float &M, float &den, float4 &a) {
        float up = M;
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) up = fmaxf(up, ml[i].x);
        const float ref = up == -INFINITY ? 0.f : up;
        const float alpha = ex2(M - ref);
        M = up;
        den *= alpha;
        a.x *= alpha, a.y *= alpha, a.z *= alpha, a.w *= alpha;
#pragma unroll
        for (int i = 0; i < kMergeAhead; ++i) {
            if (ml[i].y == 0.f) continue;
            const float e = ex2(ml[i].x - ref);
            den += e * ml[i].y;
            a.x += e * v[i].x, a.y += e * v[i].y, a.z += e * v[i].z, a.w += e * v[i].w;
        }
    };
    constexpr int kStep = kMergeThreads / 32;
    if (r1 - r0 < kMergeAhead) {  // most pairs: all their pieces at once, two items at a time
        for (int w = threadIdx.x >> 5; w < items; w += 2 * kStep) {
            int row[2], dq[2], at_row[2];
            bool on[2];
            float2 ml[2][kMergeAhead];
            float4 v[2][kMergeAhead];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                on[j] = locate(w + j * kStep, row[j], dq[j], at_row[j]);
                load(r0, dq[j], at_row[j], on[j], ml[j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float M = -INFINITY, den = 0.f;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                add(ml[j], v[j], M, den, a);
                if (on[j]) finish(row[j], dq[j], a, M, den);
            }
        }
        return;
    }
    for (int w = threadIdx.x >> 5; w < items; w += kStep) {
        int row, dq, at_row;
        const bool on = locate(w, row, dq, at_row);
        float M = -INFINITY, den = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int s = r0; s <= r1; s += kMergeAhead) {
            float2 ml[kMergeAhead];
            float4 v[kMergeAhead];
            load(s, dq, at_row, on, ml, v);
            add(ml, v, M, den, a);
        }
        if (on) finish(row, dq, a, M, den);
    }
}

namespace {

constexpr int kSimplePerSm = 2;  // CTAs
// Tables of up to this many blocks: no pair is cut, and no second kernel runs.  Sequences that fill their
// tables, 8 nodes each, whole / cut in us.  16-bit pools (four key tiles):
//   pairs of 16, 2, 240, 512 (d 64, 128, 128, 128)   32 blocks 12.1 / 15.1, 13.4 / 15.0, 23.6 / 31.8, 41.1 / 51.7
//                                                   64         15.9 / 15.3, 17.4 / 16.0, 33.1 / 40.0, 61.6 / 74.7
//   (whole wins at 48 too, but there ragged sequences gain from being cut)
// fp32, whose tiles take several times as long (two key tiles):
//   pairs of 8, 320, 800 (d 64, 128, 128)   16 blocks 24.7 / 26.3,  98.2 /  90.6, 175 / 173
//                                           32         44.5 / 37.2, 187.9 / 143.2, 328 / 310
constexpr int kWholeBlocks = 32, kWholeBlocksF32 = 16;

kv_status launch_simple(const TreeParams &pp, int d, cudaStream_t stream) {
    auto fn = d == 64 ? tree_simple_kernel<64> : tree_simple_kernel<128>;
    const int smem = d == 64 ? (int)sizeof(SimpleShared<64>) : (int)sizeof(SimpleShared<128>);
    if (kv_status st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
        return st;
    fn<<<pp.plan.runs, kSimpleThreads, smem, stream>>>(pp);
    return cuda_status(cudaGetLastError());
}

kv_status launch_merge(const TreeParams &pp, int d, int slot_rows, cudaStream_t stream) {
    const dim3 grid((unsigned)pp.plan.runs - 1, (unsigned)slot_rows / 32);
    if (d == 64)
        tree_merge_kernel<64><<<grid, kMergeThreads, 0, stream>>>(pp, slot_rows);
    else
        tree_merge_kernel<128><<<grid, kMergeThreads, 0, stream>>>(pp, slot_rows);
    return cuda_status(cudaGetLastError());
}

// How a call runs: what the workspace query and the call have to agree on.  pair_cost (tree_plan.cuh)
// is what a piece's beginning and end take in key tiles' times, measured: 64 ragged sequences 1 to
// 5 give 131.5, 124.5, 123.1, 124.0 and 125.0 us, 16 trees of two row tiles 111.7, 105.8, 107.2,
// 108.6 and 110.7; fp32, 64 sequences of 300 to 1000 tokens (32 heads over 8, d 64), 1 to 3: 235, 249 and 261 us.  min_run, the least of a run where a batch leaves CTAs without work: one row tile, a
// sequence of 3000 tokens (8 heads over 2): 17.9 us with 4, 18.3 with 5, 18.9 with 6, 20.8 with 8 and
// 24.8 with 12; two, a sequence of 8000 with 64 nodes (16 over 2): 29.8 us with 3, 27.6 with 4, 28.7
// with 6, 31.6 with 8; fp32, a sequence of 3000 (8 over 2, d 128): 30.3 us with 1, 45.6 with 2, 62.1 with 3, 79.5
// with 4, and of 20000, which fills the grid with longer runs, 74.4, 74.4, 69.9 and 85.1.
struct Shape {
    int slot_rows;                // rows of a slot of partial results
    int tile_nodes, group_nodes;  // nodes of a row tile and of a group
    int copies;                   // of each row in its tile
    int runs, pair_cost, min_run;
    bool whole;                   // no pair is cut
};
// Copies as many as fit, two row tiles where a tree has more rows than one (and they have room: the
// third part of the weights takes it).  The query, which does not know the output's type, takes the
// larger workspace: that of 16-bit output.
Shape shape_of(const kv_pool *p, int g, int max_q_len, int max_blocks, kv_dtype out_dtype) {
    if (p->dtype == KV_F32)
        return {kSimpleRows, kSimpleRows / g, kSimpleRows / g, 1, kSimplePerSm * sm_count(), 1, 1,
                max_blocks <= kWholeBlocksF32};
    Shape s{128, 128 / g, 128 / g, 1, sm_count(), 3, 4, max_blocks <= kWholeBlocks};
    if (max_q_len <= 64 / g) {
        s.copies = max_q_len <= 32 / g ? 4 : 2;
        s.tile_nodes = s.group_nodes = 128 / s.copies / g;
    } else if (max_q_len > s.tile_nodes && !(p->dtype == KV_BF16 && out_dtype == KV_F32)) {
        s.slot_rows = 256;
        s.group_nodes = 2 * s.tile_nodes;
        s.pair_cost = 2;
        s.min_run = 4;
    }
    return s;
}

// Two slots and a cut for each run.
size_t slots_bytes(const Shape &s, int d) { return 2 * (size_t)s.runs * s.slot_rows * (d + 2) * sizeof(float); }
size_t workspace_bytes_of(const Shape &s, int d) { return s.whole ? 0 : slots_bytes(s, d) + s.runs * sizeof(Cut); }

// Arguments that the query and the call refuse alike.
kv_status check(kv_pool_t p, int batch, int num_q_heads, int max_blocks, int max_q_len) {
    if (!p || batch < 0 || max_q_len < 0 || max_blocks < 0 || num_q_heads <= 0) return KV_ERR_ARG;
    if (kv_status st = require_device(p->device)) return st;
    if (p->dtype == KV_I4) return KV_ERR_UNSUPPORTED;
    if (num_q_heads % p->num_kv_heads) return KV_ERR_ARG;
    if (num_q_heads / p->num_kv_heads > 8 || max_q_len > kMaxNodes || max_blocks > kMaxBlocks ||
        (p->dtype != KV_F32 && (long long)p->num_blocks * p->num_kv_heads * 16 > INT32_MAX))
        return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

}  // namespace
}  // namespace tree
}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_tree_workspace_size(kv_pool_t p, int batch, int num_q_heads, int max_blocks, int max_q_len,
                                 size_t *bytes) {
    if (!bytes) return KV_ERR_ARG;
    if (kv_status st = tree::check(p, batch, num_q_heads, max_blocks, max_q_len)) return st;
    *bytes = 0;
    if (batch == 0 || max_q_len == 0) return KV_OK;
    const tree::Shape s = tree::shape_of(p, num_q_heads / p->num_kv_heads, max_q_len, max_blocks, p->dtype);
    *bytes = tree::workspace_bytes_of(s, p->head_dim);
    return KV_OK;
}

kv_status paged_tree_attention(kv_pool_t p, const void *q, const int32_t *cu_q, int total_q, int max_q_len,
                               const int32_t *parents, const int32_t *block_tables, int max_blocks,
                               const int32_t *seq_lens, int batch, int num_q_heads, float scale, void *out,
                               kv_dtype out_dtype, float *lse_out, void *workspace, size_t workspace_bytes,
                               void *stream) {
    if (total_q < 0) return KV_ERR_ARG;
    if (kv_status st = tree::check(p, batch, num_q_heads, max_blocks, max_q_len)) return st;
    if (!(scale > 0.f) || !std::isfinite(scale)) return KV_ERR_ARG;
    if (out_dtype != KV_F32 && out_dtype != p->dtype) return KV_ERR_UNSUPPORTED;
    if (batch == 0 || max_q_len == 0 || total_q == 0) return KV_OK;
    if (!q || !cu_q || !block_tables || !seq_lens || !out) return KV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15)
        return KV_ERR_ARG;
    const int g = num_q_heads / p->num_kv_heads;
    const tree::Shape s = tree::shape_of(p, g, max_q_len, max_blocks, out_dtype);
    if (!s.whole && (!workspace || workspace_bytes < tree::workspace_bytes_of(s, p->head_dim))) return KV_ERR_ARG;
    tree::TreeParams pp{};
    pp.plan = {cu_q, seq_lens, batch, total_q, max_q_len, max_blocks, p->num_kv_heads, s.group_nodes,
               s.tile_nodes, s.runs, s.pair_cost, s.min_run, s.whole};
    pp.copies = s.copies;
    pp.total_q = total_q;
    pp.q = q;
    pp.k = p->k;
    pp.v = p->v;
    pp.tables = block_tables;
    pp.parents = parents;
    pp.num_blocks = p->num_blocks;
    pp.hq = num_q_heads;
    pp.g = g;
    pp.scale_log2 = scale * 1.4426950408889634f;
    pp.out = out;
    pp.out_type = out_dtype;
    pp.lse = lse_out;
    pp.partial = static_cast<float *>(workspace);
    if (!s.whole) pp.cuts = reinterpret_cast<tree::Cut *>(static_cast<char *>(workspace) + tree::slots_bytes(s, p->head_dim));
    pp.err = p->err;
    if (p->dtype == KV_F32) {
        if (kv_status st = tree::launch_simple(pp, p->head_dim, as_stream(stream))) return st;
    } else {
        if (kv_status st = pool_group_maps(p)) return st;
        if (kv_status st = tree::launch_tc(pp, p->head_dim, s.slot_rows, p->dtype == KV_F16, p->gmap_k, p->gmap_v,
                                           as_stream(stream)))
            return st;
    }
    if (s.whole) return KV_OK;
    return tree::launch_merge(pp, p->head_dim, s.slot_rows, as_stream(stream));
}

}  // extern "C"
