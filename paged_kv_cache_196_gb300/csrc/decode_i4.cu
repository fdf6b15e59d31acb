// Decode attention over a 4-bit pool, and its form for a few query tokens.
//
// Maths: o = softmax(scale * q K^T) V per query head, K and V as their codes
// stand for them (i4.cuh), with a running maximum and sum over the blocks and a
// log-sum-exp merge of the partitions of one sequence, as the 16-bit decode.
//
// What bounds it.  A token's K and V take 9 D / 8 bytes per kv head against 4 D
// in 16 bits, while every code still has to become an fp16 operand.  So the
// kernel is written around the number of instructions per code: one logical
// operation and one fused multiply-add make two codes into a scaled fp16 pair
// (i4::values8: 9 instructions for 8 codes), the layout of a tile puts each
// lane's operands of the tensor core's fragments into consecutive bytes (no
// ldmatrix, no shuffles), the scales of a lane's rows are two bytes a load, a
// warp takes two blocks (NB) at a time, so that waiting, the maximum over lanes and the
// test for a new maximum are paid once per pair of blocks, and a warp of its own does
// all that copying needs.
//
// Shape.  A pair is one (sequence, kv head) with up to 8 NT of its query columns
// (head of the group, and query token where there are several).  Its blocks are
// taken in rounds: a round is NB blocks for each of a CTA's seven attending warps,
// which keep their own softmax states and meet at a pair's end.  The eighth warp
// copies a round per ring stage, reads the table a round ahead and lays out the next
// pair's queries.
// (Eight warps in all: the register file is split in four, so a ninth warp would
// cost every warp a fifth of its registers.)
//
// Balance.  The rounds of all pairs are laid end to end and cut into one equal run
// per CTA of a single wave; every CTA finds its run from the lengths on the device
// (a scan of the batch), so a captured graph stays balanced when the lengths change.
// The copies run ahead across pair boundaries.  A pair cut by runs leaves a partial
// result per CTA, which the last of them merges.  A pair counts i4_pair_cost
// rounds more than it has, for its queries and its end.
//
// Products.  S^T[16 tokens][8 columns] = K q^T and O^T[16 dims][8 columns] += V^T
// P^T on mma.sync m16n8k16 with fp32 sums.  The contraction over dimensions may run
// in any order, so lane (r, c) = (lane / 4, lane % 4) takes a quarter row of tokens
// r and r + 8 as it lies in memory, and q is laid out to match once per CTA.  O's
// rows are dimensions D/8 r + 2 f and + 1 of product f: each lane ends with D / 8
// consecutive dimensions of two columns.
//
// Measured.  64 sequences of 512 to 4096 tokens (8 kv heads of 4 query heads, 128 dims):
// 171 MB in 43.7 us, 3910 GB/s (0.58 of a device copy); 8 sequences of 32768 to 196608
// tokens (4 of 8): 437 MB in 85.8 us, 5100 GB/s (0.75), while the 16-bit decode reads
// 3.6 times the bytes at 0.92 and 0.96.  Not memory but instructions bound it: about 300
// per warp and 16 tokens, the schedulers issuing in 55 to 60% of cycles from four warps
// each; stalls are spread over fixed latencies, busy pipes and instruction fetch.  Short
// sequences lose the rest at the pieces' ends (queries, merge): 2048 pairs of 1 to 64 tokens
// take 29.3 us, a pair 3.7 us of a CTA's, whose rounds are mostly empty.  Tried and slower: one
// or three blocks a warp; 3, 5, 9 or 11 warps; four warps that copy for themselves;
// other ring depths; the products rolled into loops (89 to 95 us for the long ones).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "i4.cuh"
#include "internal.h"
#include "i4_attend.h"

namespace pkv {

constexpr int kI4Warps = 7;                      // attending warps of a CTA
constexpr int kI4Attend = kI4Warps * 32;
constexpr int kI4Threads = kI4Attend + 32;       // and the copying warp
constexpr int kI4MergeThreads = 128;             // of merge_i4_kernel
constexpr int kI4BS = 16;
constexpr int NB = 2;                 // blocks of a warp's share of a round
constexpr int kI4Round = NB * kI4Warps;  // blocks of a round
// Rounds that a pair costs besides its own (its queries and its end), for 8 NT columns.
// Measured with 0, 1, 2, 3: decode of 64 sequences 48.4, 45.0, 46.1, 47.6 us (NT = 1);
// with 1 .. 5 and 7: five drafted tokens of 16 sequences 51.8, 46.9, 44.2, 43.2, 43.6,
// 46.0 us (NT = 3).
constexpr int i4_pair_cost(int NT) { return NT == 1 ? 1 : 4; }
constexpr int kI4MinRun = 2;         // shortest run: a pair's cost and a round
constexpr int kI4ScanBatch = 4096;   // largest batch whose runs the device cuts
// Pairs per CTA of a wave beyond which runs of whole pairs (the ring and the queries carry
// over from pair to pair) replace a CTA for each: 2048 pairs of 1 to 64 tokens 39.0 us by a
// CTA each, 29.3 by runs; 2000 of 20 to 200 38.8 / 30.4; 2048 of 256 55.7 / 43.6.
constexpr int kI4UncutPairs = 2;
constexpr int kI4MaxRows = 65535;    // of a grid's third dimension
constexpr int kI4ShortPair = 8;      // rounds of a pair that may better stay whole
// The weights are 2^(s - m + 6) for a reference m that is renewed (and the state
// rescaled) only when the maximum passes it by more than 2^8: rarely after the
// first blocks, and exact mathematics, since sums and outputs share m.  They stay
// below 2^14, in fp16's range, and the largest seen is at least 2^6.
// With 16-bit output a weight is one fp16 number (off by at most 2^-11 of it), with fp32
// output two, which doubles the products with V: the rounding to a bf16 output is 8 times
// that, and the error of 64 sequences' outputs against 64 bits is 1.656e-3 where weights of
// 24 bits leave 1.646e-3 (drafted tokens in fp16: 2.30e-4, 2.07e-4).
constexpr float kI4Bias = 6.f, kI4Renew = 8.f;

struct I4Params {
    const uint16_t *q;      // rows [hq][D], bf16 or fp16
    int q_bf16;
    const int32_t *cu_q;    // null: one query token per sequence, row b
    int total_q, max_t;     // rows of q and out; most query tokens of a sequence
    const char *pool;
    const int32_t *tables;
    int max_blocks, num_blocks;
    const int32_t *seq_lens, *seq_order;
    int batch, hq, hkv, g;
    float scale_log2;       // softmax scale * log2(e) * kScaleUnit * the pool's K scale
    float v_mul;            // kScaleUnit * the pool's V scale
    // balanced: one run per CTA, at most max_splits to a pair; uncut: a run takes the
    // pairs that begin in it whole.  Otherwise CTA (split, kv head, (sequence, column
    // group)) takes part_rounds rounds; what the grid's third dimension does not hold of
    // the last follows in the first, max_splits further each time.
    int balanced, uncut;
    int part_rounds, max_splits;
    int cols;               // columns of a pair (the kernel's own)
    int col_groups;         // pairs that share a sequence's columns of one kv head
    void *out;
    int out_type;
    float *lse;
    float *ws_o, *ws_lse;   // [b][query token][hq][max_splits] partial results and their lse
    int *counters;          // null: merge_i4_kernel merges
    int *err;
};

constexpr float kLn2 = 0.6931471805599453f;

// One more arrival; what the arriving CTA's threads wrote before a barrier is visible to
// whoever sees the count (and the other way round).
KV_DEVICE int count_arrival(int *counter) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    return old;
}

KV_DEVICE float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Whether a phase is complete, without the suspension of mbarrier.try_wait.
KV_DEVICE bool phase_done(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// One lane of a converged warp, in the form that lets the compiler issue copies from
// uniform registers (under an ordinary lane test it loops over the lanes).
KV_DEVICE bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

KV_DEVICE void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 transpose of a 16-bit fragment.
KV_DEVICE uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// N words of shared memory, 16 or 8 bytes at once.
template <int N>
KV_DEVICE void load_words(const char *src, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(src);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(src);
        w[0] = u.x, w[1] = u.y;
    }
}

// Shared memory asked for at launch: the ring (a stage: a round's blocks) and the
// merge's outputs ([warp][column][D]).  With the kernel's own variables, two CTAs of
// the D = 128 decode fill an SM's to the last hundred bytes.
template <int D, int NST>
constexpr size_t i4_ring_bytes() {
    return (size_t)NST * kI4Round * 2 * 9 * D;
}
// Columns that are merged at once: with one tile of eight the shared memory of a second
// CTA per SM leaves room for four.
constexpr int i4_merge_cols(int NT) { return NT == 1 ? 4 : 8 * NT; }
template <int D, int NT>
constexpr size_t i4_merge_bytes() {
    return (size_t)kI4Warps * i4_merge_cols(NT) * D * 4;
}
template <int D, int NT, int NST>
constexpr size_t i4_smem_bytes() {
    return i4_ring_bytes<D, NST>() + i4_merge_bytes<D, NT>();
}

// A sequence: its query rows, keys, rounds, and the pairs it makes (0: left out).
struct I4Work {
    int b, q0, T, nblk, rounds, pairs;
    int L;
};

// A CTA's share of a pair, which the copying warp hands to the attending ones.
struct I4Piece {
    int b, q0, T, L;         // its sequence
    int h, cg;               // kv head, column group
    int round0, rounds;      // rounds: 0 ends the run
    int split, nsplit;       // which of the pair's pieces
};

// Row of a query head in q and out, and in the workspace.
KV_DEVICE size_t out_row(const I4Params &p, int q0, int tq, int hq) { return (size_t)(q0 + tq) * p.hq + hq; }
KV_DEVICE size_t ws_row(const I4Params &p, int b, int tq, int hq) {
    return ((size_t)b * p.max_t + tq) * p.hq + hq;
}

// round_blocks: blocks of a round; cols: columns of a pair; report: flag what is wrong.
KV_DEVICE I4Work i4_sequence(const I4Params &p, int b, int round_blocks, int cols, bool report) {
    I4Work w{};
    w.b = b;
    long long L = p.seq_lens[b];
    const long long most = (long long)p.max_blocks * kI4BS;
    if (p.cu_q) {
        w.q0 = p.cu_q[b];
        w.T = p.cu_q[b + 1] - w.q0;
        if (w.T <= 0) return w;
        if (L < w.T || L > most || w.T > p.max_t || w.q0 < 0 || (long long)w.q0 + w.T > p.total_q) {
            if (report) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
            return w;
        }
    } else {
        w.q0 = b;
        w.T = 1;
        if (L > most) {
            if (report) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
            L = most;
        }
        if (L < 0) L = 0;
    }
    w.L = (int)L;
    w.nblk = (w.L + kI4BS - 1) / kI4BS;
    w.rounds = max(1, (w.nblk + round_blocks - 1) / round_blocks);
    w.pairs = p.hkv * ((w.T * p.g + cols - 1) / cols);
    return w;
}

// The D / 32 elements of column gc's query that this lane lays out.
template <int D>
KV_DEVICE void load_query(const I4Params &p, int q0, int T, int h, int gc, int lane, uint32_t (&two)[D / 64]) {
    const int tq = T == 1 ? 0 : gc / p.g;
    const uint16_t *src = p.q + out_row(p, q0, tq, h * p.g + gc - tq * p.g) * D + lane * (D / 32);
    if constexpr (D == 128) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src));
        two[0] = u.x, two[1] = u.y;
    } else {
        two[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
    }
}

// A warp lays out the query of a column: its largest magnitude to [2^13, 2^14) by a
// power of two, so that fp16 holds it, then into the order of the fragments.
template <int D, int NT>
KV_DEVICE void put_query(const I4Params &p, const uint32_t (&two)[D / 64], int col, int lane, uint2 *fragments,
                         float *scale) {
    constexpr int kPer = D / 32;
    __half *qs = reinterpret_cast<__half *>(fragments);
    float x[kPer], m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        const float2 f = p.q_bf16 ? bf16x2_to_float2(two[i / 2]) : f16x2_to_float2(two[i / 2]);
        x[i] = f.x, x[i + 1] = f.y;
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    // exponent field of the largest; 0 (all zero or below normal) and 255 are left alone
    const int e = (int)(__float_as_uint(m) >> 23);
    const int up = e == 0 || e == 255 ? 0 : max(-126, min(126, 127 + 13 - e));
    // the score's factor is made positive (its sign goes to q), so that scaling keeps the
    // order of scores; a factor of 0 zeroes q instead, and one that is no number makes it
    // NaN (a score's factor of NaN would reach masked keys too)
    const bool zero = p.scale_log2 == 0.f, finite = fabsf(p.scale_log2) < INFINITY;
    const float mul = finite ? copysignf(zero ? 0.f : __uint_as_float((uint32_t)(127 + up) << 23), p.scale_log2) : NAN;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        // dimension d: quarter cq, word in / 8, four bits in % 4 of half in / 4 % 2
        const int d = lane * kPer + i, cq = d / (D / 4), in = d % (D / 4);
        const int to = 4 * (in / 8) + in % 4, hi = in / 4 % 2;
        qs[((((to >> 1) * NT + (col >> 3)) * 32 + (col & 7) * 4 + cq) * 2 + (to & 1)) * 2 + hi] = __float2half_rn(x[i] * mul);
    }
    if (lane == 0)
        scale[col] = zero || !finite ? 1.f : fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)(127 - up) << 23), 1e-37f);
}

// D: head dim.  NT: columns / 8 of a CTA.  EXACT: weights in two fp16 parts (fp32
// output).  TW: waits read their limit at run time (tests).  NST: ring stages; MINB:
// CTAs per SM it is built for.
template <int D, int NT, bool EXACT, bool TW, int NST, int MINB>
__global__ void __launch_bounds__(kI4Threads, MINB) decode_i4_kernel(const I4Params p) {
    constexpr int kTile = 9 * D;
    constexpr int kW = D / 32;        // words of a quarter row of K, of a lane's dims of a V pair
    constexpr int kSteps = D / 16;    // products along D
    constexpr int kRound = kI4Round;
    constexpr int kStage = kRound * 2 * kTile;
    constexpr int kCols = 8 * NT;
    constexpr int kPairCost = i4_pair_cost(NT);
    static_assert(kRound <= 32, "a lane looks after one block of a round");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    extern __shared__ __align__(128) char smem[];
    constexpr size_t kRing = i4_ring_bytes<D, NST>();
    __shared__ uint64_t full[NST], empty[NST];
    __shared__ volatile int missing[NST];  // bit i: block i of the round is not there
    constexpr int kMC = i4_merge_cols(NT);
    __shared__ uint2 s_q[2][kSteps * NT * 32];  // fragments of two pieces' queries
    __shared__ float s_scale[2][8 * NT];
    __shared__ I4Piece s_piece[2];
    __shared__ uint64_t s_qfull[2], s_qempty[2];  // of a piece's description and queries
    __shared__ float s_m[kI4Warps * kMC], s_l[kI4Warps * kMC];
    __shared__ int s_last;
    // of the scan of the batch, over before the merges' are used
    int *s_scan = reinterpret_cast<int *>(s_m), *s_most = s_scan + kI4Warps + 1;
    int *s_start = reinterpret_cast<int *>(s_l);
    __shared__ volatile int s_abort;  // a wait ran out

    if (tid == 0) {
        for (int st = 0; st < NST; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], kI4Warps);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&s_qfull[k], 1);
            mbar_init(&s_qempty[k], kI4Warps);
        }
        mbar_init_fence();
        s_abort = 0;
    }

    // ---- this CTA's run: `todo` units (rounds and pair costs) from unit `unit` of
    // sequence b0 on, whose first unit is number `base` of all
    int b0, unit, base, todo, run = 0, split = 0;
    if (p.balanced) {
        // each thread adds up a slice of the batch, then the slices are scanned
        const int per = (p.batch + kI4Threads - 1) / kI4Threads;
        const int first = tid * per, past = min(p.batch, first + per);
        int sum = 0, most = 1;
        for (int b = first; b < past; ++b) {
            const I4Work w = i4_sequence(p, b, kRound, kCols, blockIdx.x == 0);
            if (w.pairs) most = max(most, w.rounds);
            sum += w.pairs * (w.rounds + kPairCost);
        }
        int scan = sum;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, scan, y);
            if (lane >= y) scan += v;
            most = max(most, __shfl_xor_sync(0xffffffffu, most, y));
        }
        if (lane == 31) s_scan[warp] = scan, s_most[warp] = most;
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int y = 0; y <= kI4Warps; ++y) {
            if (y < warp) scan += s_scan[y];
            total += s_scan[y];
            most = max(most, s_most[y]);
        }
        // a pair of n rounds is cut into at most (n - 2) / run + 2 pieces
        run = (total + (int)gridDim.x - 1) / (int)gridDim.x;
        if (!p.uncut) run = max(run, (most + p.max_splits - 3) / (p.max_splits - 1));
        run = max(run, kI4MinRun);
        const long long at64 = (long long)blockIdx.x * run;
        if (at64 >= total) return;
        const int at = (int)at64;
        if (at >= scan - sum && at < scan) {
            int left = at - (scan - sum);
            for (int b = first; b < past; ++b) {
                const I4Work w = i4_sequence(p, b, kRound, kCols, false);
                const int n = w.pairs * (w.rounds + kPairCost);
                if (left < n) {
                    s_start[0] = b, s_start[1] = left, s_start[2] = at - left;
                    break;
                }
                left -= n;
            }
        }
        __syncthreads();
        b0 = s_start[0], unit = s_start[1], base = s_start[2];
        todo = min(run, total - at);
        if (p.uncut) {  // on to the first pair that begins in the run; none: todo <= 0
            const int per_pair = i4_sequence(p, b0, kRound, kCols, false).rounds + kPairCost, in = unit % per_pair;
            const int skip = in ? per_pair - in : 0;
            unit += skip;
            todo -= skip;
        }
    } else {
        int row = blockIdx.z;
        split = blockIdx.x;
        for (; split >= p.max_splits; split -= p.max_splits) row += gridDim.z;
        b0 = row / p.col_groups;
        const int cg = row % p.col_groups;
        if (b0 >= p.batch) return;
        const bool reports = tid == 0 && split == 0 && blockIdx.y == 0 && cg == 0;
        if (p.seq_order) {
            b0 = __ldg(p.seq_order + b0);
            if (b0 < 0 || b0 >= p.batch) {  // not a permutation of the batch
                if (reports) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
                return;
            }
        }
        const I4Work w = i4_sequence(p, b0, kRound, kCols, reports);
        const int pair = cg * p.hkv + blockIdx.y, r0 = split * p.part_rounds;
        if (pair >= w.pairs || r0 >= w.rounds) return;
        base = 0;
        unit = pair * (w.rounds + kPairCost) + kPairCost + r0;
        todo = min(p.part_rounds, w.rounds - r0);
    }
    __syncthreads();

    if (warp == kI4Warps) {
        // ================================================== the copying warp
        // Lane i looks after block i of a round; one lane issues every copy.
        I4Work w = i4_sequence(p, b0, kRound, kCols, false);
        const uint64_t policy = l2_evict_first_policy();
        int pair = 0, round = 0;
        // Moves to the next unit that is a round; false at the run's end.
        auto place = [&]() -> bool {
            while (todo > 0) {
                const int per = w.rounds + kPairCost;
                if (unit >= w.pairs * per) {
                    base += w.pairs * per;
                    w = i4_sequence(p, w.b + 1, kRound, kCols, false);
                    unit = 0;
                    continue;
                }
                pair = unit / per;
                round = unit - pair * per - kPairCost;
                if (round >= 0) return true;
                if (p.uncut) {  // begun in this run: its rounds are this CTA's too
                    unit -= round;
                    todo += round;
                    round = 0;
                    return true;
                }
                ++unit;
                --todo;
            }
            return false;
        };
        // The piece that begins at this place.
        auto describe = [&]() {
            I4Piece d{};
            d.b = w.b, d.q0 = w.q0, d.T = w.T, d.L = w.L;
            d.h = pair % p.hkv, d.cg = pair / p.hkv;
            d.round0 = round;
            d.rounds = p.uncut ? w.rounds : min(w.rounds - round, todo);
            if (p.uncut) {
                d.nsplit = 1;
            } else if (p.balanced) {
                const int v0 = base + pair * (w.rounds + kPairCost) + kPairCost;  // the pair's first round
                const int c0 = v0 / run, c1 = (v0 + w.rounds - 1) / run;
                d.nsplit = c1 - c0 + 1;
                d.split = blockIdx.x - c0;
            } else {
                d.nsplit = (w.rounds + p.part_rounds - 1) / p.part_rounds;
                d.split = split;
            }
            return d;
        };
        int id_next = -1;      // table entry of this lane's next block
        bool in_next = false;  // that block is one of the sequence's
        auto entry = [&]() {
            const int blk = round * kRound + lane;
            in_next = lane < kRound && blk < w.nblk;
            if (in_next) id_next = __ldg(p.tables + (size_t)w.b * p.max_blocks + blk);
        };
        // Hands piece number `piece` over: its description and, but for the first one's
        // (the attending warps lay that out), its queries.  False if the buffer did not
        // come free.
        auto hand = [&](const I4Piece &d, int piece) -> bool {
            constexpr int kAhead = 4;
            const int buf = piece & 1, col0 = d.cg * kCols, ncols = min(kCols, d.T * p.g - col0);
            if (piece > 0) {
                const bool bad = lane == 0 && !mbar_wait<TW>(&s_qempty[buf], ((piece - !buf * 2) >> 1) & 1, p.err);
                if (__shfl_sync(0xffffffffu, bad, 0)) return false;
            }
            if (lane == 0) s_piece[buf] = d;
            for (int first = 0; piece > 0 && d.rounds > 0 && first < ncols; first += kAhead) {
                uint32_t two[kAhead][D / 64];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    load_query<D>(p, d.q0, d.T, d.h, col0 + min(first + k, ncols - 1), lane, two[k]);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (first + k < ncols) put_query<D, NT>(p, two[k], first + k, lane, s_q[buf], s_scale[buf]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_qfull[buf]);
            return true;
        };
        bool more = place(), starts = true;  // starts: the round begins a piece
        if (more) entry();
        int issued = 0, pieces = 0;
        I4Piece d{};
        if (more) {
            d = describe();
            hand(d, pieces++);
        }
        while (more) {
            const int id = id_next, h = d.h, st = issued % NST;
            const bool inside = in_next;
            // the next round's entries are on their way while this round is copied
            ++unit;
            --todo;
            ++round;
            starts = round >= w.rounds;
            more = starts ? place() : p.uncut || todo > 0;
            if (more) entry();
            bool bad = false;
            if (lane == 0) {
                // the ring is full most of the time: look now and then, not in every free slot
                for (int i = 0; i < 256 && issued >= NST && !mbar_try_wait(&empty[st], (issued / NST - 1) & 1); ++i)
                    __nanosleep(50);
                bad = s_abort || (issued >= NST && !mbar_wait<TW>(&empty[st], (issued / NST - 1) & 1, p.err));
            }
            if (__shfl_sync(0xffffffffu, bad, 0)) {
                if (lane == 0) s_abort = 1;
                break;
            }
            const bool ok = inside && id >= 0 && id < p.num_blocks;
            const uint32_t there = __ballot_sync(0xffffffffu, ok);
            const uint32_t gone = __ballot_sync(0xffffffffu, inside && !ok);
            if (gone && lane == 0) atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
            const long long off = ((long long)id * p.hkv + h) * (2 * kTile);
            const bool leader = elect_one();
            if (leader) {
                missing[st] = (int)gone;
                if (there)
                    mbar_arrive_expect_tx(&full[st], 2 * __popc(there) * kTile);
                else
                    mbar_arrive(&full[st]);
            }
            char *dst = smem + st * kStage;
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
                const long long at = __shfl_sync(0xffffffffu, off, i);
                if ((there >> i & 1) && leader) {
                    bulk_g2s(dst + 2 * i * kTile, p.pool + at, 2 * kTile, &full[st], policy);
                }
            }
            ++issued;
            if (more && starts) {
                d = describe();
                if (!hand(d, pieces++)) {
                    if (lane == 0) s_abort = 1;
                    break;
                }
            }
        }
        if (!more) {  // the end of the run, as a piece of no rounds
            d.rounds = 0;
            if (!hand(d, pieces) && lane == 0) s_abort = 1;
        }
        // Never leave while a copy into this CTA's shared memory may be in flight.
        if (lane == 0)
            for (int k = max(0, issued - NST); k < issued; ++k) mbar_wait_drain(&full[k % NST], (k / NST) & 1, p.err);
        return;
    }

    // ====================================================== attending warps
    const int r = lane >> 2, c = lane & 3;
    // columns without a query hold zeros (later pieces may leave old ones: a column's
    // values reach no other column)
    for (int i = tid; i < 2 * kSteps * NT * 32; i += kI4Attend) s_q[0][i] = make_uint2(0u, 0u);
    for (int i = tid; i < 2 * 8 * NT; i += kI4Attend) s_scale[0][i] = 1.f;
    named_bar_sync(1, kI4Attend);
    if (lane == 0) mbar_arrive(&s_qempty[1]);  // the second piece's buffer is free

    int st = 0;
    uint32_t parity = 0;
    bool stop = false;
    // Test instantiation with a limit of 0: a round that is not there at once is a
    // wait that ran out (try_wait would sleep until it came).
    if constexpr (TW) {
        if (g_wait_limit_ns == 0) {
            stop = __any_sync(0xffffffffu, !phase_done(&full[0], 0));
            if (stop && lane == 0) {
                atomicOr(p.err, KV_DEVERR_TIMEOUT);
                s_abort = 1;
            }
        }
    }
    for (int piece = 0;; ++piece) {
        const int buf = piece & 1;
        if (!stop) stop = __any_sync(0xffffffffu, !mbar_wait<TW>(&s_qfull[buf], (piece >> 1) & 1, p.err));
        if (stop && lane == 0) s_abort = 1;
        // All warps go on or none; and the previous piece's results have been read.
        if (named_bar_or(1, kI4Attend, stop)) break;
        const volatile I4Piece &d = s_piece[buf];
        const int nrounds = d.rounds;
        if (nrounds == 0) break;
        const int round0 = d.round0, L = d.L, T = d.T, col0 = d.cg * kCols, ncols = min(kCols, T * p.g - col0);
        if (piece == 0) {
            const int q0 = d.q0, h = d.h;
            for (int col = warp; col < ncols; col += kI4Warps) {
                uint32_t two[D / 64];
                load_query<D>(p, q0, T, h, col0 + col, lane, two);
                put_query<D, NT>(p, two, col, lane, s_q[0], s_scale[0]);
            }
            named_bar_sync(1, kI4Attend);
        }

        // ---- state of columns 8 nt + 2 c and + 1 (maxima replicated over r)
        // past: the raw score that renews the reference m_run; less: kI4Bias - m_run
        float m_run[NT][2], l_run[NT][2], o[NT][kSteps][4], sc[NT][2], past[NT][2], less[NT][2];
        int lim[NT][2];  // keys that the column sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int col = 8 * nt + 2 * c + x;
                m_run[nt][x] = past[nt][x] = -INFINITY;
                l_run[nt][x] = less[nt][x] = 0.f;
                sc[nt][x] = s_scale[buf][col];
                lim[nt][x] = L - T + (T == 1 ? 1 : min((col0 + col) / p.g, T - 1) + 1);
#pragma unroll
                for (int f = 0; f < kSteps; ++f) o[nt][f][x] = o[nt][f][2 + x] = 0.f;
            }
        const int least = L - T + (T == 1 ? 0 : col0 / p.g) + 1;  // keys that every column sees

        for (int j = 0; j < nrounds && !stop; ++j) {
            const bool bad = !mbar_wait<TW>(&full[st], parity, p.err);
            stop = __any_sync(0xffffffffu, bad);
            if (stop) {
                if (lane == 0) s_abort = 1;
                break;
            }
            const char *stage = smem + st * kStage + NB * warp * 2 * kTile;
            const int tok0 = ((round0 + j) * kRound + NB * warp) * kI4BS;
            // ---- S^T = K q^T: tokens r, r + 8 of each block
            float s[NB][NT][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[n][nt][0] = s[n][nt][1] = s[n][nt][2] = s[n][nt][3] = 0.f;
            {
                uint32_t k0[NB][kW], k1[NB][kW];
                __half2 a0[NB], a1[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const char *kt = stage + 2 * n * kTile;
                    load_words<kW>(kt + r * (D / 2) + c * (D / 8), k0[n]);
                    load_words<kW>(kt + (r + 8) * (D / 2) + c * (D / 8), k1[n]);
                    uint32_t s0, s1;
                    if constexpr (D == 128) {
                        s0 = *reinterpret_cast<const uint16_t *>(kt + 8 * D + r * 8 + 2 * c);
                        s1 = *reinterpret_cast<const uint16_t *>(kt + 8 * D + (r + 8) * 8 + 2 * c);
                    } else {
                        s0 = *reinterpret_cast<const uint8_t *>(kt + 8 * D + r * 4 + c);
                        s1 = *reinterpret_cast<const uint8_t *>(kt + 8 * D + (r + 8) * 4 + c);
                    }
                    a0[n] = i4::scale_pair(s0);
                    a1[n] = i4::scale_pair(s1);
                }
                i4::Scale g0[NB], g1[NB];
#pragma unroll
                for (int wi = 0; wi < kW; ++wi) {
                    uint32_t x0[NB][4], x1[NB][4];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        if (wi == 0) {
                            g0[n] = i4::make_scale(__low2half2(a0[n]));
                            g1[n] = i4::make_scale(__low2half2(a1[n]));
                        } else if (D == 128 && wi == 2) {
                            g0[n] = i4::make_scale(__high2half2(a0[n]));
                            g1[n] = i4::make_scale(__high2half2(a1[n]));
                        }
                        i4::values8(k0[n][wi], g0[n], x0[n]);
                        i4::values8(k1[n][wi], g1[n], x1[n]);
                    }
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 bq = s_q[buf][((2 * wi + f) * NT + nt) * 32 + lane];
#pragma unroll
                            for (int n = 0; n < NB; ++n)
                                mma_16816(s[n][nt], x0[n][2 * f], x1[n][2 * f], x0[n][2 * f + 1], x1[n][2 * f + 1], bq.x, bq.y);
                        }
                }
            }
            // ---- V: token pairs c, c + 4 of each block, dimensions D / 8 r ..
            uint32_t v0[NB][kW], v1[NB][kW], vs0[NB], vs1[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const char *vt = stage + (2 * n + 1) * kTile;
                load_words<kW>(vt + c * D + 4 * ((r * kW) ^ i4::v_swizzle<D>(c)), v0[n]);
                load_words<kW>(vt + (c + 4) * D + 4 * ((r * kW) ^ i4::v_swizzle<D>(c + 4)), v1[n]);
                const int gr = D == 128 ? 2 * r : (r & ~1);
                vs0[n] = *reinterpret_cast<const uint16_t *>(vt + 8 * D + c * (D / 8) + gr);
                vs1[n] = *reinterpret_cast<const uint16_t *>(vt + 8 * D + (c + 4) * (D / 8) + gr);
            }
            // tokens past the sequence, or in a block that is not there
            const int gone = missing[st] >> (NB * warp) & ((1 << NB) - 1);
            const bool whole = !gone && tok0 + NB * kI4BS <= L;
            // the stage is in registers: its next round may come
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            if (++st == NST) {
                st = 0;
                parity ^= 1;
            }
            auto tokens = [&](int n) { return gone >> n & 1 ? 0 : min(kI4BS, L - (tok0 + n * kI4BS)); };

            // ---- softmax: s[0], s[1] token r, columns 2 c, 2 c + 1; s[2], s[3] token r + 8
            uint32_t ph[NB][NT][2], pl[NB][NT][2];
            const bool masked = !whole || tok0 + NB * kI4BS > least;
            if (masked) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int t = r + 4 * (x & 2);
                            if (t >= tokens(n) || tok0 + n * kI4BS + t >= lim[nt][x & 1]) s[n][nt][x] = -INFINITY;
                        }
            }
            // a score past a column's limit renews its reference: looked at per lane, the
            // maximum over lanes is taken only then
            bool renew = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float m = fmaxf(s[0][nt][x], s[0][nt][2 + x]);
#pragma unroll
                    for (int n = 1; n < NB; ++n) m = fmaxf(m, fmaxf(s[n][nt][x], s[n][nt][2 + x]));
                    renew |= m > past[nt][x];
                }
            if (__any_sync(0xffffffffu, renew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float m = fmaxf(s[0][nt][x], s[0][nt][2 + x]);
#pragma unroll
                        for (int n = 1; n < NB; ++n) m = fmaxf(m, fmaxf(s[n][nt][x], s[n][nt][2 + x]));
#pragma unroll
                        for (int y = 4; y <= 16; y <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
                        m = fmaxf(m * sc[nt][x], m_run[nt][x]);
                        // 2^(old - new); an empty state has a reference of -inf
                        const float a = m == m_run[nt][x] ? 1.f : ex2(m_run[nt][x] - m);
                        m_run[nt][x] = m;
                        past[nt][x] = m == -INFINITY ? -INFINITY : (m + kI4Renew) / sc[nt][x];
                        less[nt][x] = m == -INFINITY ? 0.f : kI4Bias - m;
                        l_run[nt][x] *= a;
#pragma unroll
                        for (int f = 0; f < kSteps; ++f) {
                            o[nt][f][x] *= a;
                            o[nt][f][2 + x] *= a;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float p0 = ex2(fmaf(s[n][nt][0], sc[nt][0], less[nt][0])), p1 = ex2(fmaf(s[n][nt][1], sc[nt][1], less[nt][1]));
                    const float p2 = ex2(fmaf(s[n][nt][2], sc[nt][0], less[nt][0])), p3 = ex2(fmaf(s[n][nt][3], sc[nt][1], less[nt][1]));
                    l_run[nt][0] += p0 + p2;
                    l_run[nt][1] += p1 + p3;
                    const uint32_t h01 = float2_to_f16x2(p0, p1), h23 = float2_to_f16x2(p2, p3);
                    ph[n][nt][0] = transpose8(h01);
                    ph[n][nt][1] = transpose8(h23);
                    if constexpr (EXACT) {
                        const float2 f01 = f16x2_to_float2(h01), f23 = f16x2_to_float2(h23);
                        pl[n][nt][0] = transpose8(float2_to_f16x2(p0 - f01.x, p1 - f01.y));
                        pl[n][nt][1] = transpose8(float2_to_f16x2(p2 - f23.x, p3 - f23.y));
                    }
                }
            }
            // ---- O^T += V^T P^T.  Slots past the sequence may hold anything: a scale
            // of zero makes their values zero (codes are finite).
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                __half2 a = i4::scale_pair(vs0[n]), e = i4::scale_pair(vs1[n]);
                if (!whole) {
                    uint32_t ab = *reinterpret_cast<uint32_t *>(&a), eb = *reinterpret_cast<uint32_t *>(&e);
                    const int ntok = tokens(n);
                    ab &= (2 * c < ntok ? 0xffffu : 0u) | (2 * c + 1 < ntok ? 0xffff0000u : 0u);
                    eb &= (2 * c + 8 < ntok ? 0xffffu : 0u) | (2 * c + 9 < ntok ? 0xffff0000u : 0u);
                    a = *reinterpret_cast<__half2 *>(&ab);
                    e = *reinterpret_cast<__half2 *>(&eb);
                }
                const i4::Scale g0 = i4::make_scale(a), g1 = i4::make_scale(e);
#pragma unroll
                for (int wi = 0; wi < kW; ++wi) {
                    uint32_t x0[4], x1[4];
                    i4::values8(v0[n][wi], g0, x0);
                    i4::values8(v1[n][wi], g1, x1);
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816(o[nt][2 * wi + f], x0[2 * f], x0[2 * f + 1], x1[2 * f], x1[2 * f + 1], ph[n][nt][0],
                                      ph[n][nt][1]);
                            if constexpr (EXACT)
                                mma_16816(o[nt][2 * wi + f], x0[2 * f], x0[2 * f + 1], x1[2 * f], x1[2 * f + 1], pl[n][nt][0],
                                          pl[n][nt][1]);
                        }
                }
            }
        }

        // what the loop had no need of
        const int b = d.b, q0 = d.q0, h = d.h, split = d.split, nsplit = d.nsplit;
        // ---- the warps' states to this piece's result, kMC columns at a time
        float4 *sm_o = reinterpret_cast<float4 *>(smem + kRing);  // [warp][column][D / 4], see `at`
        constexpr int kQ = D / 32;                                 // float4s of one lane's dims
        auto at = [&](int wp, int col, int rr, int i) {            // spread over the banks
            return (wp * kMC + col) * (D / 4) + rr * kQ + (i ^ ((col >> 1) & (kQ - 1)) ^ (rr & (kQ - 1)));
        };
#pragma unroll 1
        for (int pass = 0; pass < kCols / kMC; ++pass) {
            const int live = min(kMC, ncols - kMC * pass);
            if (live <= 0) break;
            if (pass > 0) named_bar_sync(1, kI4Attend);  // the previous columns have been read
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float l0 = l_run[nt][0], l1 = l_run[nt][1];
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) {
                    l0 += __shfl_xor_sync(0xffffffffu, l0, x);
                    l1 += __shfl_xor_sync(0xffffffffu, l1, x);
                }
                const int col = 8 * nt + 2 * c - kMC * pass;
                if (col < 0 || col >= live) continue;  // (an odd last column brings a spare one)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < kQ; ++i)
                        sm_o[at(warp, col + x, r, i)] = make_float4(o[nt][2 * i][x], o[nt][2 * i][2 + x],
                                                                    o[nt][2 * i + 1][x], o[nt][2 * i + 1][2 + x]);
                if (r == 0) {
                    // the weights are relative to m - kI4Bias
                    s_m[warp * kMC + col] = m_run[nt][0] - kI4Bias;
                    s_m[warp * kMC + col + 1] = m_run[nt][1] - kI4Bias;
                    s_l[warp * kMC + col] = l0;
                    s_l[warp * kMC + col + 1] = l1;
                }
            }
            named_bar_sync(1, kI4Attend);
            for (int idx = tid; idx < live * (D / 4); idx += kI4Attend) {
                const int col = idx / (D / 4), d4 = idx % (D / 4);
                float M = s_m[col];
#pragma unroll
                for (int wp = 1; wp < kI4Warps; ++wp) M = fmaxf(M, s_m[wp * kMC + col]);
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                float den = 0.f;
#pragma unroll
                for (int wp = 0; wp < kI4Warps; ++wp) {
                    const float lw = s_l[wp * kMC + col];
                    const float f = lw == 0.f ? 0.f : ex2(s_m[wp * kMC + col] - M);  // 0: saw no key
                    const float4 v = sm_o[at(wp, col, d4 / kQ, d4 % kQ)];
                    num.x += f * v.x;
                    num.y += f * v.y;
                    num.z += f * v.z;
                    num.w += f * v.w;
                    den += f * lw;
                }
                const float inv = den != 0.f ? p.v_mul / den : 0.f;  // den NaN: NaN
                const int gc = col0 + kMC * pass + col, tq = T == 1 ? 0 : gc / p.g;
                const int hq = h * p.g + (gc - tq * p.g);
                const size_t orow = out_row(p, q0, tq, hq);
                const float4 v = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
                const float lse2 = den != 0.f ? M + log2f(den) : -INFINITY;
                if (nsplit == 1) {
                    store_out4(p.out, orow * D + 4 * d4, v, p.out_type);
                    if (p.lse && d4 == 0) p.lse[orow] = lse2 * kLn2;
                } else {
                    const size_t slot = ws_row(p, b, tq, hq) * p.max_splits + split;
                    reinterpret_cast<float4 *>(p.ws_o)[slot * (D / 4) + d4] = v;
                    if (d4 == 0) p.ws_lse[slot] = lse2;
                }
            }
        }
        // the description and the queries may be replaced
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_qempty[buf]);
        if (nsplit == 1 || !p.counters) continue;
        int *counter = p.counters + ((size_t)b * p.col_groups + col0 / kCols) * p.hkv + h;
        if (nsplit > kFuseMaxSplits) {  // for merge_i4_kernel
            if (split == 0 && tid == 0) *counter = nsplit;
            continue;
        }
        // ---- the last piece to finish merges them all
        named_bar_sync(1, kI4Attend);  // every thread's part is written
        if (tid == 0) s_last = count_arrival(counter) == nsplit - 1;
        named_bar_sync(1, kI4Attend);
        if (!s_last) continue;
        for (int idx = tid; idx < ncols * (D / 4); idx += kI4Attend) {
            const int col = idx / (D / 4), d4 = idx % (D / 4);
            const int gc = col0 + col, tq = T == 1 ? 0 : gc / p.g;
            const int hq = h * p.g + (gc - tq * p.g);
            const size_t orow = out_row(p, q0, tq, hq), wrow = ws_row(p, b, tq, hq) * p.max_splits;
            const float *ls = p.ws_lse + wrow;
            const float4 *src = reinterpret_cast<const float4 *>(p.ws_o) + wrow * (D / 4) + d4;
            // a running maximum over the pieces, kAhead loads at a time
            constexpr int kAhead = 4;
            float M = -INFINITY, den = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < nsplit; s += kAhead) {
                float x[kAhead];
                float4 v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int sk = min(s + k, nsplit - 1);
                    x[k] = __ldcg(ls + sk);
                    v[k] = __ldcg(src + (size_t)sk * (D / 4));
                }
                float top = M;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) top = fmaxf(top, x[k]);
                if (top != -INFINITY) {
                    const float a = ex2(M - top);  // of nothing: 0
                    acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a, den *= a;
                }
                M = top;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float e = s + k >= nsplit || x[k] == -INFINITY ? 0.f : ex2(x[k] - M);  // NaN stays
                    acc.x += e * v[k].x;
                    acc.y += e * v[k].y;
                    acc.z += e * v[k].z;
                    acc.w += e * v[k].w;
                    den += e;
                }
            }
            const float inv = den != 0.f ? 1.f / den : 0.f;
            store_out4(p.out, orow * D + 4 * d4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.out_type);
            if (p.lse && d4 == 0) p.lse[orow] = den != 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
        }
        if (tid == 0) *counter = 0;  // ready for the next call
    }
}

// Merge of rows cut into more partitions than one CTA merges: one CTA per query
// row, its threads in groups of D / 4 that take every group-th partition.  Bound by the
// latency of its loads from L2: the splits of a row are 33 to a few hundred.
template <int D>
__global__ void __launch_bounds__(kI4MergeThreads) merge_i4_kernel(const I4Params p) {
    constexpr int kLanes = D / 4, kGroups = kI4MergeThreads / kLanes;
    const int tq = blockIdx.x / p.hq, hq = blockIdx.x % p.hq;
    const I4Work w = i4_sequence(p, blockIdx.y, kI4Round, p.cols, false);
    if (!w.pairs || tq >= w.T) return;
    const int gc = tq * p.g + hq % p.g;  // its column
    int nsplit;
    if (p.counters) {  // what the pair's first piece left, if it is for this kernel
        // Each row of the pair takes it with an arrival in the upper half; the last
        // leaves the counter at 0.
        int *counter = p.counters + ((size_t)w.b * p.col_groups + gc / p.cols) * p.hkv + hq / p.g;
        __shared__ int s_n;
        if (threadIdx.x == 0) {
            s_n = 0;
            if (*counter) {
                const unsigned x = (unsigned)atomicAdd(counter, 1 << 16);
                s_n = (int)(x & 0xffffu);
                if ((int)(x >> 16) == min(p.cols, w.T * p.g - gc / p.cols * p.cols) - 1) *counter = 0;
            }
        }
        __syncthreads();
        nsplit = s_n;
    } else {
        nsplit = (w.rounds + p.part_rounds - 1) / p.part_rounds;
    }
    if (nsplit < 2) return;
    const int tid = threadIdx.x, d4 = tid % kLanes, grp = tid / kLanes;
    const size_t orow = out_row(p, w.q0, tq, hq), wrow = ws_row(p, w.b, tq, hq);
    const float *ls = p.ws_lse + wrow * p.max_splits;
    __shared__ float s_red[kI4MergeThreads / 32];
    __shared__ float4 s_acc[kI4MergeThreads];
    __shared__ float s_den[kGroups];
    float M = -INFINITY;
    for (int s = tid; s < nsplit; s += kI4MergeThreads) M = fmaxf(M, ls[s]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    if ((tid & 31) == 0) s_red[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kI4MergeThreads / 32; ++i) M = fmaxf(M, s_red[i]);
    const float4 *src = reinterpret_cast<const float4 *>(p.ws_o) + wrow * p.max_splits * kLanes + d4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll 4
    for (int s = grp; s < nsplit; s += kGroups) {
        const float x = ls[s], e = x == -INFINITY ? 0.f : ex2(x - M);
        const float4 v = src[(size_t)s * kLanes];
        acc.x += e * v.x;
        acc.y += e * v.y;
        acc.z += e * v.z;
        acc.w += e * v.w;
        den += e;
    }
    s_acc[tid] = acc;
    if (d4 == 0) s_den[grp] = den;
    __syncthreads();
    if (grp) return;
    den = s_den[0];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 v = s_acc[i * kLanes + d4];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        den += s_den[i];
    }
    const float inv = den != 0.f ? 1.f / den : 0.f;
    store_out4(p.out, orow * D + 4 * d4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.out_type);
    if (p.lse && d4 == 0) p.lse[orow] = den != 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

// The split plan of an explicit num_splits: as split_plan, without the longest partition
// that the 16-bit kernels' table slice in shared memory allows (this kernel reads the table
// as it goes), so that 1 means whole sequences however wide the table is.  Never more
// partitions than split_plan's, whose workspace serves.  Under a table of 8192 columns, with
// that limit / without: 256 sequences of 1 to 64 tokens (8 kv heads of 4) 31.3 / 29.1 us, 500
// of 1 to 508 (2 of 3) 26.9 / 25.8.
static void i4_split_plan(int batch, int num_kv_heads, int max_blocks, int num_splits, int *part_blocks,
                          int *max_splits) {
    if (num_splits <= 0 || max_blocks <= 0) {
        split_plan(batch, num_kv_heads, max_blocks, num_splits, part_blocks, max_splits);
        return;
    }
    const long long pb = ((long long)max_blocks + num_splits - 1) / num_splits;
    *part_blocks = (int)std::min<long long>((pb + 3) / 4 * 4, INT32_MAX);
    *max_splits = (int)(((long long)max_blocks + *part_blocks - 1) / *part_blocks);
}

cudaError_t set_wait_limit_decode_i4(unsigned long long ns) { return set_wait_limit_here(ns); }

template <int D, int NT, int NST, int MINB>
static kv_status launch_i4(I4Params &p, int part_blocks, cudaStream_t s) {
    const bool exact = p.out_type == KV_F32, tw = test_waits_enabled();
    auto fn = exact ? (tw ? decode_i4_kernel<D, NT, true, true, NST, MINB>
                          : decode_i4_kernel<D, NT, true, false, NST, MINB>)
                    : (tw ? decode_i4_kernel<D, NT, false, true, NST, MINB>
                          : decode_i4_kernel<D, NT, false, false, NST, MINB>);
    constexpr size_t smem = i4_smem_bytes<D, NT, NST>();
    if (kv_status st = cuda_status(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
        return st;
    p.cols = 8 * NT;
    p.part_rounds = (part_blocks + kI4Round - 1) / kI4Round;
    const long long pairs = (long long)p.batch * p.col_groups * p.hkv;
    const long long units = pairs * (p.max_blocks / kI4Round + 1 + i4_pair_cost(NT));
    const long long wave = (long long)MINB * sm_count();
    p.uncut = p.max_splits == 1 && pairs > kI4UncutPairs * wave;
    p.balanced = ((p.max_splits > 1 && p.counters) || p.uncut) && p.batch <= kI4ScanBatch && units < (1 << 30);
    p.uncut = p.uncut && p.balanced;
    const int rows = p.batch * p.col_groups, slabs = (rows + kI4MaxRows - 1) / kI4MaxRows;
    dim3 grid(p.max_splits * slabs, p.hkv, std::min(rows, kI4MaxRows));
    if (p.balanced) grid = dim3((unsigned)std::min(wave, units));
    fn<<<grid, kI4Threads, smem, s>>>(p);
    return cuda_status(cudaGetLastError());
}

// Tiles of eight columns of a pair and pairs of one (sequence, kv head) for its columns.
static void i4_columns(int cols, int *nt, int *groups) {
    *nt = cols <= 24 ? std::max(1, (cols + 7) / 8) : 2;  // more: groups of 16 (a fourth tile of eight does not fit)
    *groups = (cols + 8 * *nt - 1) / (8 * *nt);
}

kv_status attend_i4_limits(int batch, int num_kv_heads, int cols, int max_blocks, int max_splits) {
    int nt, groups;
    i4_columns(cols, &nt, &groups);
    // the merge's grid; a count of pieces in 16 bits; keys; the grid of CTAs per partition
    if (batch > 65535 || max_splits > 65535 || num_kv_heads > 65535 || max_blocks > INT32_MAX / kI4BS ||
        (long long)batch * groups > INT32_MAX / max_splits)
        return KV_ERR_UNSUPPORTED;
    return KV_OK;
}

kv_status attend_i4(const I4Call &a) {
    kv_pool *pool = a.pool;
    const int g = a.num_q_heads / pool->num_kv_heads;
    int pb = 0, ms = 0;
    i4_split_plan(a.batch, pool->num_kv_heads, a.max_blocks, a.num_splits, &pb, &ms);
    const long long rows = (long long)a.batch * a.max_q_len;
    if (rows > INT32_MAX) return KV_ERR_UNSUPPORTED;
    const size_t need = decode_workspace_bytes((int)rows, a.num_q_heads, pool->head_dim, ms);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need)) return KV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(a.workspace) & 15) return KV_ERR_ARG;
    const int cols = a.max_q_len * g;  // of one (sequence, kv head)
    int nt, groups;
    i4_columns(cols, &nt, &groups);
    if (kv_status st = attend_i4_limits(a.batch, pool->num_kv_heads, cols, a.max_blocks, ms)) return st;
    I4Params p{};
    p.q = static_cast<const uint16_t *>(a.q);
    p.q_bf16 = a.q_dtype == KV_BF16;
    p.cu_q = a.cu_q;
    p.total_q = a.total_q;
    p.max_t = a.max_q_len;
    p.pool = static_cast<const char *>(pool->k);
    p.tables = a.block_tables;
    p.max_blocks = a.max_blocks;
    p.num_blocks = pool->num_blocks;
    p.seq_lens = a.seq_lens;
    p.seq_order = a.seq_order;
    p.batch = a.batch;
    p.hq = a.num_q_heads;
    p.hkv = pool->num_kv_heads;
    p.g = g;
    p.scale_log2 = a.scale * 1.4426950408889634f * i4::kScaleUnit * pool->k_scale;
    p.v_mul = i4::kScaleUnit * pool->v_scale;
    p.max_splits = ms;
    p.col_groups = groups;
    p.out = a.out;
    p.out_type = a.out_dtype;
    p.lse = a.lse;
    p.ws_o = static_cast<float *>(a.workspace);
    p.ws_lse = p.ws_o ? p.ws_o + (size_t)rows * a.num_q_heads * ms * pool->head_dim : nullptr;
    const bool counted = (long long)a.batch * groups * pool->num_kv_heads <= kv_pool::kCounterSlots;
    p.counters = counted ? pool->counters : nullptr;
    p.err = pool->err;
    kv_status st;
    if (pool->head_dim == 64)
        st = nt == 1 ? launch_i4<64, 1, 4, 2>(p, pb, a.stream) : KV_ERR_UNSUPPORTED;
    else
        st = nt == 1   ? launch_i4<128, 1, 3, 2>(p, pb, a.stream)
             : nt == 2 ? launch_i4<128, 2, 3, 1>(p, pb, a.stream)
                       : launch_i4<128, 3, 3, 1>(p, pb, a.stream);
    if (st != KV_OK || ms < (counted ? kFuseMaxSplits + 1 : 2)) return st;
    const dim3 mgrid(a.num_q_heads * a.max_q_len, a.batch);
    if (pool->head_dim == 64)
        merge_i4_kernel<64><<<mgrid, kI4MergeThreads, 0, a.stream>>>(p);
    else
        merge_i4_kernel<128><<<mgrid, kI4MergeThreads, 0, a.stream>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_decode_plan_i4(const int32_t *host_seq_lens, int batch, int num_kv_heads, int max_blocks,
                            int *num_splits) {
    if (!num_splits || batch < 0 || num_kv_heads <= 0 || max_blocks < 0 || (batch > 0 && !host_seq_lens))
        return KV_ERR_ARG;
    *num_splits = 1;
    if (batch == 0 || max_blocks == 0) return KV_OK;
    // The pieces that the longest pair is cut into by equal runs of one wave (the
    // kernel's own arithmetic: rounds of 14 blocks, two CTAs per SM).
    long long units = 0, most = 1;
    for (int b = 0; b < batch; ++b) {
        const long long L = std::min<long long>(std::max(host_seq_lens[b], 0), (long long)max_blocks * kI4BS);
        const long long n = std::max<long long>(1, (L + kI4Round * kI4BS - 1) / (kI4Round * kI4BS));
        units += num_kv_heads * (n + i4_pair_cost(1));
        most = std::max(most, n);
    }
    const long long wave = 2LL * sm_count(), run = std::max<long long>(kI4MinRun, (units + wave - 1) / wave);
    // Short pairs stay whole: cutting them costs a merge each and shortens little.  Cut /
    // whole: 211 pairs of 83 to 1204 tokens 15.8 / 12.5 us, 500 of 1 to 508 17.2 / 15.2;
    // but 512 of 512 to 4096 43.7 / 44.0.
    if (most < 2 || (most <= kI4ShortPair && most <= run + 3)) return KV_OK;
    const long long pieces = (most - 2) / run + 2;
    // i4_split_plan's partitions are whole multiples of four blocks: the split count that
    // gives at least as many
    for (int s = (int)std::min<long long>(pieces, max_blocks);; ++s) {
        int pb, ms;
        i4_split_plan(batch, num_kv_heads, max_blocks, s, &pb, &ms);
        *num_splits = s;
        if (ms >= pieces || pb <= 4 || s >= max_blocks) break;
    }
    return KV_OK;
}

kv_status paged_decode_attention_i4(kv_pool_t p, const void *q, kv_dtype q_dtype, const int32_t *block_tables,
                                    int max_blocks, const int32_t *seq_lens, const int32_t *seq_order, int batch,
                                    int num_q_heads, float scale, void *out, kv_dtype out_dtype, float *lse_out,
                                    int num_splits, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p || batch < 0 || num_q_heads <= 0 || max_blocks < 0 || num_splits < 0) return KV_ERR_ARG;
    if (p->dtype != KV_I4 || (q_dtype != KV_BF16 && q_dtype != KV_F16) ||
        (out_dtype != KV_F32 && out_dtype != q_dtype))
        return KV_ERR_UNSUPPORTED;
    if (num_q_heads % p->num_kv_heads) return KV_ERR_ARG;
    if (num_q_heads / p->num_kv_heads > 8) return KV_ERR_UNSUPPORTED;
    if (kv_status st = require_device(p->device)) return st;
    if (batch == 0) return KV_OK;
    if (!q || !seq_lens || !out || (max_blocks > 0 && !block_tables)) return KV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return KV_ERR_ARG;
    I4Call a{};
    a.pool = p;
    a.q = q;
    a.q_dtype = q_dtype;
    a.max_q_len = 1;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.seq_order = seq_order;
    a.batch = batch;
    a.num_q_heads = num_q_heads;
    a.scale = scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse_out;
    a.num_splits = num_splits;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    a.stream = as_stream(stream);
    return attend_i4(a);
}

}  // extern "C"
