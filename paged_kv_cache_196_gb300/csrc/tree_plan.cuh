// How tree attention spreads a ragged batch over one wave of CTAs, from the lengths
// it finds on the device (a captured step stays balanced as its sequences grow).
//
// A sequence of L tokens and T nodes is kv heads x groups pairs: a group is as many
// whole nodes as the kernel takes query rows (all heads of a kv head, row = node *
// g + head within a row tile), so a pair is what one pass over the keys of a kv head serves.
// A pair counts pair_cost units (its queries and its end) and one per key tile of 128.  The
// units of all pairs are laid end to end, sequence by sequence, and cut into equal runs, one
// per CTA.  What a run holds of a pair is a piece: a range of its key tiles, empty where
// the run's end falls among the pair's first pair_cost units.
// A pair of more than one piece leaves partial results: a run that begins inside a pair
// has its piece of it in slot 2 run, the one that it begins and does not end in slot
// 2 run + 1.  Pairs whole, one CTA each, would take 133 us where runs take 114 (64 sequences of
// 512 to 4096 tokens, 8 kv heads), and 174 where they take 99.5 (16 of 1000 to 8000).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace tree {

constexpr int kTile = 128;  // keys
// Columns of a table: 2^31 - 128 tokens, so that the end of a last key tile is an int too.
constexpr int kMaxBlocks = (1 << 27) - 8;

struct Plan {
    const int32_t *cu_q, *seq_lens;
    int batch, total_q, max_q_len, max_blocks;
    int hkv, group_nodes;  // kv heads; nodes of a group
    int tile_nodes;        // of a row tile: row of the group = node / tile_nodes * 128 + node % tile_nodes * g + head
    int runs;              // CTAs
    int pair_cost;         // units
    int min_run;           // units of the shortest run
    int whole;             // a run takes the pairs that begin in it whole: none is cut
};

struct Seq {
    int q0, nodes, len, tiles, groups;
};

// What describes a sequence, as it lies in memory.
struct RawSeq {
    int q0, q1, len;
};
KV_DEVICE RawSeq load_raw(const Plan &p, int b) {
    return RawSeq{__ldg(p.cu_q + b), __ldg(p.cu_q + b + 1), __ldg(p.seq_lens + b)};
}

// A sequence; without nodes where there are none or what describes it is out of range.
KV_DEVICE Seq make_seq(const Plan &p, const RawSeq &raw, int *err) {
    const long long q0 = raw.q0, t = raw.q1 - q0, len = raw.len;
    Seq s{0, 0, 0, 0, 0};
    if (t == 0) return s;
    if (t < 0 || t > p.max_q_len || q0 < 0 || q0 + t > p.total_q || len < t || len > (long long)p.max_blocks * 16) {
        if (err) atomicOr(err, KV_DEVERR_BLOCK_RANGE);
        return s;
    }
    s.q0 = (int)q0;
    s.nodes = (int)t;
    s.len = (int)len;
    s.tiles = (int)((len + kTile - 1) / kTile);
    s.groups = (s.nodes + p.group_nodes - 1) / p.group_nodes;
    return s;
}

KV_DEVICE Seq load_seq(const Plan &p, int b, int *err) { return make_seq(p, load_raw(p, b), err); }

KV_DEVICE long long seq_units(const Plan &p, const Seq &s) {
    return s.nodes ? (long long)p.hkv * s.groups * (s.tiles + p.pair_cost) : 0;
}

// What a CTA knows after place(): units of a run, all units, and of the unit it asked for
// the sequence (batch: none), the pair of it and that pair's first unit.
struct Place {
    long long per, total, first;
    int b, pair;
    Seq seq;
};

template <int kThreads>
struct PlaceScratch {
    long long sums[kThreads / 32];
    Place at;
};

// All threads of the CTA: the place of unit run * per.
template <int kThreads>
KV_DEVICE Place place(const Plan &p, int run, PlaceScratch<kThreads> &s, int *err) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunk = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, tid * chunk), b1 = min(p.batch, b0 + chunk);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_units(p, load_seq(p, b, err));
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
    }
    if (lane == 31) s.sums[warp] = upto;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = total;
        total += s.sums[w];
    }
    upto += before;
    const long long per = max((long long)p.min_run, (total + p.runs - 1) / p.runs);
    const long long unit = run * per;
    if (tid == 0 && unit >= total) s.at = Place{per, total, total, p.batch, 0, {}};
    if (unit < upto && unit >= upto - mine) {
        long long base = upto - mine;
        for (int b = b0; b < b1; ++b) {
            const Seq q = load_seq(p, b, nullptr);
            const long long n = seq_units(p, q);
            if (unit < base + n) {
                const int cost = q.tiles + p.pair_cost, pair = (int)((unit - base) / cost);
                s.at = Place{per, total, base + (long long)pair * cost, b, pair, q};
                break;
            }
            base += n;
        }
    }
    __syncthreads();
    return s.at;
}

// A piece: key tiles t0 .. t1 - 1 of the pair of sequence b, kv head h and node group grp.
struct Piece {
    int b, h, grp, t0, t1;
    int slot;  // of its partial results; -1: the pair is whole
    Seq seq;
};

// The pieces of a run, in order.
struct Pieces {
    long long unit, end, first;  // first: of the pair
    int b, pair, run;
    Seq seq;
    RawSeq ahead;  // of sequence b + 1: looked at when it is reached, so that nothing waits for it before

    KV_DEVICE void start(const Plan &p, const Place &at, int r) {
        run = r;
        unit = r * at.per;
        end = min(at.total, unit + at.per);
        first = at.first;
        b = at.b;
        pair = at.pair;
        seq = at.seq;
        if (unit < end) load_ahead(p);
    }
    KV_DEVICE void load_ahead(const Plan &p) {
        ahead = RawSeq{0, 0, 0};
        if (b + 1 < p.batch) ahead = load_raw(p, b + 1);
    }
    KV_DEVICE bool next(const Plan &p, Piece &out) {
        while (unit < end) {
            if (pair == p.hkv * seq.groups) {  // (a sequence without nodes has no pairs)
                pair = 0;
                ++b;
                seq = make_seq(p, ahead, nullptr);
                load_ahead(p);
                continue;
            }
            const int cost = seq.tiles + p.pair_cost;
            const int from = (int)(unit - first);
            const int to = p.whole ? cost : (int)min(end - first, (long long)cost);
            const int now = pair++;
            first += cost;
            unit = first;
            if (p.whole && from > 0) continue;  // the run before has it
            out.t0 = max(0, from - p.pair_cost);
            out.t1 = max(0, to - p.pair_cost);
            if (out.t0 >= out.t1) continue;
            out.b = b;
            out.h = seq.groups == 1 ? now : now / seq.groups;
            out.grp = now - out.h * seq.groups;
            out.slot = out.t0 == 0 && out.t1 == seq.tiles ? -1 : 2 * run + (from > 0 ? 0 : 1);
            out.seq = seq;
            return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------- cut pairs
// What the kernel that adds up cut pairs has to know of the end of a run: the pair that lies
// across it.
struct Cut {
    int q0, node0, rows, h;  // rows of the group; 0: no pair is cut here
    int r0, r1, slot0, r;    // the runs that hold its first and last tile, r0's slot, the run that begins here
};

KV_DEVICE Cut cut_of(const Plan &p, const Place &at, int r, int g) {
    Cut c{0, 0, 0, 0, 0, 0, 0, r};
    if (at.b >= p.batch || p.whole) return c;
    const int cost = at.seq.tiles + p.pair_cost;
    c.r0 = (int)((at.first + p.pair_cost) / at.per);
    c.r1 = (int)((at.first + cost - 1) / at.per);
    if (r <= c.r0 || r > c.r1) return c;
    c.slot0 = 2 * c.r0 + (at.first < c.r0 * at.per ? 0 : 1);
    c.h = at.pair / at.seq.groups;
    c.node0 = (at.pair - c.h * at.seq.groups) * p.group_nodes;
    c.rows = min(p.group_nodes, at.seq.nodes - c.node0) * g;
    c.q0 = at.seq.q0;
    return c;
}

// ---------------------------------------------------------------- the tree
// Ancestors of the nodes, 32 of them a word.
constexpr int kMaxNodes = 256;

// The bits of node i and of every node above it into out[0 .. kMaxNodes / 32); a parent
// that does not come before its node ends the walk (it has at most T steps) and is
// reported.  parents: the tree's (shared memory or global), null: each node's is the one
// before it.
template <typename Set>
KV_DEVICE void walk_up(const int32_t *parents, int i, int *err, Set set) {
    while (true) {
        set(i);
        const int up = parents ? parents[i] : i - 1;
        if (up >= i || up < -1) {
            atomicOr(err, KV_DEVERR_TREE);
            return;
        }
        if (up < 0) return;
        i = up;
    }
}

// Bits of 32 keys from key on (a position relative to the tree's first token) that a row
// with these ancestors attends: all before the tree, none behind it (bits of nodes that
// are not there are zero).
KV_DEVICE uint32_t key_bits(const uint32_t *anc, int key) {
    if (key <= -32) return 0xffffffffu;
    if (key < 0) return (0xffffffffu >> (32 + key)) | (anc[0] << -key);
    const int w = key >> 5, s = key & 31;
    if (w >= kMaxNodes / 32) return 0u;
    const uint32_t hi = w + 1 < kMaxNodes / 32 ? anc[w + 1] : 0u;
    return __funnelshift_r(anc[w], hi, s);
}

}  // namespace tree
}  // namespace pkv
