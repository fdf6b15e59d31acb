// Chunked causal prefill over a 4-bit pool.
//
// Every query tile of every head of a group reads the same K and V tiles, so a
// chunk of hundreds of query tokens would turn each code into an operand many
// times over inside the attention kernel, whose softmax warps are already what
// bounds it.  Here the batch's blocks are expanded once, to 16-bit tiles in the
// workspace laid out as a 16-bit pool's, and the tcgen05 prefill runs over them: K in
// q's type, V in fp16 (no conversion in its inner loop).  For 4 chunks of 2048
// tokens over 8192 cached ones (8 kv heads of 7, bf16) the expansion moves 47 MB in and
// 168 MB out in 35 us of the call's 1471: the products run at 1472 TFLOP/s (0.77 of a
// large bf16 matrix product), bound as in the 16-bit prefill by the softmax between the
// tensor core's two products (its pipe is busy for 65% of the time).
//
// The weights enter the second product as one fp16 number each for every output type (the
// tensor core takes 16-bit operands, and a second part would be a third product; error
// against 64 bits over mixed fp16 chunks 2.62e-4, of 24-bit weights 2.06e-4); few query
// tokens, by the decode kernel, keep two parts for fp32 output.
//
// c s / 256 is stored (exact in both types, see i4.cuh); the softmax scale and the
// output take the factor back, with the pool's scales.
//
// A chunk of few query tokens reads the cache about once, so it takes the 4-bit
// decode kernel with a column per (query token, head) instead.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "i4.cuh"
#include "i4_attend.h"
#include "internal.h"

namespace pkv {

constexpr int kExD = 128;            // head dim of the tcgen05 prefill
constexpr int kExTile = 9 * kExD;    // bytes of a 4-bit tile
constexpr int kExOut = 16 * kExD * 2;  // of an expanded one

// Whether the decode kernel with a column per (query token, head) runs instead.  It
// turns the cache's codes into operands once per 16 columns and cuts each sequence
// over the whole GPU; the expanding path does so once, writes and reads 16-bit tiles,
// and has a CTA per (kv head, 256 rows).  So few columns go by columns, and up to 96 while
// the pairs of sequence and kv head leave the expanding path's CTAs badly spread.
// Measured, columns / expanding, us: 16 pairs of 500 to 2000 tokens 20 / 23 at 96
// columns; 64 of 2000 39 / 58 at 64, 57 / 58 at 96; 128 of 1000 to 8000 113 / 155 at 64,
// 166 / 155 at 96, of 500 31 / 23 at 48; 192 of 300 to 3000 68 / 102 at 48, 131 / 103 at 96;
// 256 of 300 to 3000 64 / 102 at 32, 92 / 99 at 48, 118 / 100 at 64; 512 of 200 to 1500
// 88 / 111 at 32, 127 / 113 at 48.
static bool few_columns(int batch, int hkv, int max_q_len, int g) {
    const long long columns = (long long)max_q_len * g;
    return columns <= 32 || (columns <= 96 && columns * batch * hkv <= 80LL * sm_count());
}

template <bool BF16>
KV_DEVICE uint32_t to_k_type(uint32_t h2) {
    if constexpr (!BF16) return h2;
    const float2 f = f16x2_to_float2(h2);
    return float2_to_bf16x2(f.x, f.y);  // exact
}

// ---- The prefill's list of items, made by one CTA of the expanding kernel.
//
// A CTA takes one kv head of one item: 256 rows (query tokens x heads) and their keys,
// or, where whole query tiles would leave SMs idle, a piece of these keys.  A query tile
// of n key tiles counts n + kItemCost units (its prologue and end), so W units in all
// are an even share of W / SMs.  If the longest tile passes that by enough to pay for
// partial results (kWorth), tiles are cut into pieces of at most kPiece of a share.  Items
// go out most keys first.
// Measured, whole call, uncut / cut: one chunk of 512 after 8192 tokens, 8 kv heads of 4
// query heads, 125 / 89 us; 128 after 30000, one kv head of 8, 374 / 70; 9 chunks of 40
// to 117 after 240 to 16000, 4 of 4, 227 / 69.  Where the longest tile is near an even
// share cutting loses: 6 chunks of 33 to 700 after up to 3001 tokens, 8 of 4 (24 key
// tiles, share 22) 63 / 75 us; 4 of 256 after 4096 (34, share 30) 79 / 108.  Pieces of
// 1/2, 3/4 and 1 share: 106, 89, 104 us, 70, 70, 67 and 89, 69, 71 in the first three.
struct ListParams {
    const int32_t *cu_q, *seq_lens;
    int batch, total_q, max_q_len, max_blocks;
    int span, hkv, sms;    // query tokens of an item
    int max_items, max_slots;
    PrefillItem *items;
    PrefillCounts *counts;
    int *cuts;
    int *err;
};
constexpr int kItemCost = 2, kMinPiece = 4;   // key tiles
constexpr int kPieceNum = 3, kPieceDen = 4;
constexpr int kWorthNum = 9, kWorthDen = 8, kWorthMore = 3;
constexpr int kListThreads = 256, kListWarps = kListThreads / 32;
constexpr int kListSeqs = kListThreads;       // sequences that are put in order at once

// At most this many pieces beyond one per query tile: less than n / t for a tile, t the
// longest piece, with t + kItemCost >= kPiece W / SMs and W >= hkv (sum of n).
static long long extra_pieces(int hkv, int sms) {
    return (long long)sms * kPieceDen * (kMinPiece + kItemCost) / ((long long)hkv * kPieceNum * kMinPiece) + 1;
}

KV_DEVICE int warp_sum(int v) {
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) v += __shfl_xor_sync(0xffffffffu, v, y);
    return v;
}
KV_DEVICE int warp_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, y);
        if (lane >= y) v += u;
    }
    return v;
}

KV_DEVICE void list_items(const ListParams &p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ unsigned long long s_units;
    __shared__ int s_most;
    // of the sequences at hand: query tokens (0: left out) and keys; by rank: which, and
    // where its items, slots and cuts begin
    __shared__ int s_T[kListSeqs], s_len[kListSeqs], s_seq[kListSeqs], s_first[3][kListSeqs];
    __shared__ int s_scan[3][kListWarps];
    auto load = [&](int base) {
        int T = 0, len = 0;
        if (base + tid < p.batch) {
            const int first = p.cu_q[base + tid];
            T = p.cu_q[base + tid + 1] - first;
            len = p.seq_lens[base + tid];
            if (T < 0) T = 0;
            if (T > 0 && (len < T || len > 16LL * p.max_blocks || T > p.max_q_len || first < 0 ||
                          (long long)first + T > p.total_q)) {
                atomicOr(p.err, KV_DEVERR_BLOCK_RANGE);
                T = 0;
            }
        }
        s_T[tid] = T;
        s_len[tid] = len;
    };
    auto key_tiles = [&](int qt, int T, int len) {
        return (int)((len - T + min((long long)(qt + 1) * p.span, (long long)T) + 127) >> 7);
    };
    if (tid == 0) s_units = 0, s_most = 0;
    // ---- W and the longest tile
    for (int base = 0; base < p.batch; base += kListSeqs) {
        __syncthreads();
        load(base);
        __syncthreads();
        if (!p.max_slots) continue;  // nothing will be cut
        for (int i = warp; i < min(kListSeqs, p.batch - base); i += kListWarps) {
            const int T = s_T[i], len = s_len[i], tiles = (T + p.span - 1) / p.span;
            long long units = 0;
            for (int qt = lane; qt < tiles; qt += 32) units += key_tiles(qt, T, len) + kItemCost;
            if (units) atomicAdd(&s_units, (unsigned long long)units);
            if (lane == 0 && T) atomicMax(&s_most, (int)((len + 127LL) >> 7));
        }
    }
    __syncthreads();
    const unsigned long long all = s_units * p.hkv;
    int longest = INT32_MAX;
    if (p.max_slots && (unsigned long long)(s_most + kItemCost - kWorthMore) * kWorthDen * p.sms > all * kWorthNum &&
        s_most + kItemCost > kWorthMore)
        longest = (int)max((long long)kMinPiece,
                           (long long)min(all * kPieceNum / ((unsigned long long)p.sms * kPieceDen), 1ull << 30) + 1 - kItemCost);
    auto pieces = [&](int n) { return (int)(((long long)n + longest - 1) / longest); };
    // ---- the lists
    int before[3] = {0, 0, 0};  // items, slots, cuts of the sequences done
    for (int base = 0; base < p.batch; base += kListSeqs) {
        const int nb = min(kListSeqs, p.batch - base);
        if (p.batch > kListSeqs) {
            __syncthreads();
            load(base);
        }
        s_first[0][tid] = s_first[1][tid] = s_first[2][tid] = 0;
        __syncthreads();
        for (int i = warp; i < nb; i += kListWarps) {
            const int T = s_T[i], mine = s_len[i], tiles = (T + p.span - 1) / p.span;
            int rank = 0, items = 0, slots = 0, cuts = 0;
            for (int o = lane; o < nb; o += 32) rank += s_len[o] > mine || (s_len[o] == mine && o < i);
            for (int qt = lane; qt < tiles; qt += 32) {
                const int k = pieces(key_tiles(qt, T, mine));
                items += k;
                slots += k > 1 ? k : 0;
                cuts += k > 1;
            }
            rank = warp_sum(rank);
            items = warp_sum(items);
            slots = warp_sum(slots);
            cuts = warp_sum(cuts);
            if (lane == 0) s_seq[rank] = i, s_first[0][rank] = items, s_first[1][rank] = slots, s_first[2][rank] = cuts;
        }
        __syncthreads();
        int mine[3], to[3];
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            mine[z] = s_first[z][tid];
            to[z] = warp_scan(mine[z], lane);
            if (lane == 31) s_scan[z][warp] = to[z];
        }
        __syncthreads();
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            int at = before[z] + to[z] - mine[z];
#pragma unroll
            for (int y = 0; y < kListWarps; ++y) {
                if (y < warp) at += s_scan[z][y];
                before[z] += s_scan[z][y];
            }
            s_first[z][tid] = at;
        }
        __syncthreads();
        for (int i = warp; i < nb; i += kListWarps) {
            const int T = s_T[s_seq[i]], len = s_len[s_seq[i]], tiles = (T + p.span - 1) / p.span;
            int item = s_first[0][i], slot = s_first[1][i], cut = s_first[2][i];
            for (int last = tiles - 1; last >= 0; last -= 32) {  // the last tiles have most keys
                const int qt = last - lane;
                const int n = qt >= 0 ? key_tiles(qt, T, len) : 0, k = qt >= 0 ? pieces(n) : 0;
                const int held = k > 1 ? k : 0;
                const int items_to = warp_scan(k, lane), slots_to = warp_scan(held, lane), cuts_to = warp_scan(k > 1, lane);
                const int at = item + items_to - k, slot0 = slot + slots_to - held, cut_at = cut + cuts_to - (k > 1);
                // Query offsets that overlap could ask for more than there is room for: items
                // past it are dropped, tiles without slots come whole, k times.
                const bool room = slot0 + held <= p.max_slots;
                for (int y = 0; y < k && at + y < p.max_items; ++y)
                    p.items[at + y] =
                        room ? PrefillItem{base + s_seq[i], qt, (int)((long long)n * y / k), (int)((long long)n * (y + 1) / k),
                                           y, k, slot0, 0}
                             : PrefillItem{base + s_seq[i], qt, 0, n, 0, 1, 0, 0};
                if (k > 1 && cut_at < p.max_slots / 2) p.cuts[cut_at] = min(at, p.max_items - 1);
                item += __shfl_sync(0xffffffffu, items_to, 31);
                slot += __shfl_sync(0xffffffffu, slots_to, 31);
                cut += __shfl_sync(0xffffffffu, cuts_to, 31);
            }
        }
    }
    if (tid == 0) *p.counts = PrefillCounts{min(before[0], p.max_items), min(before[2], p.max_slots / 2)};
}

// One warp expands the K and V tiles of one (sequence, block, kv head) and writes
// the block's entry of the expanded tiles' table; the grid's first CTA makes the
// prefill's list.  Bound by memory (above: 6100 GB/s, some of the writes left in L2).
template <bool BF16>
__global__ void __launch_bounds__(256, 6) expand_i4_kernel(const char *__restrict__ k_pool,
                                                        const char *__restrict__ v_pool,
                                                        const int32_t *__restrict__ tables,
                                                        const int32_t *__restrict__ seq_lens, int max_blocks,
                                                        int num_blocks, int hkv, int32_t *__restrict__ new_table,
                                                        char *__restrict__ k_out, char *__restrict__ v_out,
                                                        const ListParams list) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the prefill waits for this grid's end
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0 && blockIdx.z == 0) list_items(list);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = blockIdx.y, i = (blockIdx.x - 1) * 8 + (threadIdx.x >> 5);
    const long long L = seq_lens[b];
    if (i >= max_blocks || 16LL * i >= L) return;
    const size_t at = (size_t)b * max_blocks + i;
    const int id = __ldg(tables + at);
    const bool ok = id >= 0 && id < num_blocks;
    if (h == 0 && lane == 0) new_table[at] = ok ? (int32_t)at : -1;
    if (!ok) return;  // the prefill reports it and leaves its keys out
    const size_t tile = ((size_t)id * hkv + h) * 2 * kExTile;
    const char *kt = k_pool + tile, *vt = v_pool + tile;
    uint4 *ko = reinterpret_cast<uint4 *>(k_out + (at * hkv + h) * kExOut);
    uint2 *vo = reinterpret_cast<uint2 *>(v_out + (at * hkv + h) * kExOut);
    // word 32 j + lane: K row 2 j + lane / 16, octet lane % 16; V pair j, the word
    // of quad lane
    uint32_t kw[8], vw[8];
    uint32_t ks[8], vs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        kw[j] = __ldg(reinterpret_cast<const uint32_t *>(kt) + 32 * j + lane);
        vw[j] = __ldg(reinterpret_cast<const uint32_t *>(vt) + 32 * j + (lane ^ i4::v_swizzle<kExD>(j)));
        ks[j] = __ldg(reinterpret_cast<const uint8_t *>(kt) + 8 * kExD + (2 * j + (lane >> 4)) * 8 + ((lane & 15) >> 1));
        vs[j] = __ldg(reinterpret_cast<const uint16_t *>(vt + 8 * kExD + j * 16) + (lane >> 2));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t x[4];
        i4::values8(kw[j], i4::make_scale(__low2half2(i4::scale_pair(ks[j]))), x);
        // (0, 4) (1, 5) (2, 6) (3, 7) -> (0, 1) (2, 3) (4, 5) (6, 7)
        ko[32 * j + lane] = make_uint4(to_k_type<BF16>(__byte_perm(x[0], x[1], 0x5410)),
                                       to_k_type<BF16>(__byte_perm(x[2], x[3], 0x5410)),
                                       to_k_type<BF16>(__byte_perm(x[0], x[1], 0x7632)),
                                       to_k_type<BF16>(__byte_perm(x[2], x[3], 0x7632)));
        i4::values8(vw[j], i4::make_scale(i4::scale_pair(vs[j])), x);
        vo[64 * j + lane] = make_uint2(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
        vo[64 * j + 32 + lane] = make_uint2(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
    }
}

// The expanding path's workspace: the lists' lengths, items, cuts, table, K tiles, V
// tiles, partial results.
struct ExpandLayout {
    long long max_items = 0, max_slots = 0, blocks = 0;
    size_t items, cuts, table, k_tiles, v_tiles, partial, bytes;
    ExpandLayout(int batch, int hkv, int g, int max_blocks, int max_q_len) {
        const int span = 2 * (128 / g), sms = sm_count();
        // a chunk is at most as long as its sequence (max_q_len may be any upper bound)
        const long long longest = std::min<long long>(max_q_len, std::max(16LL * max_blocks, 1LL));
        const long long tiles = batch * ((longest + span - 1) / span);
        const long long extra = extra_pieces(hkv, sms), most = (max_blocks + 7LL) / 8;  // key tiles of a sequence
        if (most > kMinPiece) max_slots = std::min(2 * extra, tiles * ((most + kMinPiece - 1) / kMinPiece));
        max_items = tiles + (max_slots ? extra : 0);
        // a tensor map has at least one row, so a table without columns takes a block
        blocks = (long long)batch * std::max(max_blocks, 1);
        auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
        items = sizeof(PrefillItem);
        cuts = items + (size_t)max_items * sizeof(PrefillItem);
        table = up(cuts + (size_t)(max_slots / 2) * sizeof(int));
        k_tiles = up(table + (size_t)blocks * sizeof(int32_t));
        v_tiles = k_tiles + (size_t)blocks * hkv * kExOut;
        partial = v_tiles + (size_t)blocks * hkv * kExOut;
        bytes = partial + (size_t)max_slots * hkv * kPrefillSlot * sizeof(float);
    }
};

}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_prefill_i4_workspace_size(kv_pool_t p, int batch, int num_q_heads, int max_blocks, int max_q_len,
                                       size_t *bytes) {
    if (!p || !bytes || batch < 0 || num_q_heads <= 0 || max_blocks < 0 || max_q_len < 0) return KV_ERR_ARG;
    if (p->dtype != KV_I4 || p->head_dim != kExD) return KV_ERR_UNSUPPORTED;
    if (num_q_heads % p->num_kv_heads) return KV_ERR_ARG;
    const int hkv = p->num_kv_heads, g = num_q_heads / hkv;
    // what the call refuses (it asks here too)
    if (g > 8 || batch > 65535 || hkv > 65535) return KV_ERR_UNSUPPORTED;
    if (few_columns(batch, hkv, max_q_len, g)) {
        int pb, ms;
        split_plan(batch, hkv, max_blocks, 0, &pb, &ms);
        if (kv_status st = attend_i4_limits(batch, hkv, max_q_len * g, max_blocks, ms)) return st;
        *bytes = decode_workspace_bytes(batch * max_q_len, num_q_heads, kExD, ms);
    } else {
        const ExpandLayout at(batch, hkv, g, max_blocks, max_q_len);
        if (at.blocks > INT32_MAX / 16 / hkv) return KV_ERR_UNSUPPORTED;  // a tensor map's rows; bounds the items too
        *bytes = at.bytes;
    }
    return KV_OK;
}

kv_status paged_prefill_attention_i4(kv_pool_t p, const void *q, kv_dtype q_dtype, const int32_t *cu_q, int total_q,
                                     int max_q_len, const int32_t *block_tables, int max_blocks,
                                     const int32_t *seq_lens, int batch, int num_q_heads, float scale, void *out,
                                     kv_dtype out_dtype, float *lse_out, void *workspace, size_t workspace_bytes,
                                     void *stream) {
    if (!p || batch < 0 || total_q < 0 || max_q_len < 0 || max_blocks < 0 || num_q_heads <= 0) return KV_ERR_ARG;
    if (p->dtype != KV_I4 || p->head_dim != kExD || (q_dtype != KV_BF16 && q_dtype != KV_F16) ||
        (out_dtype != KV_F32 && out_dtype != q_dtype))
        return KV_ERR_UNSUPPORTED;
    if (num_q_heads % p->num_kv_heads) return KV_ERR_ARG;
    if (num_q_heads / p->num_kv_heads > 8) return KV_ERR_UNSUPPORTED;
    if (kv_status st = require_device(p->device)) return st;
    if (batch == 0 || max_q_len == 0 || total_q == 0) return KV_OK;
    if (!q || !cu_q || !block_tables || !seq_lens || !out) return KV_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15)
        return KV_ERR_ARG;
    // what the kernels multiply scores by has to be a number above 0
    if (!(scale > 0.f) || !std::isfinite(scale * i4::kScaleUnit * p->k_scale * 1.4426950408889634f)) return KV_ERR_ARG;
    size_t need = 0;
    if (kv_status st = kv_prefill_i4_workspace_size(p, batch, num_q_heads, max_blocks, max_q_len, &need)) return st;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KV_ERR_ARG;
    if (few_columns(batch, p->num_kv_heads, max_q_len, num_q_heads / p->num_kv_heads)) {
        I4Call a{};
        a.pool = p;
        a.q = q;
        a.q_dtype = q_dtype;
        a.cu_q = cu_q;
        a.total_q = total_q;
        a.max_q_len = max_q_len;
        a.block_tables = block_tables;
        a.max_blocks = max_blocks;
        a.seq_lens = seq_lens;
        a.batch = batch;
        a.num_q_heads = num_q_heads;
        a.scale = scale;
        a.out = out;
        a.out_dtype = out_dtype;
        a.lse = lse_out;
        a.workspace = workspace;
        a.workspace_bytes = workspace_bytes;
        a.stream = as_stream(stream);
        return attend_i4(a);
    }
    const int hkv = p->num_kv_heads, g = num_q_heads / hkv, span = 2 * (128 / g);
    const ExpandLayout at(batch, hkv, g, max_blocks, max_q_len);
    // No more query tiles than the query tokens make, one begun tile a sequence.  With two
    // for every SM their keys stay whole (one, if all are of one sequence and so about
    // alike), and the launch that adds up pieces is spared: 2 us where it finds none.
    const long long tiles = (long long)total_q / span + batch;
    const bool cut = at.max_slots > 0 && tiles * hkv < (batch == 1 ? 1LL : 2LL) * sm_count();
    const long long max_items = std::min(at.max_items, tiles + (cut ? extra_pieces(hkv, sm_count()) : 0));
    const long long rows = at.blocks * hkv * 16;
    char *ws = static_cast<char *>(workspace);
    PrefillCounts *counts = reinterpret_cast<PrefillCounts *>(ws);
    int *cuts = reinterpret_cast<int *>(ws + at.cuts);
    PrefillItem *items = reinterpret_cast<PrefillItem *>(ws + at.items);
    int32_t *table = reinterpret_cast<int32_t *>(ws + at.table);
    CUtensorMap map_k, map_v;
    if (!encode_rows_map(&map_k, ws + at.k_tiles, rows) || !encode_rows_map(&map_v, ws + at.v_tiles, rows))
        return KV_ERR_CUDA;
    const ListParams list{cu_q, seq_lens, batch, total_q, max_q_len, max_blocks, span, hkv, sm_count(),
                          (int)max_items, cut ? (int)at.max_slots : 0, items, counts, cuts, p->err};
    const int columns = (max_blocks + 7) / 8;
    const dim3 grid(columns + 1, hkv, batch);  // the list's CTA is the first
    auto fn = q_dtype == KV_BF16 ? expand_i4_kernel<true> : expand_i4_kernel<false>;
    fn<<<grid, 256, 0, as_stream(stream)>>>((const char *)p->k, (const char *)p->v, block_tables, seq_lens, max_blocks,
                                            p->num_blocks, hkv, table, ws + at.k_tiles, ws + at.v_tiles, list);
    if (kv_status st = cuda_status(cudaGetLastError())) return st;
    PrefillCall a{};
    a.q = q;
    a.q_dtype = q_dtype;
    a.packed = true;
    a.items = items;
    a.counts = counts;
    a.cuts = cut ? cuts : nullptr;
    a.max_items = (int)max_items;
    a.partial = reinterpret_cast<float *>(ws + at.partial);
    a.map_k = &map_k;
    a.map_v = &map_v;
    a.cu_q = cu_q;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.block_tables = table;
    a.max_blocks = max_blocks;
    a.num_blocks = (int)at.blocks;
    a.num_kv_heads = hkv;
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.num_q_heads = num_q_heads;
    a.scale = scale * i4::kScaleUnit * p->k_scale;
    a.v_mul = i4::kScaleUnit * p->v_scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse_out;
    a.err = p->err;
    a.stream = as_stream(stream);
    return launch_prefill(a);
}

}  // extern "C"
