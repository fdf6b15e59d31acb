// Chunked causal prefill over a 4-bit pool.
//
// Every query tile of every head of a group reads the same K and V tiles, so a
// chunk of hundreds of query tokens would turn each code into an operand many
// times over inside the attention kernel, whose softmax warps are already what
// bounds it.  Here the batch's blocks are expanded once, to 16-bit tiles in the
// workspace laid out as a 16-bit pool's, and the tcgen05 prefill runs over them: K in
// q's type, V in fp16 (no conversion in its inner loop).  For 4 chunks of 2048
// tokens over 8192 cached ones the expansion moves 47 MB in and 336 MB out.
//
// c s / 256 is stored (exact in both types, see i4.cuh); the softmax scale and the
// output take the factor back, with the pool's scales.
//
// A chunk of few query tokens reads the cache about once, so it takes the 4-bit
// decode kernel with a column per (query token, head) instead.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
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
// and has a CTA per (kv head, 256 rows).  Measured with 8 kv heads, 4 query heads each,
// columns against expanding: 16 sequences of 1000 to 8000 tokens 88 / 164 us at 48
// columns, 114 / 165 at 64, 167 / 165 at 96; 2 sequences of 500 to 2000 tokens 19 / 35 at
// 96; 64 sequences of 200 to 1500 tokens (512 pairs of sequence and kv head, several for
// every SM) 88 / 112 at 32, 127 / 112 at 48.
static bool few_columns(int batch, int hkv, int max_q_len, int g) {
    return (long long)max_q_len * g <= ((long long)batch * hkv < 2LL * sm_count() ? 96 : 32);
}

template <bool BF16>
KV_DEVICE uint32_t to_k_type(uint32_t h2) {
    if constexpr (!BF16) return h2;
    const float2 f = f16x2_to_float2(h2);
    return float2_to_bf16x2(f.x, f.y);  // exact
}

// Largest batch that is put in order; its work grows with the square.
constexpr int kOrderBatch = 1024;

// One warp expands the K and V tiles of one (sequence, block, kv head) and writes
// the block's entry of the expanded tiles' table.  The grid's last rows (blockIdx.x at
// `order_at`, first head) rank the sequences, most keys first: a prefill whose longest
// tiles start last ends with a few CTAs at work.
template <bool BF16>
__global__ void __launch_bounds__(256) expand_i4_kernel(const char *__restrict__ k_pool,
                                                        const char *__restrict__ v_pool,
                                                        const int32_t *__restrict__ tables,
                                                        const int32_t *__restrict__ seq_lens, int max_blocks,
                                                        int num_blocks, int hkv, int32_t *__restrict__ new_table,
                                                        char *__restrict__ k_out, char *__restrict__ v_out,
                                                        int32_t *__restrict__ order, int order_at) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the prefill waits for this grid's end
    if ((int)blockIdx.x == order_at) {
        if (blockIdx.y) return;
        const int mine = seq_lens[blockIdx.z];
        int before = 0;
        for (int o = threadIdx.x; o < (int)gridDim.z; o += blockDim.x) {
            const int L = seq_lens[o];
            before += L > mine || (L == mine && o < (int)blockIdx.z);
        }
        __shared__ int s_before;
        if (threadIdx.x == 0) s_before = 0;
        __syncthreads();
        atomicAdd(&s_before, before);
        __syncthreads();
        if (threadIdx.x == 0) order[s_before] = blockIdx.z;
        return;
    }
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long L = seq_lens[b];
    if (i >= max_blocks || 16LL * i >= L) return;
    const size_t at = (size_t)b * max_blocks + i;
    const int id = __ldg(tables + at);
    const bool ok = id >= 0 && id < num_blocks;
    if (h == 0 && lane == 0) new_table[at] = ok ? (int32_t)at : -1;
    if (!ok) return;  // the prefill reports it and reads zeros
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

// Workspace of the expanding path: order of the batch and table, K tiles, V tiles.
static size_t expand_table_bytes(int batch, int max_blocks) {
    return ((size_t)batch * (max_blocks + 1) * sizeof(int32_t) + 1023) / 1024 * 1024;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

kv_status kv_prefill_i4_workspace_size(kv_pool_t p, int batch, int num_q_heads, int max_blocks, int max_q_len,
                                       size_t *bytes) {
    if (!p || !bytes || batch < 0 || num_q_heads <= 0 || max_blocks < 0 || max_q_len < 0) return KV_ERR_ARG;
    if (p->dtype != KV_I4 || p->head_dim != kExD) return KV_ERR_UNSUPPORTED;
    if (num_q_heads % p->num_kv_heads) return KV_ERR_ARG;
    if (num_q_heads / p->num_kv_heads > 8 || batch > 65535) return KV_ERR_UNSUPPORTED;
    if (few_columns(batch, p->num_kv_heads, max_q_len, num_q_heads / p->num_kv_heads)) {
        int pb, ms;
        split_plan(batch, p->num_kv_heads, max_blocks, 0, &pb, &ms);
        *bytes = decode_workspace_bytes(batch * max_q_len, num_q_heads, kExD, ms);
    } else {
        // a tensor map has at least one row, so a table without columns takes a block
        *bytes = expand_table_bytes(batch, max_blocks) +
                 2 * (size_t)batch * std::max(max_blocks, 1) * p->num_kv_heads * kExOut;
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
    if (batch > 65535) return KV_ERR_UNSUPPORTED;
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
    const long long blocks = (long long)batch * std::max(max_blocks, 1), rows = blocks * p->num_kv_heads * 16;
    if (rows > INT32_MAX || p->num_kv_heads > 65535) return KV_ERR_UNSUPPORTED;
    int32_t *order = static_cast<int32_t *>(workspace), *table = order + batch;
    char *k_tiles = static_cast<char *>(workspace) + expand_table_bytes(batch, max_blocks);
    char *v_tiles = k_tiles + (size_t)blocks * p->num_kv_heads * kExOut;
    CUtensorMap map_k, map_v;
    if (!encode_rows_map(&map_k, k_tiles, rows) || !encode_rows_map(&map_v, v_tiles, rows)) return KV_ERR_CUDA;
    const bool ordered = batch > 1 && batch <= kOrderBatch;
    const int columns = (max_blocks + 7) / 8;
    const dim3 grid(std::max(columns + (int)ordered, 1), p->num_kv_heads, batch);
    auto fn = q_dtype == KV_BF16 ? expand_i4_kernel<true> : expand_i4_kernel<false>;
    fn<<<grid, 256, 0, as_stream(stream)>>>((const char *)p->k, (const char *)p->v, block_tables, seq_lens, max_blocks,
                                            p->num_blocks, p->num_kv_heads, table, k_tiles, v_tiles, order,
                                            ordered ? columns : -1);
    if (kv_status st = cuda_status(cudaGetLastError())) return st;
    PrefillCall a{};
    a.q = q;
    a.q_dtype = q_dtype;
    a.packed = true;
    a.order = ordered ? order : nullptr;
    a.map_k = &map_k;
    a.map_v = &map_v;
    a.cu_q = cu_q;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.block_tables = table;
    a.max_blocks = max_blocks;
    a.num_blocks = (int)blocks;
    a.num_kv_heads = p->num_kv_heads;
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
