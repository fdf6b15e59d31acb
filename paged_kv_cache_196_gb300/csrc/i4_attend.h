// The 4-bit decode kernel's call, shared by the decode entry point and the
// prefill of a few query tokens.
#pragma once
#include "internal.h"

namespace pkv {

struct I4Call {
    kv_pool *pool;
    const void *q;
    kv_dtype q_dtype;
    const int32_t *cu_q;  // null: one query token per sequence
    int total_q, max_q_len;
    const int32_t *block_tables;
    int max_blocks;
    const int32_t *seq_lens, *seq_order;
    int batch, num_q_heads;
    float scale;
    void *out;
    kv_dtype out_dtype;
    float *lse;
    int num_splits;
    void *workspace;
    size_t workspace_bytes;
    cudaStream_t stream;
};

// KV_ERR_UNSUPPORTED: sizes past a limit of the launch.  cols: query tokens x heads of a
// (sequence, kv head); max_splits: partitions of a table row.
kv_status attend_i4_limits(int batch, int num_kv_heads, int cols, int max_blocks, int max_splits);

// Launches the attention of checked arguments; KV_ERR_ARG: the workspace is too
// small, KV_ERR_UNSUPPORTED: attend_i4_limits.
kv_status attend_i4(const I4Call &a);

}  // namespace pkv
