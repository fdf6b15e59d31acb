// Tree attention: what its kernels share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tree_plan.cuh"

namespace pkv {
namespace tree {

KV_DEVICE float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct TreeParams {
    Plan plan;
    const void *q;           // rows [total_q][hq][D], the pool's type
    const void *k, *v;       // the pool's arrays
    const int32_t *tables;   // [batch][max_blocks]
    const int32_t *parents;  // [total_q]: index within the tree, -1: none; null: chains
    int num_blocks;
    int hq, g;
    int copies;              // of each row in its tile (16-bit pools)
    int total_q;             // rows of q
    float scale_log2;        // softmax scale * log2(e)
    void *out;
    int out_type;
    float *lse;
    float *partial;          // slots of [D / 4][rows] float4 and [rows] (reference, sum)
    Cut *cuts;               // [runs]
    int *err;
};

// tree_tc.cu: 16-bit pools; one or two row tiles (`rows` = 128 or 256), tensor maps of the
// pool's K and V in groups of rows.
kv_status launch_tc(const TreeParams &pp, int d, int rows, bool f16, const CUtensorMap &tk, const CUtensorMap &tv,
                    cudaStream_t stream);

}  // namespace tree
}  // namespace pkv
