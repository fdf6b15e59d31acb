// Tiled-TMA tensor maps (CUtensorMap) for the pools, per-request contiguous
// regions and prefill queries.  Every map describes rows of 128 16-bit values
// (bf16 or fp16: the copies move bits, so one data type serves both) read as
// boxes of 16 rows x 64 values with 128-byte swizzle (the layout both the
// tcgen05 descriptors and the ldmatrix address math expect).  Group maps (tree attention)
// read a whole block as one box: 8 rows x 64 values, the other 64, the other 8 rows.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "internal.h"

namespace pkv {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static void *driver_fn(const char *name) {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion(name, &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? f
               : nullptr;
}

static EncodeTiledFn encode_fn() {
    using GetCurrentFn = CUresult (*)(CUcontext *);
    static EncodeTiledFn fn = nullptr;
    static GetCurrentFn current = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        fn = reinterpret_cast<EncodeTiledFn>(driver_fn("cuTensorMapEncodeTiled"));
        current = reinterpret_cast<GetCurrentFn>(driver_fn("cuCtxGetCurrent"));
    });
    // Encoding asks for a current context.  A host thread without one gets its device's primary context, as its
    // first runtime call that needs one would give it; one that a thread has, of its own even, stays.
    CUcontext ctx = nullptr;
    if (current && (current(&ctx) != CUDA_SUCCESS || !ctx))
        if (int dev = 0; cudaGetDevice(&dev) == cudaSuccess) cudaSetDevice(dev);
    return fn;
}

bool encode_rows_map(CUtensorMap *m, void *base, long long rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc || rows <= 0) return false;
    cuuint64_t dims[2] = {128, (cuuint64_t)rows};
    cuuint64_t strides[1] = {128 * 2};
    cuuint32_t box[2] = {64, 16};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_groups_map(CUtensorMap *m, void *base, long long rows, int dim) {
    EncodeTiledFn enc = encode_fn();
    if (!enc || rows <= 0) return false;
    cuuint64_t dims[4] = {64, 8, (cuuint64_t)dim / 64, (cuuint64_t)rows / 8};
    cuuint64_t strides[3] = {(cuuint64_t)dim * 2, 128, (cuuint64_t)dim * 16};
    cuuint32_t box[4] = {64, 8, (cuuint32_t)dim / 64, 2};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_q_map(CUtensorMap *m, const void *q, int rows, int hq, int box_heads, int box_rows, int dim) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)hq, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)hq * dim * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool's maps are made by its first call that needs them, which may be two threads' at once.
static std::mutex making;

kv_status pool_tensor_maps(kv_pool *p) {
    std::lock_guard<std::mutex> lock(making);
    if (p->tmaps_ready) return KV_OK;
    if (p->dtype == KV_F32 || p->dtype == KV_I4 || p->head_dim != 128) return KV_ERR_UNSUPPORTED;
    const long long rows = (long long)p->num_blocks * p->num_kv_heads * 16;
    if (rows > INT32_MAX) return KV_ERR_UNSUPPORTED;
    if (!encode_rows_map(&p->tmap_k, p->k, rows) || !encode_rows_map(&p->tmap_v, p->v, rows))
        return KV_ERR_CUDA;
    p->tmaps_ready = true;
    return KV_OK;
}

kv_status pool_group_maps(kv_pool *p) {
    std::lock_guard<std::mutex> lock(making);
    if (p->gmaps_ready) return KV_OK;
    if (p->dtype == KV_F32 || p->dtype == KV_I4) return KV_ERR_UNSUPPORTED;
    const long long rows = (long long)p->num_blocks * p->num_kv_heads * 16;
    if (rows > INT32_MAX) return KV_ERR_UNSUPPORTED;
    if (!encode_groups_map(&p->gmap_k, p->k, rows, p->head_dim) || !encode_groups_map(&p->gmap_v, p->v, rows, p->head_dim))
        return KV_ERR_CUDA;
    p->gmaps_ready = true;
    return KV_OK;
}

}  // namespace pkv
