// Tensor maps (TMA descriptors) of caches and queries.

#include "attn_maps.cuh"

#include <cudaTypedefs.h>

#include <mutex>

namespace attn {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode(CUtensorMap* map, int type, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return fn(map, type == MQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool kv_map(CUtensorMap* map, const mq_kv* c, const void* base, int box_dims, int box_rows) {
    // an axis of one step may have any stride: nothing steps along it
    auto stride = [](long long s, int steps) { return (cuuint64_t)(steps > 1 ? s * 2 : 16); };
    const cuuint64_t dims[4] = {(cuuint64_t)c->dim, (cuuint64_t)c->heads, (cuuint64_t)c->cap, (cuuint64_t)c->n};
    const cuuint64_t strides[3] = {stride(c->head_stride, c->heads), stride(c->row_stride, c->cap), stride(c->seq_stride, c->n)};
    const cuuint32_t box[4] = {(cuuint32_t)box_dims, 1, (cuuint32_t)box_rows, 1};
    return encode(map, c->type, base, 4, dims, strides, box);
}

bool q_map(CUtensorMap* map, const void* q, long long q_stride, long long queries, int Hq, int D, int type, int group,
           int box_queries) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)queries};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)(queries > 1 ? q_stride : (long long)Hq * D) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)box_queries};
    return encode(map, type, q, 3, dims, strides, box);
}

}  // namespace attn
