// What the kernels between attn_q|k|v and attn_o share: cache descriptors and 16-bit types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mq_internal.cuh"

namespace mq {

// n / d for 0 <= n < 2^31 by a multiplication: l = ceil(log2 d), mul = floor(2^(31 + l) / d) + 1 < 2^32 + 1,
// n / d = n mul >> (31 + l), since mul d exceeds 2^(31 + l) by at most d <= 2^l.
struct Div {
    uint32_t mul;
    int shift, d;
    __device__ __forceinline__ int of(int n) const { return (int)(((unsigned long long)(uint32_t)n * mul) >> shift); }
};
inline Div div_by(int d) {
    int l = 0;
    while ((1LL << l) < d) ++l;
    return Div{(uint32_t)(((1ULL << (31 + l)) / (uint32_t)d) + 1), 31 + l, d};
}

// All rows of a cache apart, strides multiples of 8: of the axes that have more than one
// step, the one with the least stride must clear a head, each further one all that the ones
// before it span.
inline bool kv_apart(const mq_kv* c) {
    long long st[3] = {c->seq_stride, c->row_stride, c->head_stride};
    long long n[3] = {c->n, c->cap, c->heads};
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0 || st[i] % 8 != 0 || st[i] > (1LL << 40)) return false;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (st[j] > st[j + 1]) {
                const long long a = st[j], b = n[j];
                st[j] = st[j + 1];
                n[j] = n[j + 1];
                st[j + 1] = a;
                n[j + 1] = b;
            }
    long long span = c->dim;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1) {
            if (st[i] < span) return false;
            span = st[i] * (n[i] - 1) + span;
        }
    return true;
}

// Elements from the first to one past the last of k (or v).
inline long long kv_span(const mq_kv* c) {
    return c->seq_stride * (c->n - 1) + c->row_stride * (c->cap - 1) + c->head_stride * (c->heads - 1) + c->dim;
}

// Elements from token to token at most, where there are several: bytes of it still fit 64 bits.
constexpr long long kTokenStrideMost = 1LL << 40;

// Whether `rows` rows of `width` bytes, `stride` bytes apart (at least width; of one row: anything) from a on, and the `bytes` from b
// on have a byte in common.
inline bool rows_meet(const void* a, long long rows, long long stride, long long width, const void* b, long long bytes) {
    if (!a || !b || rows <= 0 || width <= 0 || bytes <= 0) return false;
    if (rows == 1) stride = width;
    const long long at = (long long)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const long long first = at < width ? 0 : (at - width) / stride + 1;   // row that ends behind b
    return first < rows && first * stride < at + bytes;
}

inline int check_kv(const mq_kv* c, bool pointers) {
    if (!c) return MQ_ERR_NULL;
    if (c->type != MQ_F16 && c->type != MQ_BF16) return MQ_ERR_TYPE;
    if (c->n < 0 || c->cap < 0 || c->heads < 1 || c->dim < 8 || c->dim % 8 != 0 || c->dim > 256) return MQ_ERR_SHAPE;
    if (!kv_apart(c)) return MQ_ERR_SHAPE;
    if (pointers && c->n > 0 && c->cap > 0) {
        if (!c->k || !c->v) return MQ_ERR_NULL;
        if (!aligned16(c->k) || !aligned16(c->v)) return MQ_ERR_ALIGN;
    }
    return MQ_OK;
}

// launch_pdl in clusters of blocks (1, 1, 1: none).
template <typename... KArgs, typename... Args>
int launch_cluster(void (*kern)(KArgs...), dim3 cluster, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MQ_OK : MQ_ERR_LAUNCH;
}

}  // namespace mq

// Clusters of blocks.
__device__ __forceinline__ uint32_t mq_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mq_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory word of block `rank` of the cluster, at this block's address p.
__device__ __forceinline__ int mq_remote(const int* p, uint32_t rank) {
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

// Two f32 rounded to a pair of 16-bit values, `lo` in the low half.
template <typename T>
__device__ __forceinline__ uint32_t mq_pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t mq_pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t mq_pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
