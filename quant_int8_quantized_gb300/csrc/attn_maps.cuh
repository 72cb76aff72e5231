// Tensor maps (TMA descriptors) of caches and queries, and what waits for their copies.
#pragma once

#include <cuda.h>

#include "attn.cuh"
#include "tc.cuh"

namespace attn {

// Elements between steps that a tensor map can hold (2^40 bytes it cannot).
constexpr long long kStrideMost = (1LL << 39) - 8;

// [n][cap][heads][dim] of k or v (`base`) as (dim, head, row, sequence): boxes of `dims` (64: 128-byte swizzle,
// 32: 64-byte swizzle) by `rows` rows of one head; rows past the cap read as zeros.
bool kv_map(CUtensorMap* map, const mq_kv* c, const void* base, int type, int dims, int rows);

// The queries [B T][Hq][D] as (dim, head, query): a box is 64 dims of `group` heads of `queries` queries.
bool q_map(CUtensorMap* map, const void* q, long long q_stride, long long queries, int Hq, int D, int type, int group,
           int box_queries);

#ifndef MQ_WAIT_LIMIT_NS
#define MQ_WAIT_LIMIT_NS 2000000000ull   // test builds may shorten it
#endif
constexpr uint64_t kWaitLimitNs = MQ_WAIT_LIMIT_NS;

__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
        : "memory");
}
// Non-suspending test of a phase.
__device__ __forceinline__ bool mbar_ready(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(tc::smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

}  // namespace attn
