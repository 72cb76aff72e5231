// What the files of the 4-bit cache call of one another.
#pragma once

#include "mq_internal.cuh"

namespace kv4 {
// mq_kv4_read, checked; values in v_type (dst's type or MQ_F16)
int launch_read(const mq_kv4* src, const int32_t* len, const mq_kv* dst, int v_type, cudaStream_t stream);
}  // namespace kv4

namespace attn {
int take_kv4_error(unsigned* code);   // bounded waits that gave up; cleared
}  // namespace attn
