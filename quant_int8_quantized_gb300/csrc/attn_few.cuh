// Attention pieces (attn.cuh) for few query rows per key head: a decode step's heads, a few drafted
// tokens. See attn_few.cu.
#pragma once

#include "attn.cuh"

namespace attn {

struct FewArgs {
    Plan plan;
    const void* q;
    long long q_stride;
    const int32_t* len;
    float scale_log2;                               // scale * log2 e
    Pieces out;
    float* raw;       // [B][Hkv][T group][cap] scaled products of the own keys (base 2), or nullptr
    int beside;       // launched behind attn_many, whose results it does not need
};

constexpr int kFewRows = 16;      // query rows per segment
constexpr int kFewKeys = 16;      // keys per tile
constexpr int kFewExtra = 2;      // what beginning and ending a segment costs, in tiles
constexpr int kFewPerSm = 8;      // blocks (of one warp) per SM
int launch_few(const FewArgs& a, const mq_kv* prefix, const mq_kv* own, int D, int type, cudaStream_t stream);
#ifdef MQ_TEST_INJECT
bool test_skip_few(int on);
#endif
int take_few_error(unsigned* code);   // bounded waits that gave up; cleared

}  // namespace attn
