// Attention pieces (attn.cuh) for many query rows per key head: a batch on one prefix, a prompt. See
// attn_many.cu.
#pragma once

#include "attn.cuh"

namespace attn {

struct ManyArgs {
    Plan plan;
    const void* q;
    long long q_stride;
    const int32_t* len;
    float scale_log2;     // |scale| log2 e, above zero
    int negative;         // scale < 0
    Pieces out;
    int4* split;          // [G]: segment that begins in the block and goes on in others (or -1), its last block,
                          // its row tile (sequence and tile) and key head; nullptr: the call joins by row
    Out fin;              // with `split`: segments that one block holds are finished here
};

constexpr int kManyRows = 256;    // query rows per segment, at most
constexpr int kManyHalf = 128;    // rows of one half
constexpr int kManyKeys = 128;    // keys per tile

// Costs: a tile of two halves, a tile of a segment that one half would hold (its tiles alternate between the
// halves: measured at two thirds of the former), a segment's beginning and
// end (8192 tokens of 32 heads: 7 364 us, 8 362, 10 365, 13 369; 3314 of 28: 112, 113, 112, 114).
constexpr int kManyCost = 2, kManyWide = 3, kManyExtra = 7;

// Whole queries only: a segment's rows are one box of the queries' tensor map.
inline int many_rows(int group) { return kManyRows / group * group; }

inline bool many_takes(int D, int group) { return (D == 64 || D == 128) && group <= kManyRows; }
// v_type: of the values, `type` or MQ_F16.
int launch_many(const ManyArgs& a, const mq_kv* prefix, const mq_kv* own, int D, int type, int v_type, cudaStream_t stream);

}  // namespace attn
