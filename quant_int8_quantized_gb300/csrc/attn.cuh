// What the attention kernels share: the work of a call as a row of key tiles, cut into equal shares.
//
// A *segment* is one tile of query rows against the keys of one head that these rows see: a
// prefix segment (rows of all sequences) or an own segment (rows of one sequence). Its keys come
// in tiles. All segments' tiles in a row, prefix segments first, are cut into one equal run per
// block, whatever the lengths on the device are, so ragged batches stay balanced; a run may end inside a
// segment and go on in the next. What a block computes of one segment is a *piece*: the
// unnormalised output, maximum and sum of its rows over its keys, left in the workspace at place
// block + segment (both only grow along the row of tiles, so places differ). The joining kernel adds
// a row's pieces up in the order of their keys.
#pragma once

#include "heads.cuh"

namespace attn {

// The numbers of one schedule. G: blocks.
struct Plan {
    int B, T, Hq, Hkv, group;       // group = Hq / Hkv
    int prefix_rows, prefix_keys;   // rows per head of the prefix segments (B T group), or no segments
    int own_cap;                    // 0: no own segments
    int rows;                       // query rows per segment
    int keys;                       // keys per tile
    int G;
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline long long ceil_div(long long a, int b) { return (a + b - 1) / b; }

__host__ __device__ inline int prefix_tiles_of_rows(const Plan& p) {
    return p.prefix_keys > 0 ? ceil_div(p.prefix_rows, p.rows) : 0;
}
__host__ __device__ inline int prefix_segs(const Plan& p) { return prefix_tiles_of_rows(p) * p.Hkv; }
__host__ __device__ inline int own_tiles_of_rows(const Plan& p) {
    return p.own_cap > 0 ? ceil_div(p.T * p.group, p.rows) : 0;
}
__host__ __device__ inline long long all_segs(const Plan& p) {
    return prefix_segs(p) + (long long)p.B * own_tiles_of_rows(p) * p.Hkv;
}

// Own keys that the last query of row tile rt sees; rows r = t * group + g.
__host__ __device__ inline int own_seen(const Plan& p, int len, int rt) {
    const int last = (rt + 1) * p.rows < p.T * p.group ? (rt + 1) * p.rows - 1 : p.T * p.group - 1;
    const int n = len - p.T + 1 + last / p.group;
    return n > 0 ? n : 0;
}

// The block that holds tile x of W.
__device__ __forceinline__ int block_of(long long x, long long W, int G) { return (int)(((x + 1) * G - 1) / W); }

// A place in the row of tiles, moved along segment by segment. Every thread of a block holds the same.
struct Cursor {
    long long tile, end, total;   // this block's run, all tiles
    int blocks;                   // that have a run: as many as there are tiles, at most p.G
    int seg;                      // segment that holds `tile`
    int unit, head;               // its row tile (own segments: sequence * row tiles + row tile) and key head
    int seg_tiles;                // tiles of the segment
    int in;                       // tiles of it before `tile`
    bool prefix;
};

__device__ __forceinline__ int own_len_of(const Plan& p, const int32_t* len, int b) {
    return min(max(__ldca(len + b), 0), p.own_cap);
}
__device__ __forceinline__ int unit_tiles(const Plan& p, const int32_t* len, int unit, int per_seq) {
    const int b = unit / per_seq;
    return ceil_div(own_seen(p, own_len_of(p, len, b), unit - b * per_seq), p.keys);
}

// Finds the block's run. Segments follow one another as unit, then head. Threads share the
// units (sequence and row tile) and scan the sums of their tiles: THREADS threads, all of the block.
template <int THREADS>
__device__ __forceinline__ Cursor find_run(const Plan& p, const int32_t* len) {
    constexpr int kWarps = THREADS / 32;
    __shared__ long long s_sum[kWarps];
    __shared__ long long s_at[2];   // unit, tiles before it
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int per_seq = own_tiles_of_rows(p), units = p.B * per_seq;
    const int share = ceil_div(units, THREADS);
    const int u0 = min(tid * share, units), u1 = min(u0 + share, units);
    long long sum = 0;
    for (int u = u0; u < u1; ++u) sum += unit_tiles(p, len, u, per_seq);
    long long upto = sum;           // tiles of this thread's units and of those before
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) s_sum[wid] = upto;
    __syncthreads();
    long long own = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < wid) upto += s_sum[w];
        own += s_sum[w];
    }
    const int pt = p.prefix_keys > 0 ? ceil_div(p.prefix_keys, p.keys) : 0;
    const long long prefix = (long long)prefix_segs(p) * pt;
    Cursor c;
    c.total = prefix + own * p.Hkv;
    // no block in between is without a tile: a segment's pieces are those of consecutive blocks
    c.blocks = c.total < p.G ? (int)c.total : p.G;
    c.tile = c.end = 0;
    if (blockIdx.x >= c.blocks) return c;
    c.tile = c.total * blockIdx.x / c.blocks;
    c.end = c.total * (blockIdx.x + 1) / c.blocks;
    if (c.tile < prefix) {
        c.prefix = true;
        c.seg = (int)(c.tile / pt);
        c.in = (int)(c.tile - (long long)c.seg * pt);
        c.unit = c.seg / p.Hkv;
        c.head = c.seg - c.unit * p.Hkv;
        c.seg_tiles = pt;
        return c;
    }
    const long long x = c.tile - prefix;
    const long long mine = upto * p.Hkv, before = mine - sum * p.Hkv;
    if (x >= before && x < mine) {
        long long at = before;
        for (int u = u0; u < u1; ++u) {
            const long long n = (long long)unit_tiles(p, len, u, per_seq) * p.Hkv;
            if (x < at + n) {
                s_at[0] = u;
                s_at[1] = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    c.prefix = false;
    c.unit = (int)s_at[0];
    c.seg_tiles = unit_tiles(p, len, c.unit, per_seq);
    const int rest = (int)(x - s_at[1]);
    c.head = rest / c.seg_tiles;
    c.in = rest - c.head * c.seg_tiles;
    c.seg = prefix_segs(p) + c.unit * p.Hkv + c.head;
    return c;
}

// To the next segment that has tiles, once `tile` has reached the end of this one.
__device__ __forceinline__ void next_segment(const Plan& p, const int32_t* len, Cursor& c) {
    c.in = 0;
    ++c.seg;
    if (++c.head < p.Hkv) return;
    c.head = 0;
    ++c.unit;
    if (c.prefix) {
        if (c.unit < prefix_tiles_of_rows(p)) return;
        c.prefix = false;
        c.unit = 0;
    }
    const int per_seq = own_tiles_of_rows(p);
    // some unit further on has tiles: this block's run is not at its end
    while ((c.seg_tiles = unit_tiles(p, len, c.unit, per_seq)) == 0) {
        ++c.unit;
        c.seg += p.Hkv;
    }
}

// Pieces in the workspace. info[segment] = first and last block that hold tiles of it, written by
// the first; segments without tiles have no entry.
struct Pieces {
    float* o;      // [place][rows][D]
    float2* ml;    // [place][rows]: maximum (of the scaled products, base 2) and sum
    int2* info;
};

// Lets `kern` use `bytes` of dynamic shared memory (asked once per kernel and device).
bool allow_smem(const void* kern, int bytes);

}  // namespace attn
