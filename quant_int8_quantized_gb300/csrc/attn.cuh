// What the attention kernels share: the work of a call as a row of key tiles, cut into equal shares.
//
// A *segment* is one tile of query rows against the keys of one head that these rows see: a
// prefix segment (rows of all sequences), or an own segment (rows of one sequence; a prompt's own
// segments begin with the prefix's keys). Its keys come in tiles. All segments' tiles in a row, prefix
// segments first, are cut into runs of equal cost, one per block, whatever the lengths on the device
// are, so ragged batches stay balanced; a run may end inside a segment and go on in the next. What a block
// computes of one segment is a *piece*: the unnormalised output, reference (about the maximum) and sum of its rows over its
// keys, left in
// the workspace at place block + segment (both only grow along the row of tiles, so places differ). The
// joining kernels add a row's pieces up in the order of their keys.
#pragma once

#include "heads.cuh"

namespace attn {

using mq::Div;
using mq::div_by;

// The numbers of one schedule. G: blocks.
struct Plan {
    int B, T, Hq, Hkv, group;       // group = Hq / Hkv
    int prefix_rows, prefix_keys;   // rows per head (B T group) and keys of the prefix segments; 0 keys: none
    int lead_keys;                  // prefix keys at the head of each own segment
    int own_cap;
    int own;                        // there are own segments
    int own_least;                  // tiles of an own segment at least (1: rows that see no key get their zeros there)
    int rows;                       // query rows per segment
    int keys;                       // keys per tile
    int G;
    int lanes;                      // prefix segments only: blocks side by side, one row tile each, over the same keys
    Div by_group, by_per_seq;       // by group; by the row tiles of a sequence (1 where there are none)
    int wide, cost, wide_cost;      // cost of a tile with at most `wide` rows, and with more
    int extra;                      // what a segment costs beside its tiles
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ inline long long ceil_div(long long a, int b) { return (a + b - 1) / b; }

__host__ __device__ inline int prefix_tiles_of_rows(const Plan& p) {
    return p.prefix_keys > 0 ? ceil_div(p.prefix_rows, p.rows) : 0;
}
__host__ __device__ inline int prefix_segs(const Plan& p) { return prefix_tiles_of_rows(p) * p.Hkv; }
__host__ __device__ inline int own_tiles_of_rows(const Plan& p) { return p.own ? ceil_div(p.T * p.group, p.rows) : 0; }
__host__ __device__ inline long long all_segs(const Plan& p) {
    return prefix_segs(p) + (long long)p.B * own_tiles_of_rows(p) * p.Hkv;
}

// Rows of row tile rt of `all`, and what one of its key tiles costs.
__host__ __device__ inline int rows_of(const Plan& p, int all, int rt) {
    return all - rt * p.rows < p.rows ? all - rt * p.rows : p.rows;
}
__host__ __device__ inline int tile_cost(const Plan& p, int rows) { return rows > p.wide ? p.wide_cost : p.cost; }

// Own keys that the last query of row tile rt sees; rows r = t * group + g.
__device__ __forceinline__ int own_seen(const Plan& p, int len, int rt) {
    const int last = min((rt + 1) * p.rows, p.T * p.group) - 1;
    return max(0, len - p.T + 1 + p.by_group.of(last));
}

// Costs are int32: mq_attn_prefix refuses calls whose total would not fit.
// A block's run, moved along segment by segment. Every thread of a block holds the same.
struct Cursor {
    int at, end;                  // cost before the next tile, where the run ends
    int per, longer;              // runs are `per` long, the first `longer` of them one more
    int seg;                      // segment that holds the next tile
    int unit, head;               // its row tile (own segments: sequence * row tiles + row tile) and key head
    int tiles, cost;              // tiles of the segment, cost of one
    int in;                       // tiles of it before the next
    bool prefix;

    __device__ __forceinline__ bool more() const { return at < end; }
};

// The block whose run holds cost x.
__device__ __forceinline__ int block_of(const Cursor& c, int x) {
    const int head = c.longer * (c.per + 1);
    return x < head ? x / (c.per + 1) : c.longer + (x - head) / c.per;
}

__device__ __forceinline__ int own_len_of(const Plan& p, const int32_t* len, int b) {
    return p.own_cap > 0 ? min(max(__ldca(len + b), 0), p.own_cap) : 0;
}
__device__ __forceinline__ int unit_tiles(const Plan& p, const int32_t* len, int unit, int per_seq) {
    const int b = p.by_per_seq.of(unit);
    return max(p.own_least, ceil_div(p.lead_keys, p.keys) +
                                ceil_div(own_seen(p, own_len_of(p, len, b), unit - b * per_seq), p.keys));
}
__device__ __forceinline__ int unit_cost(const Plan& p, int unit, int per_seq) {
    return tile_cost(p, rows_of(p, p.T * p.group, unit - p.by_per_seq.of(unit) * per_seq));
}
__device__ __forceinline__ int seg_cost(const Plan& p, int tiles, int cost) {
    return tiles > 0 ? p.extra + tiles * cost : 0;
}
// Cost of a segment's tiles before tile i: the first one carries the segment's extra cost.
__device__ __forceinline__ int cost_before(const Plan& p, int i, int cost) { return i > 0 ? p.extra + i * cost : 0; }
// The first tile that begins at cost x of its segment or after.
__device__ __forceinline__ int tile_at(const Plan& p, int x, int cost) {
    if (x <= 0) return 0;
    return max(1, (x - p.extra + cost - 1) / cost);
}

// Tiles of the segment that belong to this run, from c.in on.
__device__ __forceinline__ int piece_tiles(const Plan& p, const Cursor& c) {
    const int base = c.at - cost_before(p, c.in, c.cost);   // cost before the segment
    return min(c.tiles, tile_at(p, c.end - base, c.cost)) - c.in;
}
// This block's number in its row of tiles, and the place there of a piece of segment seg.
__device__ __forceinline__ int block_in_lane(const Plan& p) { return p.lanes > 1 ? blockIdx.x / p.lanes : blockIdx.x; }
__host__ __device__ inline int place_of(const Plan& p, int block, int seg) {
    if (p.lanes == 1) return block + seg;
    const int lane = seg / p.Hkv;
    return lane * (p.G / p.lanes + p.Hkv) + block + seg - lane * p.Hkv;
}
// First and last block of the segment that c is at the start of.
__device__ __forceinline__ int2 blocks_of(const Plan& p, const Cursor& c) {
    return make_int2(block_in_lane(p), block_of(c, c.at + cost_before(p, c.tiles - 1, c.cost)));
}

// Finds the block's run. Segments follow one another as unit, then head. Threads share the
// units (sequence and row tile) and scan the sums of their costs: THREADS threads, all of the block.
template <int THREADS>
__device__ __forceinline__ Cursor find_run(const Plan& p, const int32_t* len) {
    if (p.lanes > 1) {              // a row of prefix tiles of one row tile, the same for all lanes
        Cursor c;
        const int lane_of = blockIdx.x % p.lanes, i = blockIdx.x / p.lanes;
        const int cost = p.wide_cost, one = seg_cost(p, ceil_div(p.prefix_keys, p.keys), cost);
        const int total = one * p.Hkv, most = total / (p.extra + cost);
        const int blocks = most < 1 ? 1 : min(most, p.G / p.lanes);
        c.at = c.end = 0;
        if (i >= blocks) return c;
        c.per = total / blocks;
        c.longer = total - c.per * blocks;
        const int begin = i * c.per + min(i, c.longer);
        c.end = begin + c.per + (i < c.longer);
        c.prefix = true;
        c.unit = lane_of;
        c.cost = cost;
        c.tiles = ceil_div(p.prefix_keys, p.keys);
        c.head = begin / one;
        c.seg = lane_of * p.Hkv + c.head;
        const int base = c.head * one;
        c.in = tile_at(p, begin - base, cost);
        c.at = base + (c.in < c.tiles ? cost_before(p, c.in, cost) : one);
        return c;
    }
    constexpr int kWarps = THREADS / 32;
    __shared__ int s_sum[kWarps];
    __shared__ int s_at[3];         // unit, cost before it, its tiles
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int per_seq = own_tiles_of_rows(p), units = p.B * per_seq;
    const int share = ceil_div(units, THREADS);
    const int u0 = min(tid * share, units), u1 = min(u0 + share, units);
    auto cost_of = [&](int u) { return seg_cost(p, unit_tiles(p, len, u, per_seq), unit_cost(p, u, per_seq)); };
    int sum = 0;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) sum += cost_of(u);
    int upto = sum;                 // cost (of one head) of this thread's units and of those before
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
    }
    if (lane == 31) s_sum[wid] = upto;
    __syncthreads();
    int own = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < wid) upto += s_sum[w];
        own += s_sum[w];
    }
    // all row tiles of the prefix are full but the last
    const int pt = ceil_div(p.prefix_keys, p.keys), prt = prefix_tiles_of_rows(p);
    const int last_cost = prt > 0 ? tile_cost(p, rows_of(p, p.prefix_rows, prt - 1)) : 0;
    const int full_cost = tile_cost(p, p.rows);
    const int full = seg_cost(p, pt, full_cost) * p.Hkv, last = prt > 0 ? seg_cost(p, pt, last_cost) * p.Hkv : 0;
    const int prefix = prt > 0 ? full * (prt - 1) + last : 0;
    Cursor c;
    const int total = prefix + own * p.Hkv;
    // every run is at least as long as the longest way between two tiles' beginnings, so none is without a
    // tile: a segment's pieces are those of consecutive blocks
    const int most = total / (p.extra + full_cost);
    const int blocks = most < 1 ? (total > 0) : min(most, p.G), i = blockIdx.x;
    c.at = c.end = 0;
    if (i >= blocks) return c;
    c.per = total / blocks;
    c.longer = total - c.per * blocks;
    const int begin = i * c.per + min(i, c.longer);
    c.end = begin + c.per + (i < c.longer);
    int base;                      // cost before the segment
    if (begin < prefix) {
        c.prefix = true;
        c.unit = min(prt - 1, full > 0 ? begin / full : 0);
        c.cost = c.unit < prt - 1 ? full_cost : last_cost;
        c.tiles = pt;
        const int one = seg_cost(p, pt, c.cost);
        c.head = (begin - c.unit * full) / one;
        c.seg = c.unit * p.Hkv + c.head;
        base = c.unit * full + c.head * one;
    } else {
        const int x = begin - prefix;
        const int mine = upto * p.Hkv, before = mine - sum * p.Hkv;
        if (x >= before && x < mine) {
            int at = before;
#pragma unroll 1
            for (int u = u0; u < u1; ++u) {
                const int n = cost_of(u) * p.Hkv;
                if (x < at + n) {
                    s_at[0] = u;
                    s_at[1] = at;
                    s_at[2] = unit_tiles(p, len, u, per_seq);
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        c.prefix = false;
        c.unit = s_at[0];
        c.tiles = s_at[2];
        c.cost = unit_cost(p, c.unit, per_seq);
        const int one = seg_cost(p, c.tiles, c.cost);
        c.head = (x - s_at[1]) / one;
        c.seg = prefix_segs(p) + c.unit * p.Hkv + c.head;
        base = prefix + s_at[1] + c.head * one;
    }
    // the run's first tile is the first that begins in it, perhaps the next segment's
    c.in = tile_at(p, begin - base, c.cost);
    c.at = base + (c.in < c.tiles ? cost_before(p, c.in, c.cost) : seg_cost(p, c.tiles, c.cost));
    return c;
}

// Past `n` tiles; at a segment's end to the next one that has tiles, if the run goes on.
__device__ __forceinline__ void advance(const Plan& p, const int32_t* len, Cursor& c, int n) {
    if (n > 0) {
        const int base = c.at - cost_before(p, c.in, c.cost);
        c.in += n;
        c.at = base + (c.in < c.tiles ? cost_before(p, c.in, c.cost) : seg_cost(p, c.tiles, c.cost));
    }
    if (c.in < c.tiles || !c.more()) return;
    c.in = 0;
    ++c.seg;
    if (++c.head < p.Hkv) return;
    c.head = 0;
    ++c.unit;
    const int per_seq = own_tiles_of_rows(p);
    if (c.prefix) {
        if (c.unit < prefix_tiles_of_rows(p)) {
            c.cost = tile_cost(p, rows_of(p, p.prefix_rows, c.unit));
            return;
        }
        c.prefix = false;
        c.unit = 0;
    }
    // some unit further on has tiles: the run is not at its end
    while ((c.tiles = unit_tiles(p, len, c.unit, per_seq)) == 0) {
        ++c.unit;
        c.seg += p.Hkv;
    }
    c.cost = unit_cost(p, c.unit, per_seq);
}

// Pieces in the workspace. info[segment] = first and last block that hold tiles of it, written by
// the first; segments without tiles have no entry.
struct Pieces {
    float* o;      // [place][rows][D]
    float2* ml;    // [place][rows]: reference (of the scaled products, base 2) and sum of 2^(product - reference)
    int2* info;
};

// Where finished rows go.
struct Out {
    void* out;     // [B T][Hq][D]
    float* lse;    // [B T][Hq], natural, or nullptr
    int f32;       // out holds f32, not the caches' type
};

constexpr float kLn2 = 0.6931471805599453f;

// Maxima (base 2, scaled) whose last place is no longer small beside the exponents taken against them. (-infinity: no key seen.)
constexpr float kLarge = 1048576.0f;
__device__ __forceinline__ bool is_large(float m) { return fabsf(m) >= kLarge && m != -INFINITY; }

// What a row's exponents are taken against for a maximum of mx: UP powers of two below it, so that f16 has room for weights
// far below the maximum's (against the maximum itself those under 2^-25 would be lost, however many there are). Any such
// reference gives the same sums but for rounding; it stands for the maximum in a piece's statistics.
template <int UP>
__device__ __forceinline__ float reference(float mx) {
    return UP == 0 || fabsf(mx) >= kLarge ? mx : mx - UP;
}

}  // namespace attn
