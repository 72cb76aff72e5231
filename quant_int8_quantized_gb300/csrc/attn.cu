// Attention over a shared prefix and each sequence's own cache: arguments, workspace, and the kernels
// that join the pieces (attn.cuh) into outputs and add up attention weights.

#include <cmath>
#include <limits>

#include "attn_few.cuh"
#include "attn_join.cuh"
#include "attn_many.cuh"
#include "attn_maps.cuh"

namespace attn {
namespace {

// Every query row, a block each: its prefix segment's pieces, then its own segment's, shared out to the block's warps
// in order.
template <typename O, int D, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const JoinArgs a) {
    constexpr int V = Lane<D>::V, W = Lane<D>::W;
    __shared__ float2 s_ml[kJoinWarps];
    __shared__ float s_o[kJoinWarps][W * V * 32];
    mq_grid_release();
    mq_grid_wait();
    const long long row = blockIdx.x;   // (b T + t) Hq + h
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int h = (int)(row % a.Hq);
    const long long bt = row / a.Hq;
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const int hk = h / a.group, tg = a.T * a.group;
    const int r_own = t * a.group + h - hk * a.group;
    // both parts' entries are read at once (an own segment without tiles has none: what lies there is not used)
    Run runs[2] = {};
    int seg0 = 0, seg1 = 0, in0 = 0, in1 = 0, last = 0;
    int2 f0 = make_int2(0, 0), f1 = f0;
    int len = 0;
    if (a.prefix.rows > 0) {
        const int r = b * tg + r_own, rt = r / a.prefix.rows;
        seg0 = rt * a.Hkv + hk;
        in0 = r - rt * a.prefix.rows;
        f0 = __ldca(a.prefix.p.info + seg0);
    }
    if (a.own.rows > 0) {
        const int rt = r_own / a.own.rows;
        last = min((rt + 1) * a.own.rows, tg) - 1;
        seg1 = a.seg0 + (b * ceil_div(tg, a.own.rows) + rt) * a.Hkv + hk;
        in1 = r_own - rt * a.own.rows;
        len = __ldca(a.len + b);
        f1 = __ldca(a.own.p.info + seg1);
    }
    if (a.prefix.rows > 0) runs[0] = run_of(a.prefix, seg0, f0, in0);
    if (a.own.rows > 0 && min(max(len, 0), a.own_cap) - a.T + 1 + last / a.group > 0) runs[1] = run_of(a.own, seg1, f1, in1);
    const int count = runs[0].count + runs[1].count, each = ceil_div(count, kJoinWarps);
    Sum<D> sum = add_pieces<D, kJoinWarps == 1 ? 16 : 8>(runs[0], runs[1], min(wid * each, count), min((wid + 1) * each, count));
    if constexpr (kJoinWarps == 1) {
        write_row<O, D>(sum, a.fin, a.lse2, row);
        return;
    }
    if (lane == 0) s_ml[wid] = make_float2(sum.m, sum.l);
    if (wid > 0)
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s_o[wid][(k * V + e) * 32 + lane] = sum.o[k][e];
    __syncthreads();
    if (wid > 0) return;
    float m = sum.m, f[kJoinWarps];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, s_ml[w].x);
    sum.l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        f[w] = exp2f(s_ml[w].x - (m == -INFINITY ? 0.0f : m));
        sum.l += s_ml[w].y == 0.0f ? 0.0f : s_ml[w].y * f[w];
    }
    sum.m = m;
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float x = sum.o[k][e] * f[0];
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w) x = fmaf(s_o[w][(k * V + e) * 32 + lane], f[w], x);
            sum.o[k][e] = x;
        }
    write_row<O, D>(sum, a.fin, a.lse2, row);
}

// The rows of the segments that one block of the first kernel began and another ended: grid x that block, y rows
// of the segment. All other rows were finished by the block that held them.
struct SplitArgs {
    Part part;
    const int4* split;
    Plan plan;
    Out fin;
};
// A warp takes eight rows: pieces of up to four blocks (there are seldom more) have a lane each, and the loads of four
// rows' outputs are under way at once (a row a warp: 12 us at 3314 tokens of 28 heads of 128, the latency of four
// rounds of warps; eight: 6).
constexpr int kSplitRows = 8, kSplitWarps = 4;
template <typename O, int D>
__global__ void __launch_bounds__(32 * kSplitWarps) attn_join_split_kernel(const SplitArgs a) {
    static_assert(D == 64 || D == 128, "as attn_many");
    constexpr int V = D / 32, kAtOnce = 4;
    mq_grid_release();
    mq_grid_wait();
    const int4 s = __ldca(a.split + blockIdx.x);
    if (s.x < 0) return;
    const int per_seq = own_tiles_of_rows(a.plan), b = a.plan.by_per_seq.of(s.z), rt = s.z - b * per_seq;
    const int rows = rows_of(a.plan, a.plan.T * a.plan.group, rt), lane = threadIdx.x & 31;
    const int in0 = (blockIdx.y * kSplitWarps + (threadIdx.x >> 5)) * kSplitRows;
    if (in0 >= rows) return;
    auto out_row = [&](int in) {
        const int r = rt * a.plan.rows + in, t = a.plan.by_group.of(r);
        return ((long long)b * a.plan.T + t) * a.plan.Hq + s.w * a.plan.group + r - t * a.plan.group;
    };
    const int2 blocks = make_int2(blockIdx.x, s.y);
    const int count = run_of(a.part, s.x, blocks, in0).count;
    if (count > 4) {
        for (int in = in0; in < min(rows, in0 + kSplitRows); ++in)
            write_row<O, D>(add_pieces<D, 4>(run_of(a.part, s.x, blocks, in), Run{}, 0, count), a.fin, nullptr, out_row(in));
        return;
    }
    const int my_row = lane >> 2, my_piece = lane & 3;
    const Run r = run_of(a.part, s.x, blocks, in0);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (my_piece < count && in0 + my_row < rows) ml = __ldca(a.part.p.ml + r.first + my_row + my_piece * r.stride);
    float x[kAtOnce][4][V];
    auto fetch = [&](int row0) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (p < count && in0 + row0 + i < rows) {
                    const float* o = a.part.p.o + (r.first + row0 + i + p * r.stride) * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 v = __ldca(reinterpret_cast<const float4*>(o));
                        x[i][p][0] = v.x, x[i][p][1] = v.y, x[i][p][2] = v.z, x[i][p][3] = v.w;
                    } else {
                        const float2 v = __ldca(reinterpret_cast<const float2*>(o));
                        x[i][p][0] = v.x, x[i][p][1] = v.y;
                    }
                }
    };
    fetch(0);
    float m = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float f = exp2f(ml.x - (m == -INFINITY ? 0.0f : m));
    float l = ml.y == 0.0f ? 0.0f : ml.y * f;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (a.fin.lse && my_piece == 0 && in0 + my_row < rows)
        a.fin.lse[out_row(in0 + my_row)] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
#pragma unroll
    for (int row0 = 0; row0 < kSplitRows; row0 += kAtOnce) {
        if (row0 > 0) fetch(row0);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int in = row0 + i;
            float y[V] = {};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float g = __shfl_sync(0xffffffffu, f, in * 4 + p);
                if (p < count)
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] = fmaf(x[i][p][e], g, y[e]);
            }
            const float by = __shfl_sync(0xffffffffu, inv, in * 4);
            if (in0 + in >= rows) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] *= by;
            const long long at = out_row(in0 + in) * 32 + lane;
            if constexpr (sizeof(O) == 4) {
                if constexpr (V == 4) reinterpret_cast<float4*>(a.fin.out)[at] = make_float4(y[0], y[1], y[2], y[3]);
                else reinterpret_cast<float2*>(a.fin.out)[at] = make_float2(y[0], y[1]);
            } else {
                if constexpr (V == 4)
                    reinterpret_cast<uint2*>(a.fin.out)[at] = make_uint2(mq_pack2<O>(y[0], y[1]), mq_pack2<O>(y[2], y[3]));
                else
                    reinterpret_cast<uint32_t*>(a.fin.out)[at] = mq_pack2<O>(y[0], y[1]);
            }
        }
    }
}

// score_out = score + sum over the rows of 2^(raw - lse2), four keys a thread (one where the rows of raw do not
// begin on 16 bytes).
template <int V>
__global__ void __launch_bounds__(128) attn_score_kernel(const float* raw, const float* lse2, const int32_t* len,
                                                         const float* score, float* score_out, int T, int Hq, int Hkv,
                                                         int cap) {
    mq_grid_release();
    mq_grid_wait();
    const int b = blockIdx.y / Hkv, hk = blockIdx.y - b * Hkv;
    const int n = min(max(__ldca(len + b), 0), cap);
    const int j = (blockIdx.x * 128 + threadIdx.x) * V;
    if (j >= n) return;
    const int group = Hq / Hkv;
    const float* s = raw + (long long)blockIdx.y * T * group * cap + j;
    const long long at = (long long)blockIdx.y * cap + j;
    float w[V] = {}, old[V];
#pragma unroll
    for (int e = 0; e < V; ++e) old[e] = j + e < n ? __ldca(score + at + e) : 0.0f;
    constexpr int kAtOnce = 8;
    const int rows = T * group;
    for (int r0 = 0; r0 < rows; r0 += kAtOnce) {
        float x[kAtOnce][V], l[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (r0 + i < rows) {
                const int t = (r0 + i) / group;
                l[i] = __ldca(lse2 + ((long long)b * T + t) * Hq + hk * group + r0 + i - t * group);
                if constexpr (V == 4) {
                    const float4 v = __ldca(reinterpret_cast<const float4*>(s + (long long)(r0 + i) * cap));
                    x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
                } else {
                    x[i][0] = __ldca(s + (long long)(r0 + i) * cap);
                }
            }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (r0 + i < rows) {
                const int seen = n - T + 1 + (r0 + i) / group;   // past it the first kernel left nothing
#pragma unroll
                for (int e = 0; e < V; ++e) w[e] += j + e < seen && x[i][e] != -INFINITY ? exp2f(x[i][e] - l[i]) : 0.0f;
            }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (j + e < n) score_out[at + e] = old[e] + w[e];
}

// The same for many query rows (a prompt): a warp takes 32 V keys and every so many rows, eight rows' products asked for at
// once; a cluster's warps share the rows out and their sums are added in order. Rows that do not see the first key are left
// out. Bound: HBM, the raw products, and the latency of a warp's few rounds. Whole calls, this way / a thread for all rows: 2000 tokens
// of 28 heads 362 us / 4704, 600: 77 / 1359, 4 sequences of five tokens 18.6 / 27.4; 8 of two (14 rows a head) 33.7 / 31.9.
constexpr int kScoreWarps = 8, kScoreCluster = 8;
template <int V>
__global__ void __launch_bounds__(32 * kScoreWarps) attn_score_rows_kernel(const float* raw, const float* lse2, const int32_t* len,
                                                                           const float* score, float* score_out, int T, int Hq,
                                                                           int Hkv, int cap) {
    constexpr int kKeys = 32 * V, kAtOnce = 8;
    __shared__ float s_warp[kScoreWarps][kKeys], s_block[kKeys];
    mq_grid_release();
    mq_grid_wait();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, C = gridDim.z, rank = blockIdx.z;
    const int b = blockIdx.y / Hkv, hk = blockIdx.y - b * Hkv, group = Hq / Hkv, rows = T * group;
    const int n = min(max(__ldca(len + b), 0), cap);
    const int j0 = blockIdx.x * kKeys, j = j0 + lane * V;
    if (j0 >= n) return;               // all of the cluster
    const float* s = raw + (long long)blockIdx.y * rows * cap + j;
    const int first = max(0, j0 - n + T) * group;      // row that sees key j0
    float w[V] = {};
    for (int r0 = first + (rank * kScoreWarps + wid) * kAtOnce; r0 < rows; r0 += C * kScoreWarps * kAtOnce) {
        float x[kAtOnce][V], l[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (r0 + i < rows && j < n) {
                const int t = (r0 + i) / group;
                l[i] = __ldca(lse2 + ((long long)b * T + t) * Hq + hk * group + r0 + i - t * group);
                if constexpr (V == 4) {
                    const float4 v = __ldcs(reinterpret_cast<const float4*>(s + (long long)(r0 + i) * cap));
                    x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
                } else {
                    x[i][0] = __ldcs(s + (long long)(r0 + i) * cap);
                }
            }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (r0 + i < rows && j < n) {
                const int seen = n - T + 1 + (r0 + i) / group;   // past it the first kernel left nothing
#pragma unroll
                for (int e = 0; e < V; ++e) w[e] += j + e < seen && x[i][e] != -INFINITY ? exp2f(x[i][e] - l[i]) : 0.0f;
            }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_warp[wid][lane * V + e] = w[e];
    __syncthreads();
    if (threadIdx.x < kKeys) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kScoreWarps; ++i) sum += s_warp[i][threadIdx.x];
        s_block[threadIdx.x] = sum;
    }
    if (C > 1) mq_cluster_sync();
    else __syncthreads();
    if (rank == 0 && threadIdx.x < kKeys && j0 + (int)threadIdx.x < n) {
        const long long at = (long long)blockIdx.y * cap + j0 + threadIdx.x;
        float sum = s_block[threadIdx.x];
        for (int i = 1; i < C; ++i) sum += __int_as_float(mq_remote(reinterpret_cast<const int*>(s_block + threadIdx.x), i));
        score_out[at] = __ldca(score + at) + sum;
    }
    if (C > 1) mq_cluster_sync();      // the others' sums stay until they are read
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// The kernel for few rows reads a part's keys and values once for each 16 query rows of a key head, mostly out of L2.
// Up to so many bytes that is quicker than the tensor-core kernel, which takes some 12 us whatever it does.
#ifndef MQ_FEW_BYTES   // (these limits: test builds send small calls to the tensor-core kernel)
#define MQ_FEW_BYTES (64LL << 20)
#endif
constexpr long long kFewBytes = MQ_FEW_BYTES;
#ifndef MQ_MANY_FROM
#define MQ_MANY_FROM 17
#endif
constexpr int kManyFrom = MQ_MANY_FROM;   // query rows per key head, at least, for the tensor-core kernel
// Bytes of the prefix from which several row tiles of it are taken side by side, and how many at most: more of them
// leave more of the blocks that they do not divide idle.
#ifndef MQ_LANES_FROM
#define MQ_LANES_FROM (24LL << 20)
#endif
constexpr long long kLanesFrom = MQ_LANES_FROM;
constexpr int kLanesMost = 8;
// A tile of two halves on one SM; what an SM's eight warps draw beside the other kernel. Both measured.
constexpr double kTileUs = 1.4, kDraw = 80e3;

// Query rows per key head above which attn_score_rows_kernel adds the weights up.
constexpr int kScoreRowsFrom = 16;

// How a call is cut: the part of each kernel, and where the workspace holds what.
struct Cut {
    Plan few, many;
    bool prefix_many, own_many, fits;
    size_t few_o, few_ml, few_info, many_o, many_ml, many_info, split, lse2, raw, bytes;
};

Cut cut_of(int B, int T, int Hq, int Hkv, int D, int prefix_keys, int own_cap, bool scores, bool part) {
    Cut c;
    const int group = Hq / Hkv;
    // bytes that the kernel for few rows would read; the weights' raw products come from it
    const long long row_tiles = ceil_div((long long)T * group, kFewRows), key_bytes = 4LL * Hkv * D;
    const long long own_rows = (long long)T * group, prefix_rows = B * own_rows;
    c.own_many = own_cap > 0 && many_takes(D, group) && !scores &&
                 (part || (own_rows >= kManyFrom && B * row_tiles * own_cap * key_bytes > kFewBytes));
    c.prefix_many = prefix_keys > 0 && !c.own_many && many_takes(D, group) && prefix_rows >= kManyFrom &&
                    ceil_div(prefix_rows, kFewRows) * prefix_keys * key_bytes > kFewBytes;
    c.fits = true;
    size_t at = 0;
    auto plan = [&](bool many, size_t* o, size_t* ml, size_t* info) {
        Plan p;
        p.B = B;
        p.T = T;
        p.Hq = Hq;
        p.Hkv = Hkv;
        p.group = group;
        p.prefix_rows = B * T * group;
        p.prefix_keys = !c.own_many && c.prefix_many == many ? prefix_keys : 0;
        p.lead_keys = many && c.own_many ? prefix_keys : 0;
        p.own = c.own_many == many && own_cap > 0;
        p.own_least = many ? 1 : 0;
        p.own_cap = p.own ? own_cap : 0;
        p.rows = many ? many_rows(group) : kFewRows;
        p.keys = many ? kManyKeys : kFewKeys;
        p.wide = many ? kManyHalf : kFewRows;
        p.cost = many ? kManyCost : 1;
        p.wide_cost = many ? kManyWide : 1;
        p.by_group = div_by(group);
        p.by_per_seq = div_by(p.own ? own_tiles_of_rows(p) : 1);
        p.lanes = 1;
        if (many && p.prefix_keys > 0 && 2LL * prefix_keys * Hkv * D * 2 > kLanesFrom) {
            // row tiles of one size side by side, where the keys would not stay in L2 from one to the next
            const int n = ceil_div(p.prefix_rows, p.rows);
            if (n > 1 && n <= kLanesMost) {
                p.lanes = n;
                p.rows = ceil_div(B * T, n) * group;
                p.lanes = ceil_div(p.prefix_rows, p.rows);
            }
        }
        const long long segs = all_segs(p);
        const long long most = (long long)prefix_segs(p) * ceil_div(p.prefix_keys, p.keys) +
                               (segs - prefix_segs(p)) * (ceil_div(p.lead_keys, p.keys) + ceil_div(p.own_cap, p.keys));
        const long long held = (long long)mq::num_sms() * (many ? 1 : kFewPerSm);
        p.extra = !many ? kFewExtra : p.own ? kManyExtra : kManyExtra / 2;
        if (most * p.wide_cost + segs * p.extra > 0x7fffffffLL) c.fits = false;
        p.G = (int)(most < held ? most : held);
        if (many && p.prefix_keys > 0 && own_cap > 0) {
            // Beside it runs the kernel for few rows, on the SMs that this one leaves: so many that both end
            // together if the caches are half full and each of its SMs draws kDraw bytes a us, but at most half.
            const double own_bytes = (double)B * Hkv * own_cap * D * 2.0, work = (double)most * kTileUs;   // us of one SM
            const int share = (int)(held / (1.0 + own_bytes / (work * kDraw)));
            if (p.G > share) p.G = share > held / 2 ? share : (int)(held / 2 < p.G ? held / 2 : p.G);
        }
        if (p.lanes > 1) p.G = p.G / p.lanes * p.lanes;
        const size_t places = segs > 0 ? (size_t)p.G + (size_t)segs : 0;
        *o = at;
        at += up16(places * p.rows * D * sizeof(float));
        *ml = at;
        at += up16(places * p.rows * sizeof(float2));
        *info = at;
        at += up16((size_t)segs * sizeof(int2));
        return p;
    };
    c.few = plan(false, &c.few_o, &c.few_ml, &c.few_info);
    c.many = plan(true, &c.many_o, &c.many_ml, &c.many_info);
    c.split = at;
    at += c.own_many ? up16((size_t)c.many.G * sizeof(int4)) : 0;
    const size_t rows = (size_t)B * T * Hq;
    c.lse2 = at;
    at += scores ? up16(rows * sizeof(float)) : 0;
    c.raw = at;
    at += scores ? up16(rows * own_cap * sizeof(float)) : 0;
    c.bytes = at;
    return c;
}

bool valid_heads(int Hq, int Hkv, int D) {
    return Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && (D == 64 || D == 96 || D == 128 || D == 256);
}

// Rows, segments and places are counted in int32, and so are keys up to the end of the last tile.
bool valid_counts(long long B, long long T, int Hq, int prefix_cap, int own_cap) {
    constexpr long long kMost = 0x3fffffff;
    constexpr int kCapMost = 0x7fffffff - 255;
    return B * T <= kMost && B * T * Hq <= kMost && prefix_cap <= kCapMost && own_cap <= kCapMost;
}

bool valid_strides(const mq_kv* c) {
    return !c || ((c->n <= 1 || c->seq_stride <= kStrideMost) && (c->cap <= 1 || c->row_stride <= kStrideMost) &&
                  (c->heads <= 1 || c->head_stride <= kStrideMost));
}

// Segments and costs fit int32; with weights, sequences times key heads a grid's y axis.
bool valid_cut(const Cut& c, int B, int Hkv, bool scores) {
    return c.fits && all_segs(c.few) <= 0x3fffffffLL && all_segs(c.many) <= 0x3fffffffLL &&
           !(scores && (long long)B * Hkv > 65535);
}

}  // namespace

int launch_join(const JoinArgs& j, int D, int out_type, cudaStream_t stream) {
    const long long rows = (long long)j.B * j.T * j.Hq;
    auto join = [&](auto o) {
        using O = decltype(o);
        // few rows: eight warps each shorten the way through a row's pieces; many: they fill the GPU by themselves, and a row's
        // few pieces leave most of eight warps idle. Whole call, one warp a row / eight: 400 rows 20.7 / 18.2 us, 560: 27.6 /
        // 25.4, 640: 28.0 / 26.8, 840 of D 64: 14.5 / 17.9, 1024: 33.0 / 35.6, 1600: 24.7 / 31.3
        const bool wide = rows <= 4LL * mq::num_sms();
        auto kern = wide ? (D == 64 ? attn_join_kernel<O, 64, 8> : D == 96 ? attn_join_kernel<O, 96, 8>
                            : D == 128 ? attn_join_kernel<O, 128, 8> : attn_join_kernel<O, 256, 8>)
                         : (D == 64 ? attn_join_kernel<O, 64, 1> : D == 96 ? attn_join_kernel<O, 96, 1>
                            : D == 128 ? attn_join_kernel<O, 128, 1> : attn_join_kernel<O, 256, 1>);
        if (!mq::allow_smem(reinterpret_cast<const void*>(kern), 0)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3((unsigned)rows), dim3(wide ? 256 : 32), 0, stream, j);
    };
    return out_type == MQ_F32 ? join(float()) : out_type == MQ_F16 ? join(__half()) : join(__nv_bfloat16());
}

}  // namespace attn

extern "C" size_t mq_attn_ws_bytes(int B, int T, int Hq, int Hkv, int D, int prefix_cap, int own_cap, int scores) {
    using namespace attn;
    if (B <= 0 || T <= 0 || prefix_cap < 0 || own_cap < 0 || !valid_heads(Hq, Hkv, D) ||
        !valid_counts(B, T, Hq, prefix_cap, own_cap))
        return 0;
    const Cut c = cut_of(B, T, Hq, Hkv, D, prefix_cap, own_cap, scores != 0, false);
    return valid_cut(c, B, Hkv, scores && own_cap > 0) ? c.bytes : 0;
}

namespace attn {

size_t part_ws_bytes(int B, int T, int Hq, int Hkv, int D, int cap) {
    if (!valid_counts(B, T, Hq, 0, cap)) return 0;
    const Cut c = cut_of(B, T, Hq, Hkv, D, 0, cap, false, true);
    return valid_cut(c, B, Hkv, false) ? c.bytes : 0;
}

int call(const void* q, long long q_stride, int B, int T, int Hq, const mq_kv* prefix, const mq_kv* own, const int32_t* own_len,
         float scale, void* out, int out_type, float* lse, const float* score, float* score_out, void* ws, size_t ws_bytes,
         cudaStream_t stream, bool part) {
    if (B < 0 || T < 0) return MQ_ERR_SHAPE;
    const mq_kv* any = own ? own : prefix;
    if (!any) return MQ_ERR_NULL;
    int rc = MQ_OK;
    if (prefix) rc = mq::check_kv(prefix, true);
    if (rc == MQ_OK && own) rc = mq::check_kv(own, true);
    if (rc != MQ_OK) return rc;
    const int Hkv = any->heads, D = any->dim, type = any->type;
    if (prefix && own && (prefix->heads != Hkv || prefix->dim != D)) return MQ_ERR_SHAPE;
    if (prefix && prefix->type != type) return MQ_ERR_TYPE;
    if (out_type != type && out_type != MQ_F32) return MQ_ERR_TYPE;
    if (!valid_heads(Hq, Hkv, D) || (prefix && prefix->n != 1) || (own && own->n != B)) return MQ_ERR_SHAPE;
    if (B == 0 || T == 0) return MQ_OK;
    const int P = prefix ? prefix->cap : 0, cap = own ? own->cap : 0;
    if (!valid_strides(prefix) || !valid_strides(own) || ((long long)B * T > 1 && q_stride > kStrideMost)) return MQ_ERR_SHAPE;
    if (!valid_counts(B, T, Hq, P, cap) || q_stride < (long long)Hq * D || q_stride % 8 != 0 || !std::isfinite(scale))
        return MQ_ERR_SHAPE;
    if (!q || !out || !ws || (own && !own_len) || (score == nullptr) != (score_out == nullptr)) return MQ_ERR_NULL;
    if (!mq::aligned16(q) || !mq::aligned16(out) || !mq::aligned16(ws) || !mq::aligned16(score) || !mq::aligned16(score_out) ||
        (!part && (!mq::aligned16(own_len) || !mq::aligned16(lse))))
        return MQ_ERR_ALIGN;
    const bool scores = score_out && cap > 0;
    Cut c = cut_of(B, T, Hq, Hkv, D, P, cap, scores, part);
    if (!valid_cut(c, B, Hkv, scores)) return MQ_ERR_SHAPE;
    if (ws_bytes < c.bytes) return MQ_ERR_SCRATCH;
    const long long all_rows = (long long)B * T * Hq, score_bytes = scores ? 4LL * B * Hkv * cap : 0;
    if (mq::rows_meet(q, (long long)B * T, 2 * q_stride, 2LL * Hq * D, out, all_rows * D * (out_type == MQ_F32 ? 4 : 2)) ||
        (score != score_out && mq::rows_meet(score, 1, score_bytes, score_bytes, score_out, score_bytes)))
        return MQ_ERR_SHAPE;   // read by some blocks while others write
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    uint8_t* base = static_cast<uint8_t*>(ws);
    auto pieces = [&](size_t o, size_t ml, size_t info) {
        return Pieces{reinterpret_cast<float*>(base + o), reinterpret_cast<float2*>(base + ml),
                      reinterpret_cast<int2*>(base + info)};
    };
    const Pieces few = pieces(c.few_o, c.few_ml, c.few_info), many = pieces(c.many_o, c.many_ml, c.many_info);
    float* lse2 = scores ? reinterpret_cast<float*>(base + c.lse2) : nullptr;
    float* raw = scores ? reinterpret_cast<float*>(base + c.raw) : nullptr;
    const Out fin = {out, lse, out_type == MQ_F32};
    constexpr float kLog2e = 1.4426950408889634f;

    if (all_segs(c.many) > 0) {
        ManyArgs m;
        m.plan = c.many;
        m.q = q;
        m.q_stride = q_stride;
        m.len = own_len;
        // the least scale above zero keeps masked products (-infinity) masked where zero would not, and moves no finite one
        // (below 2^128) by more than 2^-21
        m.scale_log2 = std::fmax(std::fabs(scale) * kLog2e, std::numeric_limits<float>::denorm_min());
        m.negative = scale < 0.0f;
        m.out = many;
        m.split = c.own_many ? reinterpret_cast<int4*>(base + c.split) : nullptr;
        m.fin = fin;
        rc = launch_many(m, P > 0 ? prefix : nullptr, c.own_many ? own : nullptr, D, type, part ? MQ_F16 : type, stream);
        if (rc != MQ_OK) return rc;
        if (c.own_many) {
            const SplitArgs s = {{many, c.many.rows, c.many}, m.split, c.many, fin};
            const int most = T * (Hq / Hkv) < c.many.rows ? T * (Hq / Hkv) : c.many.rows;
            auto join = [&](auto o) {
                using O = decltype(o);
                auto kern = D == 64 ? attn_join_split_kernel<O, 64> : attn_join_split_kernel<O, 128>;
                if (!mq::allow_smem(reinterpret_cast<const void*>(kern), 0)) return (int)MQ_ERR_LAUNCH;
                return mq::launch_pdl(kern, dim3(c.many.G, (most + kSplitRows * kSplitWarps - 1) / (kSplitRows * kSplitWarps)),
                                      dim3(32 * kSplitWarps), 0, stream, s);
            };
            return out_type == MQ_F32 ? join(float()) : out_type == MQ_F16 ? join(__half()) : join(__nv_bfloat16());
        }
    }
    if (all_segs(c.few) > 0) {
        FewArgs f;
        f.plan = c.few;
        f.q = q;
        f.q_stride = q_stride;
        f.len = own_len;
        f.scale_log2 = scale * kLog2e;
        f.out = few;
        f.raw = raw;
        f.beside = all_segs(c.many) > 0;
        rc = launch_few(f, P > 0 ? prefix : nullptr, cap > 0 ? own : nullptr, D, type, stream);
        if (rc != MQ_OK) return rc;
    }
    JoinArgs j;
    j.prefix = {c.prefix_many ? many : few, P > 0 ? (c.prefix_many ? c.many.rows : kFewRows) : 0,
                c.prefix_many ? c.many : c.few};
    j.own = {few, cap > 0 ? kFewRows : 0, c.few};
    j.len = own_len;
    j.B = B;
    j.T = T;
    j.Hq = Hq;
    j.Hkv = Hkv;
    j.group = Hq / Hkv;
    j.own_cap = cap;
    j.seg0 = prefix_segs(c.few);
    j.fin = fin;
    j.lse2 = lse2;
    rc = launch_join(j, D, out_type, stream);
    if (rc != MQ_OK || !scores) return rc;
    const int rows = T * j.group;
    if (rows > kScoreRowsFrom) {
        int C = 1;                      // some 16 rows a warp
        while (C < kScoreCluster && rows > 128 * C) C *= 2;
        auto kern = cap % 4 == 0 ? attn_score_rows_kernel<4> : attn_score_rows_kernel<1>;
        const int keys = cap % 4 == 0 ? 128 : 32;
        if (!mq::allow_smem(reinterpret_cast<const void*>(kern), 0)) return MQ_ERR_LAUNCH;
        return mq::launch_cluster(kern, dim3(1, 1, C), dim3((cap + keys - 1) / keys, B * Hkv, C), dim3(32 * kScoreWarps), 0,
                                  stream, raw, lse2, own_len, score, score_out, T, Hq, Hkv, cap);
    }
    auto score_call = [&](auto kern, int keys) {
        if (!mq::allow_smem(reinterpret_cast<const void*>(kern), 0)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3((cap + keys - 1) / keys, B * Hkv), dim3(128), 0, stream, raw, lse2, own_len,
                              score, score_out, T, Hq, Hkv, cap);
    };
    return cap % 4 == 0 ? score_call(attn_score_kernel<4>, 512) : score_call(attn_score_kernel<1>, 128);
}

}  // namespace attn

extern "C" int mq_attn_prefix(const void* q, long long q_stride, int B, int T, int Hq, const mq_kv* prefix,
                              const mq_kv* own, const int32_t* own_len, float scale, void* out, int out_type,
                              float* lse, const float* score, float* score_out, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
    return attn::call(q, q_stride, B, T, Hq, prefix, own, own_len, scale, out, out_type, lse, score, score_out, ws, ws_bytes,
                      stream, false);
}
