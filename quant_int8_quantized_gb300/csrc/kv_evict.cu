// Eviction from a cache by accumulated attention weight: per sequence and key head the `recent`
// last rows stay and, of the others, those with the largest score; kept rows keep their order.
//
// Scores become unsigned keys in the same order, and the key of the last row that is kept is found digit by
// digit: a histogram of 8 bits a round, counted in shared memory, until few rows share the digits and are compared with one
// another. Long rows are shared out to a cluster of blocks, which add their histograms up through distributed shared
// memory; each block reads its stretch of the scores from memory once. Then every warp writes the kept rows' numbers and
// scores of its own stretch in order, from the counts of the stretches before it. Counts are integers: the result does not
// depend on the order of the atomics. Bound: the rounds' barriers (8 heads of 512, all of the call: 6.6 us) and, on long
// rows, the passes over the keys (8 heads of 131072: 26 us of 47).
// Then rows and values move in a second launch, which shares them out evenly: 16 bytes at a time, every kept row read
// once and written once. Bound: HBM (256 heads of up to 4096 rows of 128, cut to 1024: 273 MB in 61 us with the selection's
// 13, 5.7 TB/s without; blocks that move what they selected themselves take longer: the machine waits for the SMs that hold
// two of them).

#include "heads.cuh"

namespace {

constexpr int kMaxCluster = 8;
constexpr int kBrief = 2048;             // scores of a head up to which a block has 256 threads, not 1024
constexpr int kMaxKeys = 40 * 1024;      // of a block's stretch that shared memory holds; longer ones are read again

constexpr int kMostRows = 0x7fffffff - 0xffff;   // loops over rows step past the last by at most 8 x 1024

// Order of floats as unsigned integers; -0 equals +0, NaN is below everything.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0u;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

struct Move {
    const uint4 *k, *v;
    uint4 *dk, *dv;
    const float* score;
    float* score_out;
    const int32_t* index;
    const int32_t* len;
    int32_t* len_out;
    long long ss, sr, sh, ds, dr, dh;   // strides in 16-byte units
    int n, heads, cap, dst_cap, keep, chunks;
    mq::Div by_blocks, by_row, by_chunks;   // blocks of a sequence, 16-byte units of a row (of all heads), of a head
    int rows;                               // of a sequence that a block moves
};

// Selection for one head of one sequence by a cluster of C blocks.
// Few warps for short rows: the rounds are then a matter of barriers and of adding the warps' histograms up.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Move a, int recent, int C, int keys_held,
                                                                   int32_t* index) {
    constexpr int kWarps = kSelThreads / 32;
    extern __shared__ uint32_t s_keys[];                  // keys of this block's stretch, if they fit
    __shared__ int s_hist[kWarps][256];
    __shared__ int s_tot[2][256], s_all[256];
    __shared__ int s_gt[kWarps], s_eq[kWarps], s_cnt[2];
    constexpr int kLast = kSelThreads / 2;
    __shared__ uint32_t s_cand[kLast], s_list[kLast];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need, s_in, s_n;
    mq_grid_release();
    mq_grid_wait();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = C > 1 ? (int)mq_cluster_rank() : 0, row = blockIdx.x / C;
    const int b = row / a.heads;
    const int n = min(max(a.len[b], 0), a.cap), keep = a.keep, dst_cap = a.dst_cap;
    const float* sc = a.score + (long long)row * a.cap;
    int32_t* out = index + (long long)row * dst_cap;
    float* so = a.score_out ? a.score_out + (long long)row * dst_cap : nullptr;
    auto take = [&](int to, int from) {          // row `from` (-1: none) is now row `to`
        out[to] = from;
        if (so) so[to] = from < 0 ? 0.0f : mq_ld_dep(sc + from);
    };
    const int step = C * kSelThreads, first = rank * kSelThreads + tid;
    if (n <= keep) {
        for (int j = first; j < dst_cap; j += step) take(j, j < n ? j : -1);
    } else {
        const int cand = n - recent;            // rows that compete for `best` places
        const int best = keep - recent;
        for (int j = first; j < recent; j += step) take(best + j, cand + j);
        for (int j = keep + first; j < dst_cap; j += step) take(j, -1);
        // (best is the same for all blocks of the cluster)
        if (best > 0) {
            const int per = ((cand + C - 1) / C + 31) / 32 * 32;
            const int base = min(rank * per, cand), mine = min(per, cand - base);
            const bool held = mine <= keys_held;
            const unsigned lower = (1u << lane) - 1u;
            if (tid == 0) s_n = 0;
            if (held) {
                constexpr int kAtOnce = 8;
                for (int j0 = tid; j0 < mine; j0 += kAtOnce * kSelThreads) {
                    float x[kAtOnce];
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        if (j0 + u * kSelThreads < mine) x[u] = mq_ld_dep(sc + base + j0 + u * kSelThreads);
#pragma unroll
                    for (int u = 0; u < kAtOnce; ++u)
                        if (j0 + u * kSelThreads < mine) s_keys[j0 + u * kSelThreads] = order_key(x[u]);
                }
            }
            __syncthreads();
            auto key = [&](int j) { return held ? s_keys[j] : order_key(mq_ld_dep(sc + base + j)); };
            uint32_t prefix = 0;
            int need = best;                    // rows still to be taken among those that share `prefix`
#pragma unroll 1
            for (int round = 0; round < 4; ++round) {
                const int shift = 24 - 8 * round;
                for (int i = lane; i < 256; i += 32) s_hist[wid][i] = 0;
                __syncwarp();
                const uint32_t above = round == 0 ? 0u : 0xffffffffu << (shift + 8);
                for (int j0 = wid * 32; j0 < mine; j0 += kSelThreads) {
                    const int j = j0 + lane;
                    const uint32_t k = j < mine ? key(j) : 0u;
                    const bool in = j < mine && (k & above) == prefix;
                    const unsigned who = __ballot_sync(0xffffffffu, in);
                    if (in) {
                        const int digit = (int)(k >> shift) & 255;
                        int same;               // a digit that all share is counted once: equal scores would queue
                        __match_all_sync(who, digit, &same);
                        if (!same) atomicAdd(&s_hist[wid][digit], 1);
                        else if (lane == __ffs(who) - 1) atomicAdd(&s_hist[wid][digit], __popc(who));
                    }
                }
                __syncthreads();
                int* tot = s_tot[round & 1];
                if (tid < 256) {
                    int t = 0;
#pragma unroll 8
                    for (int w = 0; w < kWarps; ++w) t += s_hist[w][tid];
                    if (C > 1) tot[tid] = t;
                    else s_all[tid] = t;
                }
                if (C > 1) {
                    mq_cluster_sync();
                    if (tid < 256) {
                        int t[kMaxCluster];
#pragma unroll
                        for (int r = 0; r < kMaxCluster; ++r) t[r] = r < C ? mq_remote(tot + tid, r) : 0;
#pragma unroll
                        for (int r = 1; r < kMaxCluster; ++r) t[0] += t[r];
                        s_all[tid] = t[0];
                    }
                }
                __syncthreads();
                if (wid == 0) {                  // the digit at which the rows from the top reach `need`
                    int t[8], sum = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum += t[i] = s_all[255 - (lane * 8 + i)];
                    int run = sum;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int u = __shfl_up_sync(0xffffffffu, run, o);
                        if (lane >= o) run += u;
                    }
                    int before = run - sum;
                    if (before < need && run >= need) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (before < need && before + t[i] >= need) {
                                s_prefix = prefix | (uint32_t)(255 - (lane * 8 + i)) << shift;
                                s_need = need - before;
                                s_in = t[i];
                                break;
                            }
                            before += t[i];
                        }
                    }
                }
                __syncthreads();
                prefix = s_prefix;
                need = s_need;
                const int in = s_in;
                // Few share the digits so far: each is compared with all the others, by some threads next to one another. That
                // takes in^2 steps, another round a few for each key (256 heads of 4096: up to 256 15.5 us, up to 128 13.4;
                // blocks of 65536 keys: up to 128 135 us, up to 512 122).
                if (round == 3 || in > kLast || (in > 128 && in * in > 8 * per)) continue;
                const uint32_t mask = 0xffffffffu << shift;
                for (int j0 = wid * 32; j0 < mine; j0 += kSelThreads) {
                    const int j = j0 + lane;
                    const uint32_t k = j < mine ? key(j) : 0u;
                    const bool one = j < mine && (k & mask) == prefix;
                    const unsigned who = __ballot_sync(0xffffffffu, one);
                    if (who == 0) continue;
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&s_n, __popc(who));
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & lower);
                    if (one) s_cand[at] = k;
                }
                const uint32_t* list = s_cand;
                if (C > 1) {
                    mq_cluster_sync();
                    if (tid < in) {
                        int r = 0, at = tid;
                        for (int c = mq_remote(&s_n, 0); at >= c && r < C - 1; c = mq_remote(&s_n, r)) {
                            at -= c;
                            ++r;
                        }
                        s_list[tid] = (uint32_t)mq_remote(reinterpret_cast<const int*>(s_cand) + at, r);
                    }
                    list = s_list;
                }
                __syncthreads();
                int side = 32;
                while (side * in > kSelThreads) side >>= 1;
                const int me = tid / side;
                const uint32_t k = me < in ? list[me] : 0u;
                int gt = 0, eq = 0;
                if (me < in)
                    for (int i = tid & (side - 1); i < in; i += side) {
                        gt += list[i] > k;
                        eq += list[i] == k;
                    }
                for (int o = side / 2; o >= 1; o >>= 1) {
                    gt += __shfl_xor_sync(0xffffffffu, gt, o);
                    eq += __shfl_xor_sync(0xffffffffu, eq, o);
                }
                if (me < in && gt < need && gt + eq >= need) {   // (the same value from all that are equal)
                    s_prefix = k;
                    s_need = need - gt;
                }
                __syncthreads();
                prefix = s_prefix;
                need = s_need;
                break;
            }
            // kept: key above `prefix`, and the first `need` rows of those equal to it
            const int stretch = ((mine + kWarps - 1) / kWarps + 31) / 32 * 32;
            const int j0 = min(wid * stretch, mine), j1 = min(j0 + stretch, mine);
            int gt = 0, eq = 0;
            for (int j = j0 + lane; j < j1; j += 32) {
                const uint32_t k = key(j);
                gt += k > prefix;
                eq += k == prefix;
            }
            gt = __reduce_add_sync(0xffffffffu, gt);
            eq = __reduce_add_sync(0xffffffffu, eq);
            if (lane == 0) {
                s_gt[wid] = gt;
                s_eq[wid] = eq;
            }
            __syncthreads();
            // counts of the warps before this one (a warp per lane), and of the blocks before this block
            const int wg = lane < kWarps ? s_gt[lane] : 0, we = lane < kWarps ? s_eq[lane] : 0;
            int g0 = __reduce_add_sync(0xffffffffu, lane < wid ? wg : 0), e0 = __reduce_add_sync(0xffffffffu, lane < wid ? we : 0);
            if (C > 1) {
                const int ag = __reduce_add_sync(0xffffffffu, wg), ae = __reduce_add_sync(0xffffffffu, we);
                if (tid == 0) {
                    s_cnt[0] = ag;
                    s_cnt[1] = ae;
                }
                mq_cluster_sync();
                const int bg = lane < rank ? mq_remote(&s_cnt[0], lane) : 0, be = lane < rank ? mq_remote(&s_cnt[1], lane) : 0;
                g0 += __reduce_add_sync(0xffffffffu, bg);
                e0 += __reduce_add_sync(0xffffffffu, be);
            }
            for (int i = j0; i < j1; i += 32) {
                const int j = i + lane;
                const uint32_t k = j < j1 ? key(j) : 0u;
                const bool isg = j < j1 && k > prefix, ise = j < j1 && k == prefix;
                const unsigned bg = __ballot_sync(0xffffffffu, isg), be = __ballot_sync(0xffffffffu, ise);
                const int g = g0 + __popc(bg & lower), e = e0 + __popc(be & lower);
                if (isg || (ise && e < need)) take(g + min(e, need), base + j);
                g0 += __popc(bg);
                e0 += __popc(be);
            }
            if (C > 1) mq_cluster_sync();           // the others are done with this block's counts
        }
    }
}

// dst apart from src: a block moves some whole rows of a sequence (all heads), 16 bytes of k and of v at a time.
// (evict of 256 heads: two units a thread 64.6 us, four 67.5, one 62.7, one and 512 threads 63.5)
constexpr int kMoveThreads = 256, kMoveUnits = 1;
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const Move a) {
    mq_grid_release();
    mq_grid_wait();
    const int b = a.by_blocks.of(blockIdx.x), j0 = (blockIdx.x - b * a.by_blocks.d) * a.rows;
    const int kept = min(min(max(a.len[b], 0), a.cap), a.keep);   // the same after len_out is written over len
    if (j0 == 0 && threadIdx.x == 0) a.len_out[b] = kept;
    if (j0 >= kept) return;
    const int units = min(a.rows, kept - j0) * a.by_row.d;
    const int32_t* index = a.index + (long long)b * a.heads * a.dst_cap + j0;
    for (int w0 = threadIdx.x; w0 < units; w0 += kMoveUnits * kMoveThreads) {
        uint4 x[kMoveUnits], y[kMoveUnits];
        long long to[kMoveUnits];
#pragma unroll
        for (int u = 0; u < kMoveUnits; ++u) {
            const int w = w0 + u * kMoveThreads;
            if (w >= units) continue;
            const int j = a.by_row.of(w), r = w - j * a.by_row.d, h = a.by_chunks.of(r), c = r - h * a.by_chunks.d;
            const long long from = b * a.ss + index[(long long)h * a.dst_cap + j] * a.sr + h * a.sh + c;
            to[u] = b * a.ds + (j0 + j) * a.dr + h * a.dh + c;
            x[u] = __ldcs(a.k + from);
            y[u] = __ldcs(a.v + from);
        }
#pragma unroll
        for (int u = 0; u < kMoveUnits; ++u)
            if (w0 + u * kMoveThreads < units) {
                __stcs(a.dk + to[u], x[u]);
                __stcs(a.dv + to[u], y[u]);
            }
    }
}

// In place: rows only move down (index[j] >= j), so a block that takes one head's rows in order may
// read a stretch of them, then write it: what it overwrites was read before. what0: the first of
// k (0), v (1) and scores (2) that the grid's y axis counts from.
constexpr int kInThreads = 512, kInRows = 8;

__global__ void __launch_bounds__(kInThreads) evict_in_place_kernel(const Move a, int what0) {
    mq_grid_release();
    mq_grid_wait();
    const int row = blockIdx.x;                       // sequence and head
    const long long b = row / a.heads;
    const int h = row - (int)b * a.heads;
    const int what = what0 + blockIdx.y;
    const int32_t* idx = a.index + (long long)row * a.dst_cap;
    const int kept = min(min(max(a.len[b], 0), a.cap), a.keep);   // the same after len_out is written over len
    if (what == 2) {
        const float* sc = a.score + (long long)row * a.cap;
        float* so = a.score_out + (long long)row * a.dst_cap;
        for (int j0 = 0; j0 < a.dst_cap; j0 += kInThreads) {
            const int j = j0 + threadIdx.x;
            const float x = j < kept ? mq_ld_dep(sc + idx[j]) : 0.0f;
            __syncthreads();
            if (j < a.dst_cap) so[j] = x;
            __syncthreads();
        }
        return;
    }
    uint4* p = (what == 0 ? a.dk : a.dv) + b * a.ss + h * a.sh;
    const int c = threadIdx.x % a.chunks, rt = threadIdx.x / a.chunks, per = kInThreads / a.chunks;
    for (int j0 = 0; j0 < kept; j0 += per * kInRows) {
        uint4 x[kInRows];
        bool move[kInRows];
#pragma unroll
        for (int u = 0; u < kInRows; ++u) {
            const int j = j0 + u * per + rt;
            const int at = j < kept && rt < per ? idx[j] : j;
            move[u] = at != j;
            if (move[u]) x[u] = p[at * a.sr + c];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kInRows; ++u)
            if (move[u]) p[(long long)(j0 + u * per + rt) * a.sr + c] = x[u];
        __syncthreads();
    }
}

// len_out after every block has read len (len_out may be len).
__global__ void __launch_bounds__(256) evict_len_kernel(const int32_t* len, int32_t* len_out, int n, int cap, int keep) {
    mq_grid_release();
    mq_grid_wait();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) len_out[i] = min(min(max(len[i], 0), cap), keep);
}

int launch_select(const Move& a, int recent, int C, int held, int32_t* index, unsigned rows, size_t smem,
                  cudaStream_t stream) {
    // more rows than SMs: blocks of 512 threads, two of which an SM holds (of 1024 one: 256 heads 71 us, not 64)
    const int threads = a.cap <= kBrief ? 256 : rows * C > (unsigned)mq::num_sms() ? 512 : 1024;
    auto kern = threads == 256 ? evict_select_kernel<256> : threads == 512 ? evict_select_kernel<512> : evict_select_kernel<1024>;
    if (!mq::allow_smem(reinterpret_cast<const void*>(kern), kMaxKeys * (int)sizeof(uint32_t))) return MQ_ERR_LAUNCH;
    return mq::launch_cluster(kern, dim3(C), dim3(rows * C), dim3(threads), smem, stream, a, recent, C, held, index);
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

}  // namespace

extern "C" int mq_kv_evict(const mq_kv* src, const int32_t* len, const float* score, int keep, int recent,
                           const mq_kv* dst, int32_t* len_out, float* score_out, int32_t* index,
                           cudaStream_t stream) {
    int rc = mq::check_kv(src, true);
    if (rc == MQ_OK) rc = mq::check_kv(dst, true);
    if (rc != MQ_OK) return rc;
    if (src->type != dst->type) return MQ_ERR_TYPE;
    if (src->n != dst->n || src->heads != dst->heads || src->dim != dst->dim || recent < 0 || recent > keep ||
        dst->cap < keep || src->cap > kMostRows || dst->cap > kMostRows)
        return MQ_ERR_SHAPE;
    if (src->n == 0) return MQ_OK;
    if (!len || !len_out || (src->cap > 0 && !score) || (dst->cap > 0 && !index)) return MQ_ERR_NULL;
    if (!mq::aligned16(len) || !mq::aligned16(len_out) || !mq::aligned16(score) || !mq::aligned16(score_out) ||
        !mq::aligned16(index))
        return MQ_ERR_ALIGN;
    const long long rows = (long long)src->n * src->heads;
    if (rows > 0x7fffffffLL || (long long)src->heads * (src->dim / 8) > 0x3fffffffLL) return MQ_ERR_SHAPE;
    bool in_place = false;
    if (src->cap > 0 && dst->cap > 0) {
        in_place = src->k == dst->k && src->v == dst->v && src->cap == dst->cap && src->seq_stride == dst->seq_stride &&
                   src->row_stride == dst->row_stride && src->head_stride == dst->head_stride;
        const size_t sn = (size_t)mq::kv_span(src) * 2, dn = (size_t)mq::kv_span(dst) * 2;
        if (!in_place && (overlap(src->k, sn, dst->k, dn) || overlap(src->v, sn, dst->v, dn) ||
                          overlap(src->k, sn, dst->v, dn) || overlap(src->v, sn, dst->k, dn)))
            return MQ_ERR_SHAPE;
        if (score_out && !(score_out == score && src->cap == dst->cap) &&
            overlap(score, (size_t)rows * src->cap * 4, score_out, (size_t)rows * dst->cap * 4))
            return MQ_ERR_SHAPE;
    }
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    Move a;
    a.k = static_cast<const uint4*>(src->k);
    a.v = static_cast<const uint4*>(src->v);
    a.dk = static_cast<uint4*>(dst->k);
    a.dv = static_cast<uint4*>(dst->v);
    a.score = score;
    a.score_out = score_out;
    a.index = index;
    a.len = len;
    a.len_out = len_out;
    a.ss = src->seq_stride / 8;
    a.sr = src->row_stride / 8;
    a.sh = src->head_stride / 8;
    a.ds = dst->seq_stride / 8;
    a.dr = dst->row_stride / 8;
    a.dh = dst->head_stride / 8;
    a.n = src->n;
    a.heads = src->heads;
    a.cap = src->cap;
    a.dst_cap = dst->cap;
    a.keep = keep;
    a.chunks = src->dim / 8;
    if (dst->cap > 0) {
        const bool ordered_score = score_out && score_out == score;   // they move down as rows in place do
        // a block for each 4096 scores of a head (measured: with fewer the rounds over them take longer, with more their
        // meetings), as long as the GPU holds them all at once
        int C = 1;
        while (C < kMaxCluster && src->cap > 4096 * C && rows * C * 2 <= mq::num_sms()) C *= 2;
        const int per = (src->cap + C - 1) / C + 32;
        const int held = per < kMaxKeys ? per : kMaxKeys;
        const size_t smem = (size_t)held * sizeof(uint32_t);
        if (ordered_score) a.score_out = nullptr;
        rc = launch_select(a, recent, C, held, index, (unsigned)rows, smem, stream);
        if (rc != MQ_OK) return rc;
        a.score_out = score_out;
        if (!in_place) {
            const int row = a.heads * a.chunks;
            const long long full = keep < src->cap ? keep : src->cap;
            a.rows = kMoveUnits * kMoveThreads / row > 0 ? kMoveUnits * kMoveThreads / row : 1;
            const long long each = full > 0 ? (full + a.rows - 1) / a.rows : 1, blocks = each * a.n;   // (one for len_out)
            if (blocks > 0x7fffffffLL) return MQ_ERR_SHAPE;
            a.by_blocks = mq::div_by((int)each);
            a.by_row = mq::div_by(row);
            a.by_chunks = mq::div_by(a.chunks);
            rc = mq::launch_pdl(evict_move_kernel, dim3((unsigned)blocks), dim3(kMoveThreads), 0, stream, a);
            if (rc != MQ_OK) return rc;
        }
        if (in_place || ordered_score) {
            const int what0 = in_place ? 0 : 2, count = (ordered_score ? 3 : 2) - what0;
            rc = mq::launch_pdl(evict_in_place_kernel, dim3((unsigned)rows, count), dim3(kInThreads), 0, stream, a,
                                what0);
            if (rc != MQ_OK) return rc;
        }
        if (!in_place) return MQ_OK;
    }
    return mq::launch_pdl(evict_len_kernel, dim3((a.n + 255) / 256), dim3(256), 0, stream, len, len_out, a.n, a.cap,
                          keep);
}
