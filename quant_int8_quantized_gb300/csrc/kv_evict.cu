// Eviction from a cache by accumulated attention weight: per sequence and key head the `recent`
// last rows stay and, of the others, those with the largest score; kept rows keep their order.
//
// Two launches. The first finds the kept rows: scores become unsigned keys in the same order, the
// key of the last row that is kept is found digit by digit (a histogram of 8 bits a round, counted in
// shared memory), then every warp of the block writes the kept rows of its own stretch in order,
// from the counts of the stretches before it. Counts are integers: the result does not depend on
// the order of the atomics. The second moves rows, values and scores: 16 bytes a thread, every
// kept row read once and written once.

#include "heads.cuh"

namespace {

constexpr int kSelThreads = 1024;
constexpr int kWarps = kSelThreads / 32;

// Order of floats as unsigned integers; -0 equals +0, NaN is below everything.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0u;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const float* score, const int32_t* len, int heads,
                                                                   int cap, int keep, int recent, int dst_cap,
                                                                   int32_t* index) {
    __shared__ int s_hist[kWarps][256];
    __shared__ int s_tot[256];
    __shared__ int s_gt[kWarps], s_eq[kWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int s_need;
    mq_grid_release();
    mq_grid_wait();
    const int row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int n = min(max(len[row / heads], 0), cap);
    const float* sc = score + (long long)row * cap;
    int32_t* out = index + (long long)row * dst_cap;
    if (n <= keep) {
        for (int j = tid; j < dst_cap; j += kSelThreads) out[j] = j < n ? j : -1;
        return;
    }
    const int cand = n - recent;            // rows that compete for `best` places
    const int best = keep - recent;
    for (int j = tid; j < recent; j += kSelThreads) out[best + j] = cand + j;
    for (int j = keep + tid; j < dst_cap; j += kSelThreads) out[j] = -1;
    if (best == 0) return;
    uint32_t prefix = 0;
    int need = best;                        // rows still to be taken among those that share `prefix`
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = lane; i < 256; i += 32) s_hist[wid][i] = 0;
        __syncwarp();
        const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int j = tid; j < cand; j += kSelThreads) {
            const uint32_t k = order_key(mq_ld_dep(sc + j));
            if ((k & above) == prefix) atomicAdd(&s_hist[wid][(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (tid < 256) {
            int t = 0;
            for (int w = 0; w < kWarps; ++w) t += s_hist[w][tid];
            s_tot[tid] = t;
        }
        __syncthreads();
        if (wid == 0) {                      // the digit at which the rows from the top reach `need`
            int t[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += t[i] = s_tot[255 - (lane * 8 + i)];
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
                        break;
                    }
                    before += t[i];
                }
            }
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
        __syncthreads();
    }
    // kept: key above `prefix`, and the first `need` rows of those equal to it
    const int per = ((cand + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int j0 = min(wid * per, cand), j1 = min(j0 + per, cand);
    int gt = 0, eq = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
        const uint32_t k = order_key(mq_ld_dep(sc + j));
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
    int g0 = 0, e0 = 0;
    for (int w = 0; w < wid; ++w) {
        g0 += s_gt[w];
        e0 += s_eq[w];
    }
    for (int j = j0; j < j1; j += 32) {
        const uint32_t k = j + lane < j1 ? order_key(mq_ld_dep(sc + j + lane)) : 0u;
        const bool isg = j + lane < j1 && k > prefix, ise = j + lane < j1 && k == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, isg), be = __ballot_sync(0xffffffffu, ise);
        const unsigned lower = (1u << lane) - 1u;
        const int g = g0 + __popc(bg & lower), e = e0 + __popc(be & lower);
        if (isg || (ise && e < need)) out[g + min(e, need)] = j + lane;
        g0 += __popc(bg);
        e0 += __popc(be);
    }
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
};

// dst apart from src: one thread per 16 bytes of a kept row of k and of v.
__global__ void __launch_bounds__(256) evict_move_kernel(const Move a) {
    mq_grid_release();
    mq_grid_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i < a.n) {
        const int L = min(max(a.len[i], 0), a.cap);
        a.len_out[i] = min(L, a.keep);
    }
    const long long scores = (long long)a.n * a.heads * a.dst_cap;
    if (a.score_out)
        for (long long s = i; s < scores; s += (long long)gridDim.x * 256) {
            const int at = a.index[s];
            a.score_out[s] = at < 0 ? 0.0f : a.score[s / a.dst_cap * a.cap + at];
        }
    if (a.keep == 0) return;
    const int c = (int)(i % a.chunks);
    long long r = i / a.chunks;
    const int h = (int)(r % a.heads);
    r /= a.heads;
    const int j = (int)(r % a.keep);
    const long long b = r / a.keep;
    if (b >= a.n) return;
    const int at = a.index[(b * a.heads + h) * a.dst_cap + j];
    if (at < 0) return;
    const long long from = b * a.ss + at * a.sr + h * a.sh + c, to = b * a.ds + j * a.dr + h * a.dh + c;
    const uint4 x = __ldcs(a.k + from), y = __ldcs(a.v + from);
    __stcs(a.dk + to, x);
    __stcs(a.dv + to, y);
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
        dst->cap < keep)
        return MQ_ERR_SHAPE;
    if (src->n == 0) return MQ_OK;
    if (!len || !len_out || (src->cap > 0 && !score) || (dst->cap > 0 && !index)) return MQ_ERR_NULL;
    if (!mq::aligned16(len) || !mq::aligned16(len_out) || !mq::aligned16(score) || !mq::aligned16(score_out) ||
        !mq::aligned16(index))
        return MQ_ERR_ALIGN;
    const long long rows = (long long)src->n * src->heads;
    if (rows > 0x7fffffffLL) return MQ_ERR_SHAPE;
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
    if (dst->cap > 0) {
        rc = mq::launch_pdl(evict_select_kernel, dim3((unsigned)rows), dim3(kSelThreads), 0, stream, score, len,
                            src->heads, src->cap, keep, recent, dst->cap, index);
        if (rc != MQ_OK) return rc;
    }
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
        // Scores that move in place, or beside rows that do, go through the ordered kernel.
        const bool ordered_score = score_out && (in_place || score_out == score);
        if (!in_place) {
            if (ordered_score) a.score_out = nullptr;
            const long long units = (long long)a.n * keep * a.heads * a.chunks;
            const long long blocks = ((units > a.n ? units : a.n) + 255) / 256;
            if (blocks > 0x7fffffffLL) return MQ_ERR_SHAPE;
            rc = mq::launch_pdl(evict_move_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
            if (rc != MQ_OK) return rc;
            a.score_out = score_out;
        }
        if (in_place || ordered_score) {
            const int what0 = in_place ? 0 : 2, count = (score_out ? 3 : 2) - what0;
            rc = mq::launch_pdl(evict_in_place_kernel, dim3((unsigned)rows, count), dim3(kInThreads), 0, stream, a,
                                what0);
            if (rc != MQ_OK) return rc;
        }
        if (!in_place) return MQ_OK;
    }
    return mq::launch_pdl(evict_len_kernel, dim3((a.n + 255) / 256), dim3(256), 0, stream, len, len_out, a.n, a.cap,
                          keep);
}
