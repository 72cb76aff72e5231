// Pages of caches: from one generation of sequences to the next (fork, trim, free, reserve with copy on write), and
// the pool closed up.
//
// Tables and lengths are on the device and stay there, so a serving loop can be captured. Who holds a page is counted
// from the tables themselves at every call: there is no count beside them that could disagree with them. A call is two launches.
// The first is one cluster of eight blocks, whose barriers (about a microsecond each) stand between counting, scanning and
// writing where a launch each would take two or three times that; the tables of a whole pool of 80000 pages are
// some hundred entries a thread. The second, as wide as the GPU, copies what the first has listed. A copy's
// source is a page that stays, its target one that nobody holds, so copies in any order are right.
// (4, 8 and 16 blocks: 16 beams 13.6, 14.7, 17.9 us; 256 sequences 25.2, 18.5, 18.7, whose counts are scattered.)
// Bound: the tables' part by the latency of some six barriers, copies by HBM.

#include "heads.cuh"

namespace pages {
namespace {

constexpr int kThreads = 1024, kBlocks = 8, kAll = kThreads * kBlocks;
constexpr int kChunk = 128;      // table entries of a row that a warp takes at once, four a lane

struct Space {                   // of the workspace
    int32_t* tmp;                // [m][width] kept entries
    int32_t* info;               // [m][4]: rows kept, rows added, first new page's rank, copies (0, 1)
    int32_t* held;               // [P] entries that name the page (compaction: whether any does)
    int32_t* writers;            // [P] sequences that go on inside it
    int32_t* first;              // [P] the first of them
    int32_t* free;               // [P] pages that nobody holds, in order
    int2* copies;                // [max(m, P)] page to page
    int32_t* count;              // of copies; 4 numbers
    size_t bytes;
};
Space space_of(uint8_t* ws, long long m, long long width, long long P) {
    Space s;
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t* p = ws + at;
        at += (n + 15) & ~(size_t)15;
        return p;
    };
    s.tmp = reinterpret_cast<int32_t*>(take(4 * (size_t)(m * width)));
    s.info = reinterpret_cast<int32_t*>(take(16 * (size_t)m));
    s.held = reinterpret_cast<int32_t*>(take(4 * (size_t)P));
    s.writers = reinterpret_cast<int32_t*>(take(4 * (size_t)P));
    s.first = reinterpret_cast<int32_t*>(take(4 * (size_t)P));
    s.free = reinterpret_cast<int32_t*>(take(4 * (size_t)P));
    s.copies = reinterpret_cast<int2*>(take(8 * (size_t)(m > P ? m : P)));
    s.count = reinterpret_cast<int32_t*>(take(16));
    s.bytes = at;
    return s;
}

// Sums of n numbers a thread over the cluster, in thread order: x becomes this thread's sum before it, all the whole. Once in a kernel; a
// barrier of the whole cluster has to follow before a block ends.
template <int n>
__device__ __forceinline__ void scan(int (&x)[n], int (&all)[n]) {
    __shared__ int s_warp[n][32], s_block[n];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int upto[n];
#pragma unroll
    for (int k = 0; k < n; ++k) {
        upto[k] = x[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto[k], o);
            if (lane >= o) upto[k] += y;
        }
        if (lane == 31) s_warp[k][wid] = upto[k];
    }
    __syncthreads();
    if (wid < n) {
        int y = s_warp[wid][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s_warp[wid][lane] = y;
        if (lane == 31) s_block[wid] = y;
    }
    mq_cluster_sync();
    const int rank = (int)mq_cluster_rank();
#pragma unroll
    for (int k = 0; k < n; ++k) {
        x[k] = upto[k] - x[k] + (wid > 0 ? s_warp[k][wid - 1] : 0);
        all[k] = 0;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int y = mq_remote(s_block + k, i);
            if (i < rank) x[k] += y;
            all[k] += y;
        }
    }
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }

// The pages of a warp: `steps` times 32 of them, in order.
struct Pages {
    int first, end, steps;
    __device__ __forceinline__ Pages(int P, int id) {
        steps = ceil_div(ceil_div(P, 32), kAll / 32);
        const long long at = (long long)(id >> 5) * steps * 32;
        first = (int)(at < P ? at : P);
        end = (int)(at + steps * 32 < P ? at + steps * 32 : P);
    }
    // Which of them the test holds for: lane i has those of step i (of the first 32 steps); lane 0's count is the warp's.
    template <typename F>
    __device__ __forceinline__ uint32_t read(const int32_t* held, F test, int& count) const {
        const int lane = threadIdx.x & 31;
        uint32_t mine = 0;
        int n = 0;
        for (int k0 = 0; k0 < steps; k0 += 4) {
            int x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int p = first + (k0 + k) * 32 + lane;
                x[k] = k0 + k < steps && p < end ? __ldcg(held + p) : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t b = __ballot_sync(0xffffffffu, x[k] >= 0 && test(x[k]));
                n += __popc(b);
                if (lane == k0 + k) mine = b;
            }
        }
        count = lane == 0 ? n : 0;
        return mine;
    }
    // f(page, whether the test holds, how many before it do) for each.
    template <typename F, typename G>
    __device__ __forceinline__ void each(const int32_t* held, uint32_t mine, int before, F test, G f) const {
        const int lane = threadIdx.x & 31;
        for (int k = 0; k < steps; ++k) {
            const int p = first + k * 32 + lane;
            const uint32_t b = k < 32 ? __shfl_sync(0xffffffffu, mine, k) : __ballot_sync(0xffffffffu, p < end && test(__ldcg(held + p)));
            if (p < end) f(p, b >> lane & 1, before + __popc(b & ((1u << lane) - 1)));
            before += __popc(b);
        }
    }
};

struct NextArgs {
    const int32_t *table, *len, *from, *keep, *add;
    int32_t *table_out, *len_out, *status;
    Space s;
    int n, m, width, P, R;
};

__global__ void __launch_bounds__(kThreads) next_kernel(const NextArgs a) {
    mq_grid_release();
    mq_grid_wait();
    const int id = (int)mq_cluster_rank() * kThreads + threadIdx.x, lane = threadIdx.x & 31;
    for (int p = id; p < a.P; p += kAll) {
        a.s.held[p] = a.s.writers[p] = 0;
        a.s.first[p] = 0x7fffffff;
    }
    if (id == 0) a.s.count[0] = 0;
    int longs = 0;
    for (int b = id; b < a.m; b += kAll) {
        const int f = a.from ? __ldca(a.from + b) : b;
        int L = (unsigned)f < (unsigned)a.n ? min(max(__ldca(a.len + f), 0), a.width * a.R) : 0;
        if (a.keep) L = min(L, max(__ldca(a.keep + b), 0));
        int add = a.add ? max(__ldca(a.add + b), 0) : 0;
        if (add > a.width * a.R - L) {
            add = 0;
            ++longs;
        }
        reinterpret_cast<int2*>(a.s.info)[2 * b] = make_int2(L, add);
    }
    mq_cluster_sync();
    // who holds each page, and who goes on inside it
    const int chunks = ceil_div(a.width, kChunk);
    for (long long u = id >> 5; u < (long long)a.m * chunks; u += kAll / 32) {
        const int b = (int)(u / chunks), i0 = (int)(u - (long long)b * chunks) * kChunk;
        const int f = a.from ? __ldca(a.from + b) : b;
        const int2 x = __ldcg(reinterpret_cast<const int2*>(a.s.info) + 2 * b);
        const int kept = ceil_div(x.x, a.R);
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k + lane;
            e[k] = i < kept ? __ldca(a.table + (long long)f * a.width + i) : -1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k + lane;
            if ((unsigned)e[k] < (unsigned)a.P) {
                atomicAdd(a.s.held + e[k], 1);
                if (i == kept - 1 && x.y > 0 && x.x % a.R != 0) {
                    atomicAdd(a.s.writers + e[k], 1);
                    atomicMin(a.s.first + e[k], b);
                }
            }
            if (i < a.width) a.s.tmp[(long long)b * a.width + i] = e[k];
        }
    }
    mq_cluster_sync();
    // pages wanted, in the sequences' order; pages that nobody holds, in theirs
    const int bs = ceil_div(a.m, kAll), b0 = min(id * (long long)bs, (long long)a.m), b1 = min(b0 + bs, a.m);
    int want = 0, none;
    for (int b = b0; b < b1; ++b) {
        const int2 x = __ldcg(reinterpret_cast<const int2*>(a.s.info) + 2 * b);
        const int kept = ceil_div(x.x, a.R);
        int copy = 0;
        if (x.y > 0 && x.x % a.R != 0) {
            const int e = __ldcg(a.s.tmp + (long long)b * a.width + kept - 1);
            if ((unsigned)e < (unsigned)a.P) {
                const int h = __ldcg(a.s.held + e), writers = __ldcg(a.s.writers + e), first = __ldcg(a.s.first + e);
                copy = h > 1 && !(writers == h && first == b);
            }
        }
        const int n = copy + ceil_div(x.x + x.y, a.R) - kept;
        reinterpret_cast<int2*>(a.s.info)[2 * b + 1] = make_int2(n, copy);
        want += n;
    }
    const Pages of(a.P, id);
    uint32_t empty = of.read(a.s.held, [&](int held) { return held == 0; }, none);
    int before[3] = {want, none, longs}, all[3];
    scan(before, all);
    const bool enough = all[0] <= all[1];
    int rank = before[0];
    for (int b = b0; b < b1; ++b) {
        int4 x = __ldcg(reinterpret_cast<const int4*>(a.s.info) + b);
        a.len_out[b] = enough ? x.x + x.y : x.x;
        const int n = x.z;
        a.s.info[4 * b + 2] = rank;
        rank += n;
    }
    of.each(a.s.held, empty, __shfl_sync(0xffffffffu, before[1], 0), [&](int held) { return held == 0; },
            [&](int p, bool is, int at) {
                if (is) a.s.free[at] = p;
            });
    if (id == 0) {
        a.status[0] = enough ? 0 : all[0] - all[1];
        a.status[1] = enough ? all[1] - all[0] : all[1];
        a.status[2] = all[2];
    }
    mq_cluster_sync();
    for (long long u = id >> 5; u < (long long)a.m * chunks; u += kAll / 32) {
        const int b = (int)(u / chunks), i0 = (int)(u - (long long)b * chunks) * kChunk;
        const int4 x = __ldcg(reinterpret_cast<const int4*>(a.s.info) + b);
        const int kept = ceil_div(x.x, a.R), first = kept - x.w, end = ceil_div(x.x + x.y, a.R);
        int e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k + lane;
            e[k] = i < a.width ? __ldcg(a.s.tmp + (long long)b * a.width + i) : -1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 32 * k + lane;
            if (enough && i >= first && i < end) {
                const int to = __ldcg(a.s.free + x.z + i - first);
                if (i < kept) a.s.copies[atomicAdd(a.s.count, 1)] = make_int2(e[k], to);
                e[k] = to;
            }
            if (i < a.width) a.table_out[(long long)b * a.width + i] = e[k];
        }
    }
}

struct CompactArgs {
    const int32_t *table, *len;
    int32_t *table_out, *where, *live;
    Space s;
    int n, width, P, R;
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
    mq_grid_release();
    mq_grid_wait();
    const int id = (int)mq_cluster_rank() * kThreads + threadIdx.x, lane = threadIdx.x & 31;
    for (int p = id; p < a.P; p += kAll) a.s.held[p] = 0;
    mq_cluster_sync();
    const int chunks = ceil_div(a.width, kChunk);
    auto rows = [&](auto load, auto f) {     // every entry: its place, and what it is if its sequence holds rows there
        for (long long u = id >> 5; u < (long long)a.n * chunks; u += kAll / 32) {
            const int b = (int)(u / chunks), i0 = (int)(u - (long long)b * chunks) * kChunk;
            const int used = ceil_div(min(max(__ldca(a.len + b), 0), a.width * a.R), a.R);
            int e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + 32 * k + lane;
                e[k] = i < used ? load((long long)b * a.width + i) : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + 32 * k + lane;
                if (i < a.width) f((long long)b * a.width + i, e[k]);
            }
        }
    };
    rows([&](long long at) { return __ldca(a.table + at); },
         [&](long long, int e) {
             if ((unsigned)e < (unsigned)a.P) a.s.held[e] = 1;
         });
    mq_cluster_sync();
    const Pages of(a.P, id);
    auto is_live = [](int held) { return held != 0; };
    int first[1], all[1];
    const uint32_t lives = of.read(a.s.held, is_live, first[0]);
    scan(first, all);
    const int U = all[0], before = __shfl_sync(0xffffffffu, first[0], 0);
    // places below U that are free, in order; live pages before page U
    of.each(a.s.held, lives, before, is_live, [&](int p, bool is, int at) {
        if (p == U) a.s.count[1] = at;
        if (!is && p < U) a.s.free[p - at] = p;
    });
    if (id == 0) {
        if (U == a.P) a.s.count[1] = U;
        a.live[0] = U;
    }
    mq_cluster_sync();
    const int below = __ldcg(a.s.count + 1);
    if (id == 0) a.s.count[0] = U - below;
    of.each(a.s.held, lives, before, is_live, [&](int p, bool is, int at) {
        int to = is ? p : -1;
        if (is && p >= U) {
            to = __ldcg(a.s.free + at - below);
            a.s.copies[at - below] = make_int2(p, to);
        }
        a.where[p] = to;
    });
    mq_cluster_sync();
    rows(
        [&](long long at) {
            const int e = __ldca(a.table + at);
            return (unsigned)e < (unsigned)a.P ? __ldcg(a.where + e) : e;
        },
        [&](long long at, int e) { a.table_out[at] = e; });
}

// ---------------------------------------------------------------------------------------------- copies

constexpr int kCopyThreads = 256, kAtOnce = 4;
constexpr int kPart = kCopyThreads * kAtOnce * 16;      // bytes that a block moves at once

struct CopyArgs {
    uint8_t* data;
    long long page_stride, layer_stride, page_bytes;
    const int2* copies;
    const int32_t* count;
    int layers, parts;
};
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyArgs a) {
    mq_grid_release();
    mq_grid_wait();
    const long long units = (long long)__ldca(a.count) * a.layers * a.parts;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long cl = u / a.parts;
        const int part = (int)(u - cl * a.parts);
        const int2 c = __ldca(a.copies + cl / a.layers);
        uint8_t* layer = a.data + (cl % a.layers) * a.layer_stride;
        const uint4* src = reinterpret_cast<const uint4*>(layer + c.x * a.page_stride);
        uint4* dst = reinterpret_cast<uint4*>(layer + c.y * a.page_stride);
        const long long i0 = (long long)part * (kPart / 16) + threadIdx.x, end = a.page_bytes / 16;
        uint4 x[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (i0 + k * kCopyThreads < end) x[k] = __ldcs(src + i0 + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (i0 + k * kCopyThreads < end) __stcs(dst + i0 + k * kCopyThreads, x[k]);
    }
}

// per_sm: blocks an SM at most. Blocks that take turns on an SM leave it to the scheduler where there is room: 1.6 GB of pages moved
// with 8 an SM (all resident) 266 us, 64: 247.
int launch_copies(const mq_pool* pool, const Space& s, long long most, int per_sm, cudaStream_t stream) {
    CopyArgs a;
    a.data = static_cast<uint8_t*>(pool->data);
    a.page_stride = pool->page_stride;
    a.layer_stride = pool->layers > 1 ? pool->layer_stride : 0;
    a.page_bytes = pool->page_bytes;
    a.copies = s.copies;
    a.count = s.count;
    a.layers = pool->layers;
    a.parts = (int)((pool->page_bytes + kPart - 1) / kPart);
    const long long units = most * pool->layers * a.parts, held = (long long)per_sm * mq::num_sms();
    if (units == 0) return MQ_OK;
    return mq::launch_pdl(copy_kernel, dim3((unsigned)(units < held ? units : held)), dim3(kCopyThreads), 0, stream, a);
}

int check_pool(const mq_pool* p, bool pointers) {
    if (!p) return MQ_ERR_NULL;
    if (p->layers < 1 || p->n_pages < 0 || p->n_pages > (1 << 28) || p->page_rows < 1 || p->page_bytes < 16 || p->page_bytes % 16 != 0 ||
        p->page_bytes > (1LL << 30) || p->page_stride % 16 != 0 || p->page_stride < 0 || p->page_stride > (1LL << 40))
        return MQ_ERR_SHAPE;
    if (p->layers > 1 && (p->layer_stride % 16 != 0 || p->layer_stride < 0 || p->layer_stride > (1LL << 40) || p->layers > (1 << 20)))
        return MQ_ERR_SHAPE;
    // all pages apart: layers of pages, or pages of layers
    const long long inner = p->page_stride * (p->n_pages > 0 ? p->n_pages - 1 : 0) + p->page_bytes;
    const bool by_layer = (p->n_pages <= 1 || p->page_stride >= p->page_bytes) && (p->layers == 1 || p->layer_stride >= inner);
    const bool by_page = p->layers > 1 && p->layer_stride >= p->page_bytes &&
                         (p->n_pages <= 1 || p->page_stride >= p->layer_stride * (p->layers - 1) + p->page_bytes);
    if (!by_layer && !by_page) return MQ_ERR_SHAPE;
    if (pointers && p->n_pages > 0) {
        if (!p->data) return MQ_ERR_NULL;
        if (!mq::aligned16(p->data)) return MQ_ERR_ALIGN;
    }
    return MQ_OK;
}

bool valid_table(long long n, long long width, int page_rows) {
    return n >= 0 && width >= 0 && n * (width + 1) <= 0x7fffffffLL && n <= (1 << 28) && width * page_rows <= 0x7fffffffLL;
}

// A range of bytes that a call writes or reads.
struct Bytes {
    const void* p;
    long long n;
    bool meets(const Bytes& b) const { return mq::rows_meet(p, 1, n, n, b.p, b.n); }
};
bool meets_pool(const mq_pool* p, const Bytes& b) {
    if (p->n_pages == 0) return false;
    const long long step = p->n_pages > 1 ? p->page_stride : p->page_bytes, next = p->layers > 1 ? p->layer_stride : 0;
    const uint8_t* data = static_cast<const uint8_t*>(p->data);
    if (!b.meets({data, next * (p->layers - 1) + step * (p->n_pages - 1) + p->page_bytes})) return false;
    for (int i = 0; i < p->layers; ++i)      // (between pages of one layer may lie other things)
        if (mq::rows_meet(data + i * next, p->n_pages, step, p->page_bytes, b.p, b.n)) return true;
    return false;
}
// What is written lies apart from all else and from the pool, but that written[i] may be read[i] for the first `in_place` of
// them (the new tables go through the workspace, a sequence's old length is read before its new one is written).
template <int W, int R>
bool apart(const mq_pool* pool, const Bytes (&written)[W], const Bytes (&read)[R], int in_place) {
    for (int i = 0; i < W; ++i) {
        if (meets_pool(pool, written[i])) return false;
        for (int j = 0; j < i; ++j)
            if (written[i].meets(written[j])) return false;
        for (int j = 0; j < R; ++j)
            if (written[i].meets(read[j]) && !(i == j && i < in_place && written[i].p == read[j].p)) return false;
    }
    for (const Bytes& b : read)
        if (meets_pool(pool, b)) return false;
    return true;
}

template <typename Args>
int launch_tables(void (*kern)(Args), const Args& a, cudaStream_t stream) {
    return mq::launch_cluster(kern, dim3(kBlocks), dim3(kBlocks), dim3(kThreads), 0, stream, a);
}

}  // namespace
}  // namespace pages

extern "C" size_t mq_pages_ws_bytes(const mq_pool* pool, int n, int width) {
    using namespace pages;
    if (check_pool(pool, false) != MQ_OK || !valid_table(n, width, pool->page_rows)) return 0;
    return space_of(nullptr, n, width, pool->n_pages).bytes;
}

extern "C" int mq_pages_next(const mq_pool* pool, const int32_t* table, const int32_t* len, int n, int width, const int32_t* from,
                             const int32_t* keep, const int32_t* add, int32_t* table_out, int32_t* len_out, int m, int32_t* status,
                             void* ws, size_t ws_bytes, cudaStream_t stream) {
    using namespace pages;
    int rc = check_pool(pool, true);
    if (rc != MQ_OK) return rc;
    if (!valid_table(n, width, pool->page_rows) || !valid_table(m, width, pool->page_rows) || (!from && m > 0 && n != m))
        return MQ_ERR_SHAPE;
    if (!status || !ws) return MQ_ERR_NULL;
    if ((n > 0 && (!len || (width > 0 && !table))) || (m > 0 && (!len_out || (width > 0 && !table_out)))) return MQ_ERR_NULL;
    for (const void* p : {(const void*)table, (const void*)len, (const void*)from, (const void*)keep, (const void*)add,
                          (const void*)table_out, (const void*)len_out, (const void*)status, (const void*)ws})
        if (!mq::aligned16(p)) return MQ_ERR_ALIGN;
    const long long used = (long long)mq_pages_ws_bytes(pool, m, width);
    if (ws_bytes < (size_t)used) return MQ_ERR_SCRATCH;
    const Bytes written[] = {{table_out, 4LL * m * width}, {len_out, 4LL * m}, {status, 12}, {ws, used}};
    const Bytes read[] = {{table, 4LL * n * width}, {len, 4LL * n}, {from, 4LL * m}, {keep, 4LL * m}, {add, 4LL * m}};
    if (!apart(pool, written, read, 2)) return MQ_ERR_SHAPE;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    const Space s = space_of(static_cast<uint8_t*>(ws), m, width, pool->n_pages);
    const NextArgs a = {table, len, from, keep, add, table_out, len_out, status, s, n, m, width, pool->n_pages, pool->page_rows};
    rc = launch_tables(next_kernel, a, stream);
    return rc != MQ_OK || !add ? rc : launch_copies(pool, s, m, 16, stream);
}

extern "C" int mq_pages_compact(const mq_pool* pool, const int32_t* table, const int32_t* len, int n, int width, int32_t* table_out,
                                int32_t* where, int32_t* live, void* ws, size_t ws_bytes, cudaStream_t stream) {
    using namespace pages;
    int rc = check_pool(pool, true);
    if (rc != MQ_OK) return rc;
    if (!valid_table(n, width, pool->page_rows)) return MQ_ERR_SHAPE;
    if (!live || !ws || (pool->n_pages > 0 && !where)) return MQ_ERR_NULL;
    if (n > 0 && (!len || (width > 0 && (!table || !table_out)))) return MQ_ERR_NULL;
    for (const void* p : {(const void*)table, (const void*)len, (const void*)table_out, (const void*)where, (const void*)live, (const void*)ws})
        if (!mq::aligned16(p)) return MQ_ERR_ALIGN;
    const long long used = (long long)mq_pages_ws_bytes(pool, n, width);
    if (ws_bytes < (size_t)used) return MQ_ERR_SCRATCH;
    const Bytes written[] = {{table_out, 4LL * n * width}, {where, 4LL * pool->n_pages}, {live, 4}, {ws, used}};
    const Bytes read[] = {{table, 4LL * n * width}, {len, 4LL * n}};
    if (!apart(pool, written, read, 1)) return MQ_ERR_SHAPE;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    const Space s = space_of(static_cast<uint8_t*>(ws), n, width, pool->n_pages);
    const CompactArgs a = {table, len, table_out, where, live, s, n, width, pool->n_pages, pool->page_rows};
    rc = launch_tables(compact_kernel, a, stream);
    if (rc != MQ_OK) return rc;
    const long long most = (long long)n * width < pool->n_pages ? (long long)n * width : pool->n_pages;
    return launch_copies(pool, s, most, 64, stream);
}
