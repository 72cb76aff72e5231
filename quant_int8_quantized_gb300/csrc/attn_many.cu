// Attention pieces for many query rows per key head, on the tensor cores (tcgen05).
//
// A segment is 256 query rows, two halves of 128 (the lanes of tensor memory), against tiles of 128 keys.
// For each half and tile: S = Q K^T (128 x 128, f32, tensor memory), a thread per row turns its row
// into probabilities (running maximum and sum in its registers), writes them back over S as 16-bit
// pairs, and O += P V with P as the left operand out of tensor memory. Both operands that come from
// shared memory are laid out by TMA with the 128-byte swizzle: K as it lies (a key's dims are
// contiguous, the product's K axis), V as it lies too (its dims are the product's N axis: the
// descriptor of the transposed kind).
//
// The halves take turns: while one half's threads work on their tile, the tensor cores do the other half's
// products (a tile of both halves and of D = 128 in 1.4 us, of which the products alone are 1.3; without the turns some
// blocks stay in step and take up to 2.1). A segment of at most 128 rows gives both halves the same rows and every other
// tile. The reference that the exponents are taken against is renewed only when a row passes the maximum behind it by 2^8
// (the sums are the same in any scale, and 2^8 does not bring a 16-bit value near its end), so O in tensor memory is hardly
// ever scaled again.
//
// 384 threads, one block per SM: warps 0-3 and 4-7 the rows of the halves, warp 8 copies (TMA), warps 9 and 10 a
// half's products each (one warp for both issued too slowly), warp 11 walks the block's run and hands its pieces
// to the others through a small ring, so that nobody else divides or reads lengths on the way. The register file is shared
// out again to give a row's thread its 128 products. Shared memory at D = 128: Q (64 KB), a ring of four K and
// V tiles (32 KB each), and 32 KB through which the rows' outputs go out whole. The next piece's Q is on its
// way as soon as the last product with this one's is done, and its first products run beside the output.
// Bound: the tensor cores. Measured: 2048 tokens of 32 heads of 128 behind 16384 keys in 342 us, 1.71 PFLOP/s; 3314 of 28 behind
// 1000 in 112 us, 1.12 PFLOP/s, where the pieces' first tiles and outputs weigh more; the same with heads of 64 in 87 us, 0.72
// PFLOP/s: half the products for as many exponentials.
// Waits are bounded; a wait that runs out is recorded (mq_device_status), the block drains its own copies
// and products, frees tensor memory and returns.

#include <map>
#include <mutex>
#include <type_traits>

#include "attn_few.cuh"
#include "attn_many.cuh"
#include "attn_maps.cuh"

namespace attn {
namespace {

__device__ unsigned int g_attn_error;   // bit 0: a bounded wait gave up
#ifdef MQ_TEST_INJECT
// Test builds only: block 0 leaves out its first tile of keys, whose barrier then never completes.
__device__ int g_test_skip_tile;
#endif

constexpr int kThreads = 384;
// Registers a thread: what the launch gives to 384 threads, and after sharing out again (2 x 208 + 88 = 3 x 168).
constexpr int kLaunchRegs = 168, kRowRegs = 208, kOtherRegs = 88;
constexpr int kHalf = kManyHalf;
constexpr int kKeys = kManyKeys;
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 8.0f;           // powers of two by which a row may pass the maximum that its reference comes from
// f16 holds weights up to 2^15 and down to 2^-24: the row's reference lies 2^7 below that maximum.
template <typename T>
constexpr int kUp = std::is_same<T, __half>::value ? 7 : 0;
// Of rows whose maxima are large (attn.cuh) the products are scaled and rounded, as the maximum itself was, before the
// reference is taken off. Otherwise one fused step does both, and what it keeps of a product past the maximum's last place is
// 2^-5 at most; from 2^28 that would be powers of two by which the weights leave their type.

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;                       // 128-byte columns of a row
    static constexpr int kChunkBytes = 128 * 128;                // 128 rows of one
    static constexpr int kTileBytes = kChunks * kChunkBytes;     // a K or V tile, a half of Q
    static constexpr int kQChunk = 2 * kChunkBytes;              // 256 rows of one column of Q
    static constexpr int kRing = D == 128 ? 4 : 8;
    static constexpr int kStageBytes = 4096;                     // a warp's part of the way out: 32 rows of 128 bytes
    static constexpr int kSmem = 1024 + (2 + kRing) * kTileBytes + 8 * kStageBytes;
};

// A piece of the block's run, as warp 11 hands it out. n == 0: the run is over.
struct Piece {
    int n, in;           // tiles, and those of the segment before them
    int lead;            // tiles of the shared prefix at the segment's head (own segments)
    int place, head;     // of the piece; key head
    int b, bt;           // sequence; first query, counted over the batch
    int rows, len;       // query rows; keys of the part
    int see;             // keys that the segment's first query sees (prefix: all)
    int prefix, twin;    // twin: both halves hold the same rows, half h the tiles of its parity
    int whole;           // all of the segment's tiles
};
constexpr int kPieces = 4;
constexpr int kReaders = 11;             // warps that read one

struct Bars {
    uint64_t full[8], empty[8];
    uint64_t q_full, q_free;
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t order[2];                     // the other half has issued its tile's products
    uint64_t twin_full[4], twin_free[4];   // per quarter: half 1's rows of a twin segment are there / were taken
    uint64_t piece_full[kPieces], piece_free[kPieces];
    uint64_t drained[2];
    float2 twin_ml[kHalf];
    Piece piece[kPieces];
    uint32_t tmem;
    int abort;
};

// Whole warp, or any set of threads of one whose outcome need not be uniform with the others.
__device__ bool wait_long(Bars& b, uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer();
    for (;;) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*(volatile int*)&b.abort) return false;
        if (tc::globaltimer() - t0 > kWaitLimitNs) {
            atomicOr(&g_attn_error, 1u);
            *(volatile int*)&b.abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wwait(Bars& b, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_ready(bar, parity) || wait_long(b, bar, parity));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Matrix descriptors of 128-byte-swizzled tiles: the low word holds the address and the distance of 64-element
// chunks, the high word is the same for all of them (atoms of 8 rows, 1024 bytes apart).
//   K-major (Q, K): rows of 64 elements of the product's K axis; chunks are stepped through by address.
//   the other axis contiguous (V): rows are steps of the product's K axis, `lbo` bytes between chunks of its N axis.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) { return saddr >> 4 | (lbo >> 4) << 16; }

// A product whose operands are all in uniform registers costs its issue slot and no more; 64-bit descriptors
// computed for each took longer to issue than the tensor cores to multiply.
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 da, db; mov.b64 da, {%1, %4}; mov.b64 db, {%2, %4}; setp.ne.b32 p, %5, 0;"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(kDescHigh), "n"(ACC ? 1 : 0)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 db; mov.b64 db, {%2, %4}; setp.ne.b32 p, %5, 0;"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }" ::"r"(d),
        "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(kDescHigh), "r"(acc)
        : "memory");
}
// The same in every lane, and known to be.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The pieces of a run, as a reader steps through them.
struct Reader {
    int slot = 0;
    uint32_t phase = 0;
    // The next piece, or false (the run is over, or a wait ran out: alive says which).
    __device__ __forceinline__ bool next(Bars& b, Piece& p, bool& alive) {
        if (!(alive = wwait(b, &b.piece_full[slot], phase))) return false;
        p = b.piece[slot];
        return p.n > 0;
    }
    __device__ __forceinline__ void done(Bars& b) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&b.piece_free[slot]);
        if (++slot == kPieces) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// T: of queries and keys (and of narrow outputs). V: of values, and of the weights for the product with them.
template <typename T, typename V, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const ManyArgs a, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap pk,
                     const __grid_constant__ CUtensorMap pv, const __grid_constant__ CUtensorMap ok,
                     const __grid_constant__ CUtensorMap ov) {
    using C = Cfg<D>;
    extern __shared__ uint8_t s_raw[];
    __shared__ Bars s_bars;
    Bars& bars = s_bars;
    uint8_t* s_q = s_raw + ((1024 - (tc::smem_u32(s_raw) & 1023)) & 1023);   // [column][256 rows]
    uint8_t* s_ring = s_q + 2 * C::kTileBytes;
    uint8_t* s_stage = s_ring + C::kRing * C::kTileBytes;
    const Plan& p = a.plan;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 2);      // a half each
        }
        tc::mbar_init(&bars.q_full, 1);
        tc::mbar_init(&bars.q_free, 2);
        for (int h = 0; h < 2; ++h) {
            tc::mbar_init(&bars.s_full[h], 1);
            tc::mbar_init(&bars.p_ready[h], 4);    // a warp each
            tc::mbar_init(&bars.pv_done[h], 1);
            tc::mbar_init(&bars.drained[h], 1);
            tc::mbar_init(&bars.order[h], 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&bars.twin_full[i], 1);
            tc::mbar_init(&bars.twin_free[i], 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            tc::mbar_init(&bars.piece_full[i], 1);
            tc::mbar_init(&bars.piece_free[i], kReaders);
        }
        bars.abort = 0;
        tc::fence_mbar_init();
    }
    if (wid == 9) tc::tmem_alloc(&bars.tmem, kTmemCols);
    if (wid == 8 && lane == 0) {
        tc::prefetch_tensormap(&qm);
        tc::prefetch_tensormap(&pk);
        tc::prefetch_tensormap(&pv);
        tc::prefetch_tensormap(&ok);
        tc::prefetch_tensormap(&ov);
    }
    mq_grid_wait();
    mq_grid_release();   // only now: what is launched behind may run beside this kernel without waiting for it
    tc::tc_fence_before();
    Cursor c = find_run<kThreads>(p, a.len);   // holds block barriers
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (wid < 8) {
        tc::setmaxnreg_inc<kRowRegs>();
        // ---------------------------------------------------------------- rows: a thread each
        const int h = wid >> 2, quarter = wid & 3, row = quarter * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)quarter * 32 << 16);
        const uint32_t s_col = lane_base + h * 128, o_col = lane_base + 256 + h * 128;
        // unit u (16 bytes) of row r of the warp's stage: 128 bytes a row, units xor row % 8
        uint8_t* stage = s_stage + wid * C::kStageBytes;
        auto unit_of = [&](int r, int u) { return reinterpret_cast<uint4*>(stage + r * 128 + ((u ^ (r & 7)) << 4)); };
        const int my_unit = lane & 7, my_row = lane >> 3;         // on the way out 8 lanes take a row's 128 bytes
        uint32_t phase = 0, twin_phase = 0;   // phase: of the next tile's s_full; its pv_done follows in step
        bool alive = true;
        Reader reader;
        Piece g;
        while (reader.next(bars, g, alive)) {
            const int half0 = g.twin ? 0 : h * kHalf;             // rows of the segment before this half's
            const int r = half0 + row, q_in = p.by_group.of(r);   // this thread's row; its query in the segment
            const int n_rows = g.rows - half0 - quarter * 32;     // rows of the warp that count
            const int own_sees = g.prefix ? g.see : g.see + q_in;
            float m = -INFINITY, l = 0.0f;                    // reference (base 2, scaled) and sum
            float limit = -INFINITY;                          // of a tile's maximum that needs no other reference
            const int step = g.twin ? 2 : 1, j0 = g.twin ? h : 0;
            for (int j = j0; j < g.n; j += step) {
                if (!(alive = wwait(bars, &bars.s_full[h], phase))) break;
                phase ^= 1;
                if (n_rows <= 0) {                             // none of the warp's rows counts
                    if (lane == 0) tc::mbar_arrive(&bars.p_ready[h]);
                    continue;
                }
                tc::tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tc::tmem_ld32(s_col + k * 32, s[k]);
                tc::tmem_ld_wait();
                const int tile = g.in + j;
                const bool lead = tile < g.lead;
                const int k0 = (lead ? tile : tile - g.lead) * kKeys;
                const int seen = lead ? p.lead_keys : own_sees;
                if (__any_sync(0xffffffffu, k0 + kKeys > seen)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (k0 + k * 32 + i >= seen) s[k][i] = 0xff800000u;   // -infinity
                }
                float mx4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx4[k] = __uint_as_float(s[k][0]);
#pragma unroll
                    for (int i = 1; i < 32; ++i) mx4[k] = fmaxf(mx4[k], __uint_as_float(s[k][i]));
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                float2 sum[2] = {};
                bool weighed = false;
                // (lanes past the rows hold anything)
                if (__any_sync(0xffffffffu, lane < n_rows && mx > limit)) {   // the first key that a row sees, among others
                    // a row's own matter: what its neighbours do must not show in it
                    const bool grew = j == j0 || (lane < n_rows && mx - m > kGrow + kUp<V>);
                    if (__any_sync(0xffffffffu, grew)) {
                        const float now = grew ? reference<kUp<V>>(mx) : m;
                        const float f = now == -INFINITY ? 1.0f : exp2_fast(m - now);
                        m = now;
                        limit = is_large(m) ? -INFINITY : m + (kGrow + kUp<V>);
                        l *= f;
                        if (j > j0) {
                            // the product before this one must be done with O
                            if (!(alive = wwait(bars, &bars.pv_done[h], phase))) break;
                            tc::tc_fence_after();
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                uint32_t o[16];
                                tc::tmem_ld16(o_col + k * 16, o);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tc::tmem_st16(o_col + k * 16, o);
                            }
                        }
                    }
                    if (__any_sync(0xffffffffu, lane < n_rows && is_large(m))) {
                        // the products again, 32 at a time (P's columns up to here lie before the products that are left)
                        weighed = true;
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            uint32_t x[32], pr[16];
                            tc::tmem_ld32(s_col + k * 32, x);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float y = __uint_as_float(x[i]), base = m == -INFINITY ? 0.0f : m;
                                float e = exp2_fast(is_large(m) ? __fmul_rn(y, a.scale_log2) - base : fmaf(y, a.scale_log2, -base));
                                if (k0 + k * 32 + i >= seen) e = 0.0f;
                                (i & 1 ? sum[i >> 1 & 1].y : sum[i >> 1 & 1].x) += e;
                                x[i] = __float_as_uint(e);
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) pr[i] = mq_pack2<V>(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                            tc::tmem_st16(s_col + k * 16, pr);
                        }
                    }
                }
                if (!weighed) {
                    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pr[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = f2_fma(make_float2(__uint_as_float(s[k][2 * i]), __uint_as_float(s[k][2 * i + 1])),
                                                    f2_dup(a.scale_log2), f2_dup(-base));
                            const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                            sum[i & 1] = f2_add(sum[i & 1], e);
                            pr[i] = mq_pack2<V>(e.x, e.y);
                        }
                        tc::tmem_st16(s_col + k * 16, pr);
                    }
                }
                sum[0] = f2_add(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars.p_ready[h]);
            }
            if (!alive) break;
            if (j0 < g.n && !(alive = wwait(bars, &bars.pv_done[h], phase ^ 1))) break;
            // A twin segment's rows are joined by half 0's threads, which reach the other half's output in the same
            // lanes of tensor memory: f scales the own one, f1 the other.
            float f = 1.0f, f1 = 0.0f;
            const bool both = g.twin && g.n > 1;
            if (both) {
                if (h == 1) {
                    bars.twin_ml[row] = make_float2(m, l);
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars.twin_full[quarter]);
                    alive = wwait(bars, &bars.twin_free[quarter], twin_phase);
                } else if ((alive = wwait(bars, &bars.twin_full[quarter], twin_phase))) {
                    const float2 o = bars.twin_ml[row];
                    const float mm = fmaxf(m, o.x), mb = mm == -INFINITY ? 0.0f : mm;
                    f = exp2_fast(m - mb);
                    f1 = exp2_fast(o.x - mb);
                    l = l * f + o.y * f1;
                    m = mm;
                }
                if (!alive) break;
                twin_phase ^= 1;
            }
            if (!(g.twin && h == 1)) {
                tc::tc_fence_after();
                // Rows go out whole, 128 bytes at a time through the stage: in 16 bits or f32 where they are finished,
                // as they are (f32) to the piece's place otherwise.
                const bool finish = a.split && g.whole;
                const long long place = (long long)g.place * p.rows + half0 + quarter * 32;
                const long long out_row = finish ? ((long long)g.bt + q_in) * p.Hq + g.head * p.group + r - q_in * p.group
                                                 : place + lane;
                const bool narrow = finish && !a.fin.f32;
                const int row_bytes = D * (narrow ? 2 : 4);
                uint8_t* to = static_cast<uint8_t*>(finish ? a.fin.out : a.out.o) + out_row * row_bytes;
                if (finish) {
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    f *= inv;
                    f1 *= inv;
                    if (a.fin.lse && lane < n_rows) a.fin.lse[out_row] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
                } else if (lane < n_rows) {
                    a.out.ml[out_row] = make_float2(m, l);
                }
                uint8_t* row_to[8];                      // rows my_row + 4 i, this lane's unit
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    row_to[i] = reinterpret_cast<uint8_t*>(
                                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), my_row + 4 * i)) + my_unit * 16;
                auto load = [&](int col, uint32_t (&o)[32]) {   // 32 columns of the rows' outputs, scaled
                    tc::tmem_ld32(o_col + col, o);
                    tc::tmem_ld_wait();
                    if (both) {
                        uint32_t x[32];
                        tc::tmem_ld32(o_col + 128 + col, x);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f + __uint_as_float(x[i]) * f1);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    }
                };
#pragma unroll 1
                for (int col = 0, off = 0; col < D; off += 128) {
                    uint32_t o[32];
                    load(col, o);
                    if (narrow) {
#pragma unroll 1
                        for (int part = 0;; ++part) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                uint32_t y[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    y[i] = mq_pack2<T>(__uint_as_float(o[u * 8 + 2 * i]), __uint_as_float(o[u * 8 + 2 * i + 1]));
                                *unit_of(lane, part * 4 + u) = make_uint4(y[0], y[1], y[2], y[3]);
                            }
                            col += 32;
                            if (part == 1) break;
                            load(col, o);
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *unit_of(lane, u) = make_uint4(o[u * 4], o[u * 4 + 1], o[u * 4 + 2], o[u * 4 + 3]);
                        col += 32;
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (my_row + 4 * i < n_rows) *reinterpret_cast<uint4*>(row_to[i] + off) = *unit_of(my_row + 4 * i, my_unit);
                    __syncwarp();
                }
                tc::tc_fence_before();
                if (both) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars.twin_free[quarter]);
                }
            }
            reader.done(bars);
        }
    } else {
        tc::setmaxnreg_dec<kOtherRegs>();
        bool alive = true;
        Reader reader;
        Piece g;
        if (wid == 8) {
            // ------------------------------------------------------------ copies: Q of a piece, K and V of its tiles
            int slot = 0, issued = 0;
            uint32_t phase = 0, q_phase = 0;
            bool q_issued = false;
            while (reader.next(bars, g, alive)) {
                if (!(alive = wwait(bars, &bars.q_free, q_phase ^ 1))) break;
                if (tc::elect_one()) {
                    tc::mbar_arrive_expect_tx(&bars.q_full, C::kChunks * 128 * p.rows);
#pragma unroll
                    for (int k = 0; k < C::kChunks; ++k)
                        tma_load_3d(s_q + k * C::kQChunk, &qm, k * 64, g.head * p.group, g.bt, &bars.q_full);
                }
                __syncwarp();
                q_issued = true;
                q_phase ^= 1;
                for (int j = 0; alive && j < g.n; ++j) {
                    const int tile = g.in + j;
                    const bool shared = g.prefix || tile < g.lead;
                    const int k0 = (shared ? tile : tile - g.lead) * kKeys;
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!(alive = wwait(bars, &bars.empty[slot], phase ^ 1))) break;
#ifdef MQ_TEST_INJECT
                        const bool skip = g_test_skip_tile && blockIdx.x == 0 && issued == 0;
#else
                        constexpr bool skip = false;
#endif
                        if (!skip && tc::elect_one()) {
                            const CUtensorMap* map = shared ? (kv ? &pv : &pk) : (kv ? &ov : &ok);
                            tc::mbar_arrive_expect_tx(&bars.full[slot], C::kTileBytes);
#pragma unroll
                            for (int k = 0; k < C::kChunks; ++k)
                                tma_load_4d(tc::smem_u32(s_ring) + slot * C::kTileBytes + k * C::kChunkBytes, map, k * 64, g.head, k0,
                                            shared ? 0 : g.b, &bars.full[slot]);
                        }
                        __syncwarp();
                        ++issued;
                        if (++slot == C::kRing) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                }
                if (!alive) break;
                reader.done(bars);
            }
            if (!alive) {   // copies in flight must land before the block leaves
                if (q_issued) tc::mbar_wait(&bars.q_full, q_phase ^ 1, kWaitLimitNs);
                for (int i = 0; i < C::kRing && i < issued; ++i) {
                    if (--slot < 0) {
                        slot = C::kRing - 1;
                        phase ^= 1;
                    }
                    tc::mbar_wait(&bars.full[slot], phase, kWaitLimitNs);
                }
            }
        } else if (wid < 11) {
            // ------------------------------------------------------------ products of half h
            const int h = wid - 9;
            constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u, v_fmt = std::is_same<V, __nv_bfloat16>::value ? 1u : 0u;
            const uint32_t idesc_qk = tc::instr_desc(kHalf, kKeys, fmt) | (a.negative ? 1u << 13 : 0u);
            const uint32_t idesc_pv = tc::instr_desc(kHalf, D, v_fmt) | 1u << 16;   // V: the N axis contiguous
            constexpr uint32_t kTileLow = C::kTileBytes >> 4;
            const uint32_t ring = tc::smem_u32(s_ring);
            const uint32_t s_tm = uniform(tmem + h * 128), o_tm = uniform(tmem + 256 + h * 128);
            const uint32_t q_low = uniform(desc_low(tc::smem_u32(s_q), 16));
            const uint32_t k_low = uniform(desc_low(ring, 16)), v_low = uniform(desc_low(ring, C::kChunkBytes));
            int slot = 0;                        // ring slot of the piece's first K tile, and the phase there
            uint32_t phase = 0, q_phase = 0, p_phase = 0, turn = h ^ 1;
            auto step_slots = [&](int n) {       // n < kRing slots on
                slot += n;
                if (slot >= C::kRing) {
                    slot -= C::kRing;
                    phase ^= 1;
                }
            };
            // S = Q K^T with the K tile in `slot`; one lane. twice: the other half does not use the tile. last: nor
            // this half Q again.
            auto qk = [&](uint32_t q_at, bool twice, bool last) {
                const uint32_t kl = k_low + slot * kTileLow;
                mma_ss<false>(s_tm, q_at, kl, idesc_qk);
#pragma unroll
                for (int k = 1; k < D / 16; ++k)
                    mma_ss<true>(s_tm, q_at + (((k / 4) * C::kQChunk + (k % 4) * 32) >> 4),
                                 kl + (((k / 4) * C::kChunkBytes + (k % 4) * 32) >> 4), idesc_qk);
                tc::mma_commit(&bars.s_full[h]);
                tc::mma_commit(&bars.empty[slot]);
                if (twice) tc::mma_commit(&bars.empty[slot]);
                if (last) tc::mma_commit(&bars.q_free);
            };
            while (reader.next(bars, g, alive)) {
                const int step = g.twin ? 2 : 1;
                int t = g.twin ? h : 0;
                const uint32_t q_at = q_low + (g.twin ? 0 : h * (C::kChunkBytes >> 4));
                if (!(alive = wwait(bars, &bars.q_full, q_phase))) break;
                q_phase ^= 1;
                if (t > 0) step_slots(2);
                if (t < g.n) {
                    if (!(alive = wwait(bars, &bars.full[slot], phase))) break;
                    tc::tc_fence_after();
                    if (tc::elect_one()) qk(q_at, g.twin, t + step >= g.n);
                    __syncwarp();
                } else if (lane == 0) {
                    tc::mbar_arrive(&bars.q_free);
                }
                bool first = true;
                for (; t < g.n; t += step) {
                    step_slots(1);               // this tile's V
                    const int v_slot = slot;
                    if (!(alive = wwait(bars, &bars.full[slot], phase))) break;
                    const int tile = g.in + t, past = (tile - g.lead + 1) * kKeys - g.len;
                    if (past > 0 && !g.prefix && tile >= g.lead) {
                        // rows past the length may hold anything: zeros times a probability of zero
                        for (int u = lane; u < past * 8; u += 32)
#pragma unroll
                            for (int k = 0; k < C::kChunks; ++k)
                                *reinterpret_cast<uint4*>(s_ring + slot * C::kTileBytes + k * C::kChunkBytes +
                                                          (kKeys - past) * 128 + u * 16) = make_uint4(0, 0, 0, 0);
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    step_slots(g.twin ? 3 : 1);  // the half's next K
                    const bool more = t + step < g.n;
                    if (more && !(alive = wwait(bars, &bars.full[slot], phase))) break;
                    // The halves issue by turns, a tile's PV and the next one's QK together: issued side by side they
                    // would end side by side, and both halves' threads would wait for them at once, tile after tile.
                    if (!(alive = wwait(bars, &bars.order[h], turn))) break;
                    turn ^= 1;
                    if (!(alive = wwait(bars, &bars.p_ready[h], p_phase))) break;
                    p_phase ^= 1;
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
                        const uint32_t vl = v_low + v_slot * kTileLow;
                        mma_ts(o_tm, s_tm, vl, idesc_pv, !first);
#pragma unroll
                        for (int k = 1; k < kKeys / 16; ++k) mma_ts(o_tm, s_tm + k * 8, vl + (k * 2048 >> 4), idesc_pv, 1);
                        tc::mma_commit(&bars.pv_done[h]);
                        tc::mma_commit(&bars.empty[v_slot]);
                        if (g.twin) tc::mma_commit(&bars.empty[v_slot]);
                        if (more) qk(q_at, g.twin, t + 2 * step >= g.n);
                        tc::mbar_arrive(&bars.order[h ^ 1]);
                    }
                    __syncwarp();
                    first = false;
                }
                if (!alive) break;
                if (g.twin && h == 1 && (g.n & 1)) {   // half 0 has one tile more
                    if (!(alive = wwait(bars, &bars.order[1], turn))) break;
                    turn ^= 1;
                    if (lane == 0) tc::mbar_arrive(&bars.order[0]);
                }
                // t stands at the half's first tile past the piece, `slot` at that tile's K: back to the piece's end
                for (int n = 2 * (t - g.n); n > 0; --n)
                    if (--slot < 0) {
                        slot = C::kRing - 1;
                        phase ^= 1;
                    }
                reader.done(bars);
            }
            if (tc::elect_one()) tc::mma_commit(&bars.drained[h]);
            __syncwarp();
            tc::mbar_wait(&bars.drained[h], 0, kWaitLimitNs);
        } else {
            // ------------------------------------------------------------ the run's pieces
            const int per_seq = own_tiles_of_rows(p);
            int4 split = make_int4(-1, 0, 0, 0);
            int slot = 0;
            uint32_t phase = 0;
            advance(p, a.len, c, 0);
            for (;;) {
                g.n = 0;
                if (c.more()) {
                    g.n = piece_tiles(p, c);
                    g.in = c.in;
                    g.place = place_of(p, block_in_lane(p), c.seg);
                    g.head = c.head;
                    g.prefix = c.prefix;
                    g.b = c.prefix ? 0 : p.by_per_seq.of(c.unit);
                    const int rt = c.prefix ? c.unit : c.unit - g.b * per_seq;
                    const int t0 = p.by_group.of(rt * p.rows);
                    g.bt = g.b * p.T + t0;
                    g.rows = rows_of(p, c.prefix ? p.prefix_rows : p.T * p.group, rt);
                    g.len = c.prefix ? p.prefix_keys : own_len_of(p, a.len, g.b);
                    g.see = c.prefix ? g.len : g.len - p.T + 1 + t0;
                    g.lead = c.prefix ? 0 : ceil_div(p.lead_keys, kKeys);
                    g.twin = g.rows <= kHalf;
                    g.whole = c.in == 0 && g.n == c.tiles;
                    if (c.in == 0) {
                        const int2 f = blocks_of(p, c);
                        if (lane == 0) a.out.info[c.seg] = f;
                        if (!g.whole) split = make_int4(c.seg, f.y, c.unit, c.head);
                    }
                }
                if (!(alive = wwait(bars, &bars.piece_free[slot], phase ^ 1))) break;
                if (lane == 0) {
                    bars.piece[slot] = g;
                    tc::mbar_arrive(&bars.piece_full[slot]);
                }
                __syncwarp();
                if (++slot == kPieces) {
                    slot = 0;
                    phase ^= 1;
                }
                if (g.n == 0) break;
                advance(p, a.len, c, g.n);
            }
            if (lane == 0 && a.split) a.split[blockIdx.x] = split;
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (wid == 9) tc::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

// The register split assumes the launch's count (asked once per kernel).
bool regs_as_planned(const void* kern) {
    static std::mutex mu;
    static std::map<const void*, bool> done;
    std::lock_guard<std::mutex> lk(mu);
    const auto it = done.find(kern);
    if (it != done.end()) return it->second;
    cudaFuncAttributes fa;
    const bool ok = cudaFuncGetAttributes(&fa, kern) == cudaSuccess && fa.numRegs == kLaunchRegs;
    done.emplace(kern, ok);
    return ok;
}

}  // namespace

int launch_many(const ManyArgs& a, const mq_kv* prefix, const mq_kv* own, int D, int type, int v_type, cudaStream_t stream) {
    CUtensorMap qm, pk, pv, ok, ov;
    const mq_kv* p = prefix ? prefix : own;   // a part that is not there is never read
    const mq_kv* o = own ? own : prefix;
    if (!q_map(&qm, a.q, a.q_stride, (long long)a.plan.B * a.plan.T, a.plan.Hq, D, type, a.plan.group,
               a.plan.rows / a.plan.group) ||
        !kv_map(&pk, p, p->k, type, 64, kManyKeys) || !kv_map(&pv, p, p->v, v_type, 64, kManyKeys) ||
        !kv_map(&ok, o, o->k, type, 64, kManyKeys) || !kv_map(&ov, o, o->v, v_type, 64, kManyKeys))
        return MQ_ERR_LAUNCH;
    auto go = [&](auto kern, int smem) {
        if (!regs_as_planned(reinterpret_cast<const void*>(kern))) return (int)MQ_ERR_LAUNCH;
        if (!mq::allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3(a.plan.G), dim3(kThreads), smem, stream, a, qm, pk, pv, ok, ov);
    };
    auto of = [&](auto t, auto v) {
        using T = decltype(t);
        using V = decltype(v);
        return D == 64 ? go(attn_many_kernel<T, V, 64>, Cfg<64>::kSmem) : go(attn_many_kernel<T, V, 128>, Cfg<128>::kSmem);
    };
    if (type == MQ_F16) return of(__half(), __half());
    return v_type == MQ_F16 ? of(__nv_bfloat16(), __half()) : of(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace attn

namespace mq {
int take_attn_device_error(cudaStream_t stream, unsigned* code) {
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MQ_ERR_LAUNCH;
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, attn::g_attn_error, sizeof(v)) != cudaSuccess) return MQ_ERR_LAUNCH;
    unsigned few = 0;
    if (attn::take_few_error(&few) != MQ_OK) return MQ_ERR_LAUNCH;
    if (v) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(attn::g_attn_error, &zero, sizeof(zero)) != cudaSuccess) return MQ_ERR_LAUNCH;
    }
    *code = v | few;
    return MQ_OK;
}
}  // namespace mq

#ifdef MQ_TEST_INJECT
// Test builds only: bit 0: attn_many, bit 1: attn_few leaves out a copy.
extern "C" int mq_test_inject_attn(int bits) {
    const int many = bits & 1;
    return cudaMemcpyToSymbol(attn::g_test_skip_tile, &many, sizeof(many)) == cudaSuccess && attn::test_skip_few(bits >> 1 & 1)
               ? MQ_OK
               : MQ_ERR_LAUNCH;
}
#endif
