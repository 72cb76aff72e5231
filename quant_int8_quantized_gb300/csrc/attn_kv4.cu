// Attention over a 4-bit cache on pages (kv4.cuh).
//
// Few query rows per key head (a decode step, drafted tokens): a block is one warp with a run of its own of the row of key
// tiles (attn.cuh), as in attn_few.cu. A tile is 32 or 64 keys of a head (keys_of), one contiguous copy of 17 D bytes for each 16 of
// them, or a copy a page where pages are smaller than that, into a ring of stages. HBM would give an SM some 23 bytes a clock, 43
// numbers, and a warp's instruction serves 32 lanes: what bounds is the number of instructions per number, so everything is laid out
// to spend few on it.
//  - Keys and values are the left operands (16 x 16) of the warp-wide products, the queries the right ones (16 x 8): eight
//    rows' products cost what sixteen would the other way round, and the numbers become operands once for all rows.
//  - A lane's operands are consecutive bytes of the page (kv4.cuh): 16-byte loads without conflicts, then one or two
//    bit operations and one fused multiply-add a pair of numbers. n d is exact in either 16-bit type.
//  - S^T = K Q^T comes out with keys in rows; the exponentials, in pairs of queries, go through an 8 x 8 transposition (one
//    instruction) to become the right operand of O^T += V^T P^T.
//  - The maximum that the exponents are taken against is renewed when a row passes it by 2^8 (each row by itself, so that
//    no row's bits depend on its neighbours), which leaves one vote a tile.
// Measured: 64 sequences of 9000 to 20000 rows, 40 query and 8 key heads of 128 (1 GB), 191 us, 5.3 TB/s (its copies alone 157 to 166, all
// but them 164); one of 1000 rows, 9 us with the join, which is latency.
// Many rows (a prompt): the rows in use are read once into 16 bits in the workspace and mq_attn_prefix's tensor-core kernel
// takes them from there; n d being exact, both ways compute the same products, and both hold values and weights in f16.

#include <cmath>
#include <type_traits>

#include "attn_join.cuh"
#include "attn_many.cuh"
#include "attn_maps.cuh"
#include "kv4.cuh"
#include "kv4_calls.cuh"

namespace attn {
namespace {

__device__ unsigned int g_kv4_error;   // bit 0: a bounded wait gave up
#ifdef MQ_TEST_INJECT
__device__ int g_kv4_skip_tile;        // test builds only: block 0 leaves out its first tile
#endif

constexpr int keys_of(int D, int NT) { return D <= 64 || (D <= 128 && NT == 2) ? 64 : 32; }    // of a tile (measured)
constexpr int kStep = 32;              // keys that are multiplied at once

template <int D, int NT>
struct Shape {
    static constexpr int kKeys = keys_of(D, NT);
    static constexpr int kTile = kKeys / kv4::kBlockRows * kv4::block_bytes(D);
    static constexpr int kStages = D <= 64 || D > 128 || NT > 1 ? 2 : 3;   // (a third for 32 rows: no difference)
    static constexpr int kStage = kTile + 16;                        // a tile, its barrier
    static constexpr int kRing = kStages * kStage;
    static constexpr int kScales = kStep / 2 * (D / 32) * 16;        // a step's
    // more than eight rows: their operands (D / 8 registers of a lane for each eight) lie in shared memory, where the lane alone
    // reads them (24 rows: 46 us for 40 with them in registers, which spilled more). -Xptxas -v still shows spills, bytes stored / loaded:
    // 128 dims, 25 to 32 rows 364 / 292 (bf16 260 / 196); 256 dims, 9 to 16 rows 172 / 156 (132 / 112); 96 dims, 9 to 16 rows 48 / 52
    static constexpr bool kQueries = NT > 1;
    static constexpr int kSmem = kRing + kScales + (kQueries ? NT * (D / 32) * 512 : 0);
    // warps an SM, as registers allow (the outputs alone are D NT / 4 of a lane's); the same number on each of its four parts: 14
    // took 15 % longer than 12 or 16
    static constexpr int kPerSm = D * NT <= 64 ? 16 : (D <= 96 && NT <= 2) || NT == 1 && D <= 128 ? 12 : 8;
};

struct Kv4Args {
    Plan plan;
    kv4::Cache c;
    const void* q;
    long long q_stride;
    const int32_t* len;
    float scale_log2;
    Pieces out;
    int4* split;          // [G]: the segment that begins in the block and goes on in others (or -1), its last block, its row tile (sequence and
                          // tile) and key head
    Out fin;
};

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <typename T>                     // with nothing added
__device__ __forceinline__ void first_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Non-suspending test of a phase.
__device__ __forceinline__ bool bar_ready(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {   // 8 x 8 16-bit numbers, row i in lanes 4 i ..
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x) {          // 2^x within 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void put(uint32_t* to, const uint32_t (&x)[4]) { *reinterpret_cast<uint4*>(to) = make_uint4(x[0], x[1], x[2], x[3]); }

constexpr float kNone = -INFINITY;
// Weights are rounded to f16 and reach 2^15: the reference lies 2^7 below a maximum, which may grow by 2^8.
constexpr int kUp = 7;
constexpr float kGrow = 8.0f;

// A piece as the copying side hands it to the multiplying side. n == 0: the run is over.
struct Piece {
    int n, key0;         // tiles, first key
    int seg, head;
    int b, r0;           // sequence, first row
    int rows, len;       // rows: with kWhole where it is all of its segment, to be finished
};
constexpr int kWhole = 256;

// FIN: blocks finish the segments that they hold.
template <typename T, int D, int NT, bool FIN>
__global__ void __launch_bounds__(32, Shape<D, NT>::kPerSm) attn_kv4_kernel(const Kv4Args a) {
    using C = Shape<D, NT>;
    constexpr int nb = D / 32, kBlock = kv4::block_bytes(D), kStages = C::kStages, kKeys = C::kKeys;
    constexpr bool kHalf = std::is_same<T, __half>::value;
    // keys in the queries' type; values and weights in f16, which has room for both and more bits for the weights
    using KeyFactor = typename std::conditional<kHalf, kv4::Eighth, kv4::Scale<T>>::type;
    using Factor = kv4::Eighth;
    constexpr float kKeyUnit = kHalf ? 8.0f : 1.0f, kUnit = 8.0f;      // of the numbers that they make
    constexpr int KW = Factor::kWords;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ Piece s_piece[kStages + 1];
    uint32_t* const s_value = reinterpret_cast<uint32_t*>(s_ring + C::kRing);    // [block of dims][pair of rows][KW]
    uint4* const s_query = reinterpret_cast<uint4*>(s_ring + C::kRing + C::kScales);   // [eight rows][block of dims][lane]
    mq_grid_release();
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc::mbar_init(reinterpret_cast<uint64_t*>(s_ring + i * C::kStage + C::kTile), 1);
        tc::fence_mbar_init();
    }
    mq_grid_wait();
    const Plan& p = a.plan;
    const int tg = p.T * p.group, per_seq = own_tiles_of_rows(p);
    const int g = lane >> 2, t = lane & 3;

    if (FIN && lane == 0) a.split[blockIdx.x] = make_int4(-1, -1, -1, -1);

    // ---------------------------------------------------------------- copies, kStages - 1 tiles ahead
    Cursor c = find_run<32>(p, a.len);
    advance(p, a.len, c, 0);
    int left = 0, handed = 0, key = 0;                 // tiles of the copied piece left, pieces handed over
    int head = 0, seq = 0, issued = 0;
    // a tile lies on `parts` pages, `part` bytes on each; lane i holds the place of part i - at from the next one on
    const int parts = max(1, kKeys >> a.c.shift), part = C::kTile / parts, part_rows = kKeys / parts;
    const uint32_t all_parts = (1u << parts) - 1, ring = tc::smem_u32(s_ring);
    int at = 32;
    const uint8_t* src = nullptr;
    uint32_t there = 0;                                // the parts that are on a page
    uint32_t bad[kStages] = {};                        // parts on no page, of the tile that is multiplied next (0) and those behind it
    // Tiles that issue() may be called for, without another look: 0 where the run is over.
    auto look = [&] {
        if (left == 0) {
            Piece q;
            q.n = 0;
            if (c.more()) {
                q.n = piece_tiles(p, c);
                q.key0 = c.in * kKeys;
                q.seg = c.seg;
                q.head = c.head;
                q.b = p.by_per_seq.of(c.unit);
                q.r0 = (c.unit - q.b * per_seq) * p.rows;
                q.rows = min(p.rows, tg - q.r0);
                q.len = own_len_of(p, a.len, q.b);
                const bool whole = FIN && c.in == 0 && q.n == c.tiles;
                if (whole) q.rows += kWhole;
                if (lane == 0 && c.in == 0) {
                    const int2 blocks = blocks_of(p, c);
                    if (!FIN) a.out.info[c.seg] = blocks;
                    else if (!whole) a.split[blockIdx.x] = make_int4(c.seg, blocks.y, c.unit, c.head);
                }
                head = c.head;
                seq = q.b;
                key = q.key0;
                left = q.n;
                at = 32;
                advance(p, a.len, c, q.n);
            }
            __syncwarp();
            if (lane == 0) s_piece[handed] = q;
            __syncwarp();
            if (++handed == kStages + 1) handed = 0;
            if (left == 0) return 0;
        }
        if (at + parts > 32) {                         // the next 32 parts' places, a lane each
            at = 0;
            const unsigned row = (unsigned)key + lane * part_rows;      // (up to 1984 past a cache's end: past 2^31, too)
            const int page = row >> a.c.shift < (unsigned)a.c.width ? a.c.page(seq, (int)row) : -1;
            src = page >= 0 ? a.c.block(page, head, (int)row, kBlock) : nullptr;
            there = __ballot_sync(0xffffffffu, src != nullptr);
        }
        return min(left, (32 - at) / parts);
    };
    auto issue = [&](int off) {                        // the next tile, to the stage at `off`
        const uint32_t mine = there >> at & all_parts;
        bad[kStages - 1] = mine ^ all_parts;
#ifdef MQ_TEST_INJECT
        const bool skip = g_kv4_skip_tile && blockIdx.x == 0 && issued == 0;
#else
        constexpr bool skip = false;
#endif
        if (!skip && (unsigned)(lane - at) < (unsigned)parts) {
            const uint32_t to = ring + off, bar = to + C::kTile;
            if (lane == at) expect(bar, __popc(mine) * part);
            if (src) bulk_load(to + (lane - at) * part, src, part, bar);
        }
        at += parts;
        ++issued;
    };
    auto passed = [&](int n) {                         // after n of them
        left -= n;
        key += n * kKeys;
    };
    auto shift = [&] {
#pragma unroll
        for (int k = 1; k < kStages; ++k) bad[k - 1] = bad[k];
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        if (look() > 0) {
            issue(i * C::kStage);
            passed(1);
        }
        shift();
    }

    // ---------------------------------------------------------------- products
    auto from = [](const uint8_t* q) {
        return [q](auto type, int i) { return reinterpret_cast<const decltype(type)*>(q)[i]; };
    };
    const float scale = fminf(fmaxf(a.scale_log2 * kKeyUnit, -3.4028234663852886e38f), 3.4028234663852886e38f);
    int taken = 0, taken_tiles = 0, off = 0, free_off = C::kRing - C::kStage;    // stages: of the next tile, and the one free
    uint32_t phase = 0;
    bool alive = true;
    while (alive) {
        Piece w = s_piece[taken];
        if (w.n == 0) break;
        const bool whole = FIN && w.rows > kWhole;
        if (whole) w.rows -= kWhole;
        if (++taken == kStages + 1) taken = 0;
        // query rows 8 j + g (zeros past the last) as right operands, eight consecutive dims for each block of 32
        uint4 qf[C::kQueries ? 1 : NT][C::kQueries ? 1 : nb];
        int seen[NT][2];               // keys that rows 8 j + 2 t, 8 j + 2 t + 1 see
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int in = 8 * j + g, r = w.r0 + in, ti = p.by_group.of(r), h = w.head * p.group + r - ti * p.group;
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                            ((long long)w.b * p.T + ti) * a.q_stride + (long long)h * D + 8 * t);
#pragma unroll
            for (int b = 0; b < nb; ++b) {
                const uint4 v = in < w.rows ? __ldca(q + 4 * b) : make_uint4(0, 0, 0, 0);
                if constexpr (C::kQueries) s_query[(j * nb + b) * 32 + lane] = v;
                else qf[j][b] = v;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) seen[j][e] = w.len - p.T + 1 + p.by_group.of(w.r0 + 8 * j + 2 * t + e);
        }
        const int all_see = w.len - p.T + 1 + p.by_group.of(w.r0);     // every row sees the keys before
        float o[2 * nb][NT][4];
#pragma unroll
        for (int i = 0; i < 2 * nb; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
        // Rows' references, and (this lane's) sums. Where registers allow, what every step wants of a reference m is held instead of it:
        // what is added to the products for the exponents (-m; 0: no key seen yet) and the product from which on m is renewed.
        constexpr bool kHeld = NT <= 2;
        float minus[NT][2], limit[kHeld ? NT : 1][2] = {};
        float2 l[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                minus[j][e] = kHeld ? 0.0f : INFINITY;
                if constexpr (kHeld) limit[j][e] = kNone;
            }
            l[j] = make_float2(0.0f, 0.0f);
        }
        auto limit_of = [&](int j, int e) { return kHeld ? limit[kHeld ? j : 0][e] : (kUp + kGrow) - minus[j][e]; };
        auto less_of = [&](int j, int e) { return kHeld || minus[j][e] != INFINITY ? minus[j][e] : 0.0f; };
        auto minus_of = [&](int j, int e) { return kHeld && limit[kHeld ? j : 0][e] == kNone ? INFINITY : minus[j][e]; };   // -m

        int k0 = w.key0, ahead = 0;    // ahead: tiles to go before the copying side has to look
        bool more = true;              // it has some
#pragma unroll 1
        for (int ti = w.n; ti > 0; --ti) {
            if (ahead == 0) {
                const int n = look();
                more = n > 0;
                ahead = more ? min(n, ti) : ti;
                passed(more ? ahead : 0);
            }
            --ahead;
            if (more) issue(free_off);
            if (!(alive = __all_sync(0xffffffffu, bar_ready(ring + off + C::kTile, phase) ||
                                                      tc::mbar_wait(reinterpret_cast<uint64_t*>(s_ring + off + C::kTile), phase, kWaitLimitNs))))
                break;
            uint8_t* const tile = s_ring + off;
            const uint32_t none_of = bad[0];
            shift();
            ++taken_tiles;
            free_off = off;
            off += C::kStage;
            if (off == C::kRing) {
                off = 0;
                phase ^= 1;
            }
#pragma unroll 1
            for (int in = 0; in < kKeys; in += kStep, k0 += kStep) {
                if (kKeys > kStep && k0 >= w.len) break;
                uint8_t* const st = tile + in / kv4::kBlockRows * kBlock;
                // The values' scales as the numbers need them, once for all lanes: half a pair of rows each. Those of rows that
                // are on no page or past the end are zero, whatever lies there.
                {
                    uint32_t vc[(nb + 3) / 4];
                    if constexpr (nb % 2 == 0) kv4::bytes<nb>(from(st + (lane >> 4) * kBlock + kv4::value_scale_at(D) + (lane & 15) * nb), vc);
                    const int pair = (lane >> 4) * 8 + ((lane & 15) >> 1);        // of the step's 16
                    uint32_t keep = ~0u;
                    if (none_of || k0 + kStep > w.len) {
                        if (none_of >> ((in + lane) / part_rows) & 1) {       // (once in the stage: keys' scales are read row by row)
#pragma unroll
                            for (int b = 0; b < nb; ++b) st[(lane >> 4) * kBlock + kv4::key_scale_at(D) + (lane & 15) * nb + b] = 0;
                            tc::fence_proxy_async_smem();
                        }
                        const bool gone = none_of >> ((in + 2 * pair) / part_rows) & 1;
                        keep = (!gone && k0 + 2 * pair < w.len ? 0x00ff00ffu : 0u) | (!gone && k0 + 2 * pair + 1 < w.len ? 0xff00ff00u : 0u);
                    }
                    if constexpr (nb % 2 == 0) {
#pragma unroll
                        for (int i = 0; i < (nb + 3) / 4; ++i) vc[i] &= keep;
#pragma unroll
                        for (int i = 0; i < nb / 2; ++i) {
                            uint32_t y[KW];
                            Factor::of(kv4::both(vc, i)).to(y);
                            put(s_value + (((lane & 1) * (nb / 2) + i) * 16 + pair) * KW, y);
                        }
                    } else {
                        const uint8_t* q = st + (lane >> 4) * kBlock + kv4::value_scale_at(D) + (pair & 7) * 2 * nb;
                        for (int b = lane & 1; b < nb; b += 2) {
                            uint32_t y[KW];
                            Factor::of((q[2 * b] & keep & 255) << 8 | (q[2 * b + 1] & keep >> 8 & 255) << 24).to(y);
                            put(s_value + (b * 16 + pair) * KW, y);
                        }
                    }
                    __syncwarp();
                }
                float s[2][NT][4];
                // Blocks of 16 keys by turns where there are few rows: a product waits for the one before it in its sum.
                constexpr int kAtOnce = NT == 1 ? 2 : 1;
#pragma unroll
                for (int blk0 = 0; blk0 < 2; blk0 += kAtOnce) {
                    uint32_t kw[kAtOnce][2][nb], ks[kAtOnce][2][(nb + 3) / 4];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const uint8_t* at = st + (blk0 + i) * kBlock;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            kv4::words<nb>(from(at + (u * 32 + lane) * nb * 4), kw[i][u]);
                            kv4::bytes<nb>(from(at + kv4::key_scale_at(D) + (g + 8 * u) * nb), ks[i][u]);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < nb; b += 2) {
                        KeyFactor f[kAtOnce][2];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u) f[i][u] = KeyFactor::of(kv4::both(ks[i][u], b / 2));
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (b + e < nb) {
                                uint32_t x0[kAtOnce][4], x1[kAtOnce][4];
#pragma unroll
                                for (int i = 0; i < kAtOnce; ++i) {
                                    kv4::numbers(kw[i][0][b + e], f[i][0].half(e), x0[i]);
                                    kv4::numbers(kw[i][1][b + e], f[i][1].half(e), x1[i]);
                                }
                                uint4 q[NT];
#pragma unroll
                                for (int j = 0; j < NT; ++j)
                                    q[j] = C::kQueries ? s_query[(j * nb + b + e) * 32 + lane] : qf[C::kQueries ? 0 : j][C::kQueries ? 0 : b + e];
#pragma unroll
                                for (int j = 0; j < NT; ++j)
#pragma unroll
                                    for (int i = 0; i < kAtOnce; ++i) {
                                        if (b + e == 0) first_mma<T>(s[blk0 + i][j], x0[i][0], x1[i][0], x0[i][1], x1[i][1], q[j].x, q[j].y);
                                        else mma<T>(s[blk0 + i][j], x0[i][0], x1[i][0], x0[i][1], x1[i][1], q[j].x, q[j].y);
                                    }
#pragma unroll
                                for (int j = 0; j < NT; ++j)
#pragma unroll
                                    for (int i = 0; i < kAtOnce; ++i) mma<T>(s[blk0 + i][j], x0[i][2], x1[i][2], x0[i][3], x1[i][3], q[j].z, q[j].w);
                            }
                    }
                }
                // row (key) 16 blk + g + 8 (e / 2), column (query) 8 j + 2 t + e % 2
                float mx[NT][2];
                bool grew = false;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 x = f2_mul(make_float2(s[blk][j][2 * u], s[blk][j][2 * u + 1]), f2_dup(scale));
                            s[blk][j][2 * u] = x.x, s[blk][j][2 * u + 1] = x.y;
                        }
                    if (k0 + kStep > all_see) {
#pragma unroll
                        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (k0 + 16 * blk + g + 8 * (e >> 1) >= seen[j][e & 1]) s[blk][j][e] = kNone;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[j][e] = fmaxf(fmaxf(fmaxf(s[0][j][e], s[0][j][e + 2]), s[1][j][e]), s[1][j][e + 2]);
                        grew |= mx[j][e] > limit_of(j, e);
                    }
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float alpha[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) mx[j][e] = fmaxf(mx[j][e], __shfl_xor_sync(0xffffffffu, mx[j][e], x));
                            const bool up = mx[j][e] > limit_of(j, e);
                            const float was = minus_of(j, e), now = up ? -reference<kUp>(mx[j][e]) : was;
                            alpha[e] = up ? exp2_fast(now - was) : 1.0f;
                            minus[j][e] = kHeld && now == INFINITY ? 0.0f : now;
                            if constexpr (kHeld) limit[j][e] = (kUp + kGrow) - now;
                        }
                        l[j] = f2_mul(l[j], make_float2(alpha[0], alpha[1]));
#pragma unroll
                        for (int i = 0; i < 2 * nb; ++i) {
                            o[i][j][0] *= alpha[0], o[i][j][1] *= alpha[1];
                            o[i][j][2] *= alpha[0], o[i][j][3] *= alpha[1];
                        }
                    }
                }
                uint32_t pf[2][NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float2 less = make_float2(less_of(j, 0), less_of(j, 1));
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 x = f2_add(make_float2(s[blk][j][2 * u], s[blk][j][2 * u + 1]), less);
                            const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                            l[j] = f2_add(l[j], e);
                            pf[blk][j][u] = transposed(mq_pack2<__half>(e.x, e.y));
                        }
                    }
                }
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    const uint8_t* at = st + blk * kBlock;
                    uint32_t vw[2][nb];
#pragma unroll
                    for (int u = 0; u < 2; ++u) kv4::words<nb>(from(at + kv4::value_at(D) + (u * 32 + lane) * nb * 4), vw[u]);
#pragma unroll
                    for (int b = 0; b < nb; ++b) {
                        uint32_t x0[4], x1[4], f[KW];
                        kv4::words<KW>(from(reinterpret_cast<const uint8_t*>(s_value + (16 * b + 8 * blk + t) * KW)), f);
                        kv4::numbers(vw[0][b], Factor::from(f), x0);
                        kv4::words<KW>(from(reinterpret_cast<const uint8_t*>(s_value + (16 * b + 8 * blk + 4 + t) * KW)), f);
                        kv4::numbers(vw[1][b], Factor::from(f), x1);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            mma<__half>(o[2 * b][j], x0[0], x0[1], x1[0], x1[1], pf[blk][j][0], pf[blk][j][1]);
                            mma<__half>(o[2 * b + 1][j], x0[2], x0[3], x1[2], x1[3], pf[blk][j][0], pf[blk][j][1]);
                        }
                    }
                }
                __syncwarp();      // scales, and after the last step the stage, may be written again
            }
        }
        if (!alive) break;
        const long long place = ((long long)blockIdx.x + w.seg) * p.rows;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = e ? l[j].y : l[j].x;
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                const int r = 8 * j + 2 * t + e;
                if (r >= w.rows) continue;
                if (FIN && whole) {
                    const int ti = p.by_group.of(w.r0 + r);
                    const long long row = ((long long)w.b * p.T + ti) * p.Hq + w.head * p.group + w.r0 + r - ti * p.group;
                    const float by = sum == 0.0f ? 0.0f : kUnit / sum;       // no key seen (a NaN or infinite sum stays one)
                    if (g == 0 && a.fin.lse) a.fin.lse[row] = sum == 0.0f ? kNone : -minus_of(j, e) * kLn2 + logf(sum);
#pragma unroll
                    for (int b = 0; b < nb; ++b) {
                        const float y[4] = {o[2 * b][j][e] * by, o[2 * b][j][e + 2] * by, o[2 * b + 1][j][e] * by, o[2 * b + 1][j][e + 2] * by};
                        const long long to = row * D + 32 * b + 4 * g;
                        if (a.fin.f32) *reinterpret_cast<float4*>(static_cast<float*>(a.fin.out) + to) = make_float4(y[0], y[1], y[2], y[3]);
                        else *reinterpret_cast<uint2*>(static_cast<T*>(a.fin.out) + to) = make_uint2(mq_pack2<T>(y[0], y[1]), mq_pack2<T>(y[2], y[3]));
                    }
                    continue;
                }
                if (g == 0) a.out.ml[place + r] = make_float2(-minus_of(j, e), sum);
                float* to = a.out.o + (place + r) * D + 4 * g;
#pragma unroll
                for (int b = 0; b < nb; ++b)
                    *reinterpret_cast<float4*>(to + 32 * b) =
                        make_float4(o[2 * b][j][e] * kUnit, o[2 * b][j][e + 2] * kUnit, o[2 * b + 1][j][e] * kUnit, o[2 * b + 1][j][e + 2] * kUnit);
            }
    }
    if (!alive) {   // a copy never came: recorded; those still in flight must land before the block leaves
        if (lane == 0) atomicOr(&g_kv4_error, 1u);
        for (int i = taken_tiles; i < issued; ++i) {
            tc::mbar_wait(reinterpret_cast<uint64_t*>(s_ring + off + C::kTile), phase, kWaitLimitNs);
            off += C::kStage;
            if (off == C::kRing) {
                off = 0;
                phase ^= 1;
            }
        }
    }
}

// The rows of the segments that one block of the first kernel began and another ended: grid x that block, y rows.
template <typename O, int D>
__global__ void __launch_bounds__(32) join_split_kernel(const Kv4Args a) {
    mq_grid_release();
    mq_grid_wait();
    const Plan& p = a.plan;
    const int4 s = __ldca(a.split + blockIdx.x);
    if (s.x < 0 || s.y < (int)blockIdx.x || s.y >= p.G) return;
    const int per_seq = own_tiles_of_rows(p), b = p.by_per_seq.of(s.z), r0 = (s.z - b * per_seq) * p.rows;
    const int rows = min(p.rows, p.T * p.group - r0);
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        const int ti = p.by_group.of(r0 + r);
        const Run run = {&a.out, ((long long)blockIdx.x + s.x) * p.rows + r, p.rows, s.y - (int)blockIdx.x + 1};
        write_row<O, D>(add_pieces<D, 8>(run, Run{}, 0, run.count), a.fin, nullptr,
                        ((long long)b * p.T + ti) * p.Hq + s.w * p.group + r0 + r - ti * p.group);
    }
}

// Tiles of eight rows that a segment has for `rows` rows of a key head; what registers allow is 4 of 128 dims.
int tiles_of_rows(long long rows, int D) {
    const int most = D <= 128 ? 4 : 2;
    const long long eights = (rows + 7) / 8, tiles = (eights + most - 1) / most;
    return (int)((eights + tiles - 1) / tiles);
}

constexpr int kFinMost = 2;     // tiles of eight rows in kernels that finish segments

template <typename F>
int with_kernel(int D, int type, int nt, bool fin, F f) {
    auto go = [&](auto t) {
        using T = decltype(t);
        auto of = [&](auto d) {
            constexpr int W = decltype(d)::value;
            auto with = [&](auto n) {
                constexpr int NT = decltype(n)::value;
                if constexpr (NT <= kFinMost)
                    if (fin) return f(attn_kv4_kernel<T, W, NT, true>, Shape<W, NT>::kSmem, Shape<W, NT>::kPerSm);
                return f(attn_kv4_kernel<T, W, NT, false>, Shape<W, NT>::kSmem, Shape<W, NT>::kPerSm);
            };
            if (nt == 1) return with(std::integral_constant<int, 1>());
            if constexpr (W <= 128) {
                if (nt == 3) return with(std::integral_constant<int, 3>());
                if (nt == 4) return with(std::integral_constant<int, 4>());
            }
            return with(std::integral_constant<int, 2>());
        };
        switch (D) {
            case 64: return of(std::integral_constant<int, 64>());
            case 96: return of(std::integral_constant<int, 96>());
            case 128: return of(std::integral_constant<int, 128>());
            default: return of(std::integral_constant<int, 256>());
        }
    };
    return type == MQ_F16 ? go(__half()) : go(__nv_bfloat16());
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Bytes of 16-bit rows at once, unless one sequence has more.
#ifndef MQ_KV4_READ_BYTES
#define MQ_KV4_READ_BYTES (1LL << 30)
#endif
constexpr long long kReadBytes = MQ_KV4_READ_BYTES;

// Whether the rows in use are read into 16 bits for the tensor-core kernel: where that is expected to take less time than walking the
// 4-bit rows once for each tile of query rows, if the caches are as long as the tables allow. Measured, in us (walked / read): 4
// sequences of 8192 rows, 8 key heads of 128, 80 query rows a head 74 / 92, 120: 92 / 92, 160: 110 / 89, 480: 290 / 94; of 6000 rows, 4 heads of
// 64, 224: 33 / 54, 448: 55 / 55; one of 1500, 4 heads of 128, 448: 28 / 42, 896: 30 / 42.
bool worth_reading(int B, int at_once, long long rows, int Hkv, int D, int cap, int nt) {
#ifdef MQ_KV4_READ_FROM    // (test builds)
    return rows >= MQ_KV4_READ_FROM;
#else
    const double width = D / 128.0, keys = (double)B * Hkv * cap;
    const double walk = keys / 32 * ((rows + 8 * nt - 1) / (8 * nt)) * width * (1.5e-3 + 0.33e-3 * nt);
    return walk > 30.0 * ((B + at_once - 1) / at_once) + keys * D * 4 / 3.3e6 + keys * D * 4 * (double)rows / 1.2e9;
#endif
}

// Segments for each block, at least, for blocks to finish those that they hold.
#ifndef MQ_KV4_SPLIT_FROM      // (test builds: 0)
#define MQ_KV4_SPLIT_FROM 1
#endif

// How a call is cut.
struct Kv4Cut {
    bool read, fits;
    int nt, at_once;               // read: sequences at once
    Plan plan;
    bool split;                    // segments that one block holds are finished by it
    size_t kv, o, ml, info, bytes; // read: bytes of the 16-bit keys (and of the values)
};

Kv4Cut cut_kv4(int B, int T, int Hq, int Hkv, int D, int cap) {
    Kv4Cut c = {};
    const int group = Hq / Hkv;
    const long long rows = (long long)T * group;
    c.fits = true;
    c.nt = tiles_of_rows(rows, D);
    const long long one = 2LL * cap * Hkv * D;                 // bytes of a sequence's keys in 16 bits
    const long long most_at_once = one > 0 ? kReadBytes / (2 * one) : B;
    c.at_once = (int)(most_at_once < 1 ? 1 : most_at_once < B ? most_at_once : B);
    c.read = cap > 0 && many_takes(D, group) && worth_reading(B, c.at_once, rows, Hkv, D, cap, c.nt);
    if (c.read) {
        c.kv = up16((size_t)one * c.at_once);
        size_t ws = part_ws_bytes(c.at_once, T, Hq, Hkv, D, cap);
        c.fits = ws > 0;
        if (B % c.at_once) {
            const size_t rest = part_ws_bytes(B % c.at_once, T, Hq, Hkv, D, cap);
            if (rest > ws) ws = rest;
        }
        c.bytes = 2 * c.kv + ws;
        return c;
    }
    Plan& p = c.plan;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = group;
    p.own_cap = cap;
    p.own = 1;
    p.rows = 8 * c.nt;
    p.keys = keys_of(D, c.nt);
    p.wide = p.rows;
    p.cost = p.wide_cost = 1;
    p.lanes = 1;
    p.by_group = div_by(group);
    p.by_per_seq = div_by(own_tiles_of_rows(p));
    const long long segs = cap > 0 ? all_segs(p) : 0, most = segs * ceil_div(cap, p.keys);
    int per_sm = 1;
    with_kernel(D, MQ_F16, c.nt, false, [&](auto, int, int n) { return per_sm = n; });
    const long long held = (long long)mq::num_sms() * per_sm;
    // Beginning and ending a segment costs about a tile. Where there are few tiles, and their pieces few bytes to join, each has a
    // warp of its own (one sequence of 1000 rows: 8.8 us, with runs of two tiles and more 9.9, of three 11.0; 32 queries of 7 heads on
    // 1500 rows, 22 MB of pieces: 27.9, 22.2, 26.4).
    p.extra = most <= 2 * held && most * p.rows * D * 4 <= 12 << 20 ? 0 : 1;
    if (most + segs * p.extra > 0x7fffffffLL || segs > 0x3fffffffLL) c.fits = false;
    p.G = (int)(most < held ? most : held);
    // Where there are fewer segments than blocks most lie in several, and each row has a warp to add its pieces up (attn_join_kernel);
    // else most lie in one or two (512 sequences of up to 2000 rows: 144 us that way, 140 this; 2048 of up to 300: 201 and 135).
    c.split = c.nt <= kFinMost && segs >= (long long)MQ_KV4_SPLIT_FROM * p.G;
    p.own_least = c.split ? 1 : 0;
    const size_t places = (size_t)p.G + (size_t)segs;
    c.o = 0;
    c.ml = up16(places * p.rows * D * sizeof(float));
    c.info = c.ml + up16(places * p.rows * sizeof(float2));
    c.bytes = c.info + up16(c.split ? (size_t)p.G * sizeof(int4) : (size_t)segs * sizeof(int2));
    return c;
}

bool valid_kv4(long long B, long long T, int Hq, int Hkv, int D, int cap) {
    constexpr long long kMost = 0x3fffffff;
    return Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && kv4::valid_dim(D) && cap >= 0 && cap <= 0x7fffffff - 255 && B * T <= kMost &&
           B * T * Hq <= kMost;
}

}  // namespace

int take_kv4_error(unsigned* code) {
    if (cudaMemcpyFromSymbol(code, g_kv4_error, sizeof(*code)) != cudaSuccess) return MQ_ERR_LAUNCH;
    const unsigned zero = 0;
    return *code && cudaMemcpyToSymbol(g_kv4_error, &zero, sizeof(zero)) != cudaSuccess ? MQ_ERR_LAUNCH : MQ_OK;
}

}  // namespace attn

#ifdef MQ_TEST_INJECT
extern "C" int mq_test_inject_kv4(int on) {
    return cudaMemcpyToSymbol(attn::g_kv4_skip_tile, &on, sizeof(on)) == cudaSuccess ? MQ_OK : MQ_ERR_LAUNCH;
}
#endif

extern "C" size_t mq_attn_kv4_ws_bytes(int B, int T, int Hq, int Hkv, int D, int cap) {
    using namespace attn;
    if (B <= 0 || T <= 0 || !valid_kv4(B, T, Hq, Hkv, D, cap)) return 0;
    const Kv4Cut c = cut_kv4(B, T, Hq, Hkv, D, cap);
    return c.fits ? c.bytes : 0;
}

extern "C" int mq_attn_kv4(const void* q, int type, long long q_stride, int B, int T, int Hq, const mq_kv4* cache,
                           const int32_t* len, float scale, void* out, int out_type, float* lse, void* ws, size_t ws_bytes,
                           cudaStream_t stream) {
    using namespace attn;
    if (B < 0 || T < 0) return MQ_ERR_SHAPE;
    int rc = kv4::check(cache, true);
    if (rc != MQ_OK) return rc;
    if ((type != MQ_F16 && type != MQ_BF16) || (out_type != type && out_type != MQ_F32)) return MQ_ERR_TYPE;
    const int Hkv = cache->heads, D = cache->dim, cap = cache->width * cache->page_rows;
    if (cache->n != B || !valid_kv4(B, T, Hq, Hkv, D, cap)) return MQ_ERR_SHAPE;
    if (B == 0 || T == 0) return MQ_OK;
    if (q_stride < (long long)Hq * D || q_stride % 8 != 0 || ((long long)B * T > 1 && q_stride > kStrideMost) || !std::isfinite(scale))
        return MQ_ERR_SHAPE;
    if (!q || !out || !ws || !len) return MQ_ERR_NULL;
    if (!mq::aligned16(q) || !mq::aligned16(out) || !mq::aligned16(ws) || !mq::aligned16(len) || !mq::aligned16(lse))
        return MQ_ERR_ALIGN;
    const Kv4Cut c = cut_kv4(B, T, Hq, Hkv, D, cap);
    if (!c.fits) return MQ_ERR_SHAPE;
    if (ws_bytes < c.bytes) return MQ_ERR_SCRATCH;
    const long long rows = (long long)B * T * Hq, out_bytes = rows * D * (out_type == MQ_F32 ? 4 : 2);
    if (mq::rows_meet(q, (long long)B * T, 2 * q_stride, 2LL * Hq * D, out, out_bytes) ||
        kv4::meets_pages(cache, out, out_bytes))
        return MQ_ERR_SHAPE;   // read by some blocks while others write
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    uint8_t* base = static_cast<uint8_t*>(ws);
    if (c.read) {
        for (int b = 0; b < B; b += c.at_once) {
            const int n = B - b < c.at_once ? B - b : c.at_once;
            mq_kv4 part = *cache;
            part.n = n;
            part.table += b * cache->table_stride;
            const mq_kv kv = {base, base + c.kv, (long long)cap * Hkv * D, (long long)Hkv * D, D, type, n, cap, Hkv, D};
            rc = kv4::launch_read(&part, len + b, &kv, MQ_F16, stream);
            if (rc != MQ_OK) return rc;
            const long long at = (long long)b * T;
            rc = call(static_cast<const uint16_t*>(q) + at * q_stride, q_stride, n, T, Hq, nullptr, &kv, len + b, scale,
                      static_cast<uint8_t*>(out) + at * Hq * D * (out_type == MQ_F32 ? 4 : 2), out_type,
                      lse ? lse + at * Hq : nullptr, nullptr, nullptr, base + 2 * c.kv, ws_bytes - 2 * c.kv, stream, true);
            if (rc != MQ_OK) return rc;
        }
        return MQ_OK;
    }
    const Pieces pieces = {reinterpret_cast<float*>(base + c.o), reinterpret_cast<float2*>(base + c.ml),
                           reinterpret_cast<int2*>(base + c.info)};
    if (c.plan.G > 0) {
        Kv4Args f;
        f.plan = c.plan;
        f.c = kv4::cache_of(cache);
        f.q = q;
        f.q_stride = q_stride;
        f.len = len;
        f.scale_log2 = scale * 1.4426950408889634f;
        f.out = pieces;
        f.split = c.split ? reinterpret_cast<int4*>(base + c.info) : nullptr;
        f.fin = {out, lse, out_type == MQ_F32};
        rc = with_kernel(D, type, c.nt, c.split, [&](auto kern, int smem, int) {
            if (!mq::allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
            return mq::launch_pdl(kern, dim3(c.plan.G), dim3(32), smem, stream, f);
        });
        if (rc != MQ_OK) return rc;
        if (c.split) {
            auto join = [&](auto o) {
                using O = decltype(o);
                auto kern = D == 64 ? join_split_kernel<O, 64> : D == 96 ? join_split_kernel<O, 96>
                            : D == 128 ? join_split_kernel<O, 128> : join_split_kernel<O, 256>;
                if (!mq::allow_smem(reinterpret_cast<const void*>(kern), 0)) return (int)MQ_ERR_LAUNCH;
                const int rows = T * (Hq / Hkv) < c.plan.rows ? T * (Hq / Hkv) : c.plan.rows;
                return mq::launch_pdl(kern, dim3(c.plan.G, rows), dim3(32), 0, stream, f);
            };
            return out_type == MQ_F32 ? join(float()) : out_type == MQ_F16 ? join(__half()) : join(__nv_bfloat16());
        }
    }
    JoinArgs j = {};
    j.own = {pieces, cap > 0 ? c.plan.rows : 0, c.plan};
    j.len = len;
    j.B = B;
    j.T = T;
    j.Hq = Hq;
    j.Hkv = Hkv;
    j.group = Hq / Hkv;
    j.own_cap = cap;
    j.fin = {out, lse, out_type == MQ_F32};
    return launch_join(j, D, out_type, stream);
}
