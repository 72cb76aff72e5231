// Attention over a 4-bit cache on pages (kv4.cuh).
//
// Few query rows per key head (a decode step, drafted tokens): a block is one warp with a run of its own of the row of key
// tiles (attn.cuh), as in attn_few.cu. A tile is 32 keys of a head, one contiguous copy of 17 D bytes (two where pages have
// 16 rows) into a ring of stages. HBM would give an SM some 23 bytes a clock, 43 numbers, and a warp's instruction serves
// 32 lanes: what bounds is the number of instructions per number, so everything is laid out to spend few on it.
//  - Keys and values are the left operands (16 x 16) of the warp-wide products, the queries the right ones (16 x 8): eight
//    rows' products cost what sixteen would the other way round, and the numbers become operands once for all rows.
//  - A lane's operands are consecutive bytes of the page (kv4.cuh): 16-byte loads without conflicts, then one or two
//    bit operations and one fused multiply-add a pair of numbers. n d is exact in either 16-bit type.
//  - S^T = K Q^T comes out with keys in rows; the exponentials, in pairs of queries, go through an 8 x 8 transposition (one
//    instruction) to become the right operand of O^T += V^T P^T.
//  - The maximum that the exponents are taken against is renewed when a row passes it by 2^8 (each row by itself, so that
//    no row's bits depend on its neighbours), which leaves one vote a tile.
// Many rows (a prompt): the rows in use are read once into 16 bits in the workspace and mq_attn_prefix's tensor-core kernel
// takes them from there; n d being exact, both ways compute the same products.

#include <cmath>
#include <type_traits>

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

constexpr int kTileExtra = 2;          // what beginning and ending a segment costs, in tiles

constexpr int keys_of(int D) { return D <= 128 ? 64 : 32; }   // of a tile
constexpr int kStep = 32;              // keys that are multiplied at once

template <int D, int NT>
struct Shape {
    static constexpr int kKeys = keys_of(D);
    static constexpr int kTile = kKeys / kv4::kBlockRows * kv4::block_bytes(D);
    static constexpr int kStages = D <= 64 ? 3 : 2;
    static constexpr int kRing = kStages * kTile;
    static constexpr int kSmem = kRing + kStep / 2 * (D / 32) * 8;   // stages; a step's value scales
    // warps an SM: registers (the outputs alone are D NT / 4 of a lane's)
    static constexpr int kPerSm = D * NT <= 64 ? 14 : D * NT <= 128 ? 11 : 8;
};

struct Kv4Args {
    Plan plan;
    kv4::Cache c;
    const void* q;
    long long q_stride;
    const int32_t* len;
    float scale_log2;
    Pieces out;
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
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

constexpr float kNone = -INFINITY;
// Weights reach 2^15 in f16 and 2^8 in bf16: the reference lies 2^7 (f16) below a maximum, which may grow by 2^8.
template <typename T>
constexpr int kUp = std::is_same<T, __half>::value ? 7 : 0;
constexpr float kGrow = 8.0f;

// A piece as the copying side hands it to the multiplying side. n == 0: the run is over.
struct Piece {
    int n, key0;         // tiles, first key
    int seg, head;
    int b, r0;           // sequence, first row
    int rows, len;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32, Shape<D, NT>::kPerSm) attn_kv4_kernel(const Kv4Args a) {
    using C = Shape<D, NT>;
    constexpr int nb = D / 32, kBlock = kv4::block_bytes(D), kStages = C::kStages, kKeys = C::kKeys;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ Piece s_piece[kStages + 1];
    __shared__ uint64_t s_full[kStages];
    __shared__ uint32_t s_bad[kStages];    // blocks of the tile that are on no page
    uint2* const s_scale = reinterpret_cast<uint2*>(s_ring + C::kRing);   // [row pair of the step][nb]
    mq_grid_release();
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&s_full[i], 1);
        tc::fence_mbar_init();
    }
    mq_grid_wait();
    const Plan& p = a.plan;
    const int tg = p.T * p.group, per_seq = own_tiles_of_rows(p);
    const int g = lane >> 2, t = lane & 3;

    // ---------------------------------------------------------------- copies, kStages - 1 tiles ahead
    Cursor c = find_run<32>(p, a.len);
    advance(p, a.len, c, 0);
    int left = 0, handed = 0, key = 0, in_slot = 0;    // tiles of the copied piece left, pieces handed over
    int head = 0, seq = 0, issued = 0;
    int pages_at = 0, pages = -1;                      // lane i: page pages_at + i of the sequence
    // a tile lies on `parts` pages, `part` bytes on each
    const int parts = max(1, kKeys >> a.c.shift), part = C::kTile / parts, part_shift = min(a.c.shift, kKeys == 64 ? 6 : 5);
    auto copy = [&] {
        bool fresh = false;
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
                if (lane == 0 && c.in == 0) a.out.info[c.seg] = blocks_of(p, c);
                head = c.head;
                seq = q.b;
                key = q.key0;
                left = q.n;
                fresh = true;
                advance(p, a.len, c, q.n);
            }
            __syncwarp();
            if (lane == 0) s_piece[handed] = q;
            __syncwarp();
            if (++handed == kStages + 1) handed = 0;
        }
        if (left > 0) {
            const int first = key >> a.c.shift;
            if (fresh || first + parts - pages_at > 32) {
                pages_at = first;
                const int i = first + lane;
                const int e = i < a.c.width ? __ldca(a.c.table + seq * a.c.table_stride + i) : -1;
                pages = (unsigned)e < (unsigned)a.c.n_pages ? e : -1;
            }
            const int page = __shfl_sync(0xffffffffu, pages, first - pages_at + min(lane, parts - 1));
            const bool there = lane < parts && page >= 0;
            const uint32_t all = __ballot_sync(0xffffffffu, there);
#ifdef MQ_TEST_INJECT
            const bool skip = g_kv4_skip_tile && blockIdx.x == 0 && issued == 0;
#else
            constexpr bool skip = false;
#endif
            if (!skip) {
                uint64_t* bar = &s_full[in_slot];
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(bar, __popc(all) * part);
                    s_bad[in_slot] = ~all & ((1u << parts) - 1);
                }
                if (there)
                    bulk_load(tc::smem_u32(s_ring) + in_slot * C::kTile + lane * part,
                              a.c.block(page, head, key, kBlock), part, bar);
            }
            __syncwarp();
            ++issued;
            key += kKeys;
            --left;
            if (++in_slot == kStages) in_slot = 0;
        }
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy();

    // ---------------------------------------------------------------- products
    auto from = [](const uint8_t* q) {
        return [q](auto type, int i) { return reinterpret_cast<const decltype(type)*>(q)[i]; };
    };
    int taken = 0, slot = 0, taken_tiles = 0;
    uint32_t phase = 0;
    bool alive = true;
    while (alive) {
        const Piece w = s_piece[taken];
        if (w.n == 0) break;
        if (++taken == kStages + 1) taken = 0;
        // query rows 8 j + g (zeros past the last) as right operands, eight consecutive dims for each block of 32
        uint32_t qf[NT][nb][4];
        int seen[NT][2];               // keys that rows 8 j + 2 t, 8 j + 2 t + 1 see
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int in = 8 * j + g, r = w.r0 + in, ti = p.by_group.of(r), h = w.head * p.group + r - ti * p.group;
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                            ((long long)w.b * p.T + ti) * a.q_stride + (long long)h * D + 8 * t);
#pragma unroll
            for (int b = 0; b < nb; ++b) {
                const uint4 v = in < w.rows ? __ldca(q + 4 * b) : make_uint4(0, 0, 0, 0);
                qf[j][b][0] = v.x, qf[j][b][1] = v.y, qf[j][b][2] = v.z, qf[j][b][3] = v.w;
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
        float m[NT][2], l[NT][2];      // references and (this lane's) sums
#pragma unroll
        for (int j = 0; j < NT; ++j) m[j][0] = m[j][1] = kNone, l[j][0] = l[j][1] = 0.0f;

#pragma unroll 1
        for (int ti = 0; ti < w.n; ++ti) {
            copy();
            if (!(alive = __all_sync(0xffffffffu, mbar_ready(&s_full[slot], phase) ||
                                                      tc::mbar_wait(&s_full[slot], phase, kWaitLimitNs))))
                break;
            uint8_t* const tile = s_ring + slot * C::kTile;
            const uint32_t bad = s_bad[slot];
            ++taken_tiles;
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
#pragma unroll 1
            for (int in = 0; in < kKeys; in += kStep) {
                const int k0 = w.key0 + ti * kKeys + in;
                if (k0 >= w.len) break;
                uint8_t* const st = tile + in / kv4::kBlockRows * kBlock;
                if (bad || k0 + kStep > w.len) {
                    // scales of rows that are on no page, and of values past the end: zero, whatever lies there
                    const int blk = lane >> 4, r = lane & 15;
                    uint8_t* s = st + blk * kBlock;
                    const bool none = bad >> ((in + lane) >> part_shift) & 1;
                    if (none || k0 + lane >= w.len)
#pragma unroll
                        for (int b = 0; b < nb; ++b) {
                            s[kv4::value_scale_at(D) + (r >> 1) * 2 * nb + 2 * b + (r & 1)] = 0;
                            if (none) s[kv4::key_scale_at(D) + r * nb + b] = 0;
                        }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                // the values' scales as the numbers need them, once for all lanes: nb / 2 pairs of rows a lane
                {
                    const uint8_t* at = st + (lane >> 4) * kBlock + kv4::value_scale_at(D) + (lane & 15) * nb;
                    if constexpr (nb % 2 == 0) {
                        uint32_t c[(nb + 3) / 4];
                        kv4::bytes<nb>(from(at), c);
                        uint32_t x[nb];
#pragma unroll
                        for (int i = 0; i < nb / 2; ++i) {
                            const kv4::Scale<T> sc = kv4::Scale<T>::of(kv4::both(c, i));
                            x[2 * i] = *reinterpret_cast<const uint32_t*>(&sc.mul);
                            x[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&sc.off);
                        }
                        uint32_t* to = reinterpret_cast<uint32_t*>(s_scale) + lane * nb;
                        if constexpr (nb == 2) *reinterpret_cast<uint2*>(to) = make_uint2(x[0], x[1]);
                        else
#pragma unroll
                            for (int i = 0; i < nb / 4; ++i)
                                reinterpret_cast<uint4*>(to)[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    } else {
                        for (int i = lane; i < kStep / 2 * nb; i += 32) {
                            const int pair = i / nb, b = i - pair * nb;
                            const uint8_t* q = st + (pair >> 3) * kBlock + kv4::value_scale_at(D) + (pair & 7) * 2 * nb + 2 * b;
                            const kv4::Scale<T> sc = kv4::Scale<T>::of((uint32_t)q[0] << 8 | (uint32_t)q[1] << 24);
                            s_scale[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&sc.mul), *reinterpret_cast<const uint32_t*>(&sc.off));
                        }
                    }
                }
                float s[2][NT][4];
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    const uint8_t* at = st + blk * kBlock;
                    uint32_t kw[2][nb], ks[2][(nb + 3) / 4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        kv4::words<nb>(from(at + (u * 32 + lane) * nb * 4), kw[u]);
                        kv4::bytes<nb>(from(at + kv4::key_scale_at(D) + (g + 8 * u) * nb), ks[u]);
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) s[blk][j][0] = s[blk][j][1] = s[blk][j][2] = s[blk][j][3] = 0.0f;
#pragma unroll
                    for (int b = 0; b < nb; b += 2) {
                        const kv4::Scale<T> s0 = kv4::Scale<T>::of(kv4::both(ks[0], b / 2)), s1 = kv4::Scale<T>::of(kv4::both(ks[1], b / 2));
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (b + e < nb) {
                                uint32_t x0[4], x1[4];
                                kv4::numbers(kw[0][b + e], kv4::half_of(s0, e), x0);
                                kv4::numbers(kw[1][b + e], kv4::half_of(s1, e), x1);
#pragma unroll
                                for (int j = 0; j < NT; ++j) {
                                    mma<T>(s[blk][j], x0[0], x1[0], x0[1], x1[1], qf[j][b + e][0], qf[j][b + e][1]);
                                    mma<T>(s[blk][j], x0[2], x1[2], x0[3], x1[3], qf[j][b + e][2], qf[j][b + e][3]);
                                }
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
                        for (int e = 0; e < 4; ++e) s[blk][j][e] *= a.scale_log2;
                    if (k0 + kStep > all_see) {
#pragma unroll
                        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (k0 + 16 * blk + g + 8 * (e >> 1) >= seen[j][e & 1]) s[blk][j][e] = kNone;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[j][e] = fmaxf(fmaxf(s[0][j][e], s[0][j][e + 2]), fmaxf(s[1][j][e], s[1][j][e + 2]));
                        grew |= mx[j][e] > m[j][e] + (kUp<T> + kGrow);
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
                            const float now = mx[j][e] > m[j][e] + (kUp<T> + kGrow) ? reference<kUp<T>>(mx[j][e]) : m[j][e];
                            alpha[e] = now == m[j][e] ? 1.0f : exp2_fast(m[j][e] - now);
                            m[j][e] = now;
                            l[j][e] *= alpha[e];
                        }
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
                    const float safe[2] = {m[j][0] == kNone ? 0.0f : m[j][0], m[j][1] == kNone ? 0.0f : m[j][1]};
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float e0 = exp2_fast(s[blk][j][2 * u] - safe[0]), e1 = exp2_fast(s[blk][j][2 * u + 1] - safe[1]);
                            l[j][0] += e0;
                            l[j][1] += e1;
                            pf[blk][j][u] = transposed(mq_pack2<T>(e0, e1));
                        }
                    }
                }
                __syncwarp();      // the scales are there
#pragma unroll
                for (int blk = 0; blk < 2; ++blk) {
                    const uint8_t* at = st + blk * kBlock;
                    uint32_t vw[2][nb], vs[2][2 * nb];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        kv4::words<nb>(from(at + kv4::value_at(D) + (u * 32 + lane) * nb * 4), vw[u]);
                        kv4::words<2 * nb>(from(reinterpret_cast<const uint8_t*>(s_scale + (8 * blk + 4 * u + t) * nb)), vs[u]);
                    }
#pragma unroll
                    for (int b = 0; b < nb; ++b) {
                        uint32_t x0[4], x1[4];
                        kv4::numbers(vw[0][b], kv4::Scale<T>::from(vs[0][2 * b], vs[0][2 * b + 1]), x0);
                        kv4::numbers(vw[1][b], kv4::Scale<T>::from(vs[1][2 * b], vs[1][2 * b + 1]), x1);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            mma<T>(o[2 * b][j], x0[0], x0[1], x1[0], x1[1], pf[blk][j][0], pf[blk][j][1]);
                            mma<T>(o[2 * b + 1][j], x0[2], x0[3], x1[2], x1[3], pf[blk][j][0], pf[blk][j][1]);
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
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], x);
                const int r = 8 * j + 2 * t + e;
                if (r < w.rows) {
                    if (g == 0) a.out.ml[place + r] = make_float2(m[j][e], l[j][e]);
                    float* to = a.out.o + (place + r) * D + 4 * g;
#pragma unroll
                    for (int b = 0; b < nb; ++b)
                        *reinterpret_cast<float4*>(to + 32 * b) =
                            make_float4(o[2 * b][j][e], o[2 * b][j][e + 2], o[2 * b + 1][j][e], o[2 * b + 1][j][e + 2]);
                }
            }
    }
    if (!alive) {   // a copy never came: recorded; those still in flight must land before the block leaves
        if (lane == 0) atomicOr(&g_kv4_error, 1u);
        for (int i = taken_tiles; i < issued; ++i) {
            tc::mbar_wait(&s_full[slot], phase, kWaitLimitNs);
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
}

// Tiles of eight rows that a segment has for `rows` rows of a key head; what registers allow is 4 of 128 dims.
int tiles_of_rows(long long rows, int D) {
    const int most = D <= 128 ? 4 : 2;
    return rows >= 8LL * most ? most : (int)((rows + 7) / 8);
}

template <typename F>
int with_kernel(int D, int type, int nt, F f) {
    auto go = [&](auto t) {
        using T = decltype(t);
        auto of = [&](auto d) {
            constexpr int W = decltype(d)::value;
            if (nt == 1) return f(attn_kv4_kernel<T, W, 1>, Shape<W, 1>::kSmem, Shape<W, 1>::kPerSm);
            if constexpr (W <= 128) {
                if (nt == 3) return f(attn_kv4_kernel<T, W, 3>, Shape<W, 3>::kSmem, Shape<W, 3>::kPerSm);
                if (nt == 4) return f(attn_kv4_kernel<T, W, 4>, Shape<W, 4>::kSmem, Shape<W, 4>::kPerSm);
            }
            return f(attn_kv4_kernel<T, W, 2>, Shape<W, 2>::kSmem, Shape<W, 2>::kPerSm);
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

// From so many query rows per key head on the rows are read into 16 bits for the tensor-core kernel.
#ifndef MQ_KV4_READ_FROM
#define MQ_KV4_READ_FROM 129
#endif
constexpr int kReadFrom = MQ_KV4_READ_FROM;
// Bytes of 16-bit rows at once, unless one sequence has more.
#ifndef MQ_KV4_READ_BYTES
#define MQ_KV4_READ_BYTES (1LL << 30)
#endif
constexpr long long kReadBytes = MQ_KV4_READ_BYTES;

// How a call is cut.
struct Kv4Cut {
    bool read, fits;
    int nt, at_once;               // read: sequences at once
    Plan plan;
    size_t kv, o, ml, info, bytes; // read: bytes of the 16-bit keys (and of the values)
};

Kv4Cut cut_kv4(int B, int T, int Hq, int Hkv, int D, int cap) {
    Kv4Cut c = {};
    const int group = Hq / Hkv;
    const long long rows = (long long)T * group;
    c.fits = true;
    c.read = cap > 0 && many_takes(D, group) && rows >= kReadFrom;
    if (c.read) {
        const long long one = 2LL * cap * Hkv * D;             // of a sequence's keys
        const long long most = one > 0 ? kReadBytes / (2 * one) : B;
        c.at_once = (int)(most < 1 ? 1 : most < B ? most : B);
        c.kv = up16((size_t)one * c.at_once);
        size_t ws = mq_attn_ws_bytes(c.at_once, T, Hq, Hkv, D, 0, cap, 0);
        c.fits = ws > 0;
        if (B % c.at_once) {
            const size_t rest = mq_attn_ws_bytes(B % c.at_once, T, Hq, Hkv, D, 0, cap, 0);
            if (rest > ws) ws = rest;
        }
        c.bytes = 2 * c.kv + ws;
        return c;
    }
    c.nt = tiles_of_rows(rows, D);
    Plan& p = c.plan;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.group = group;
    p.own_cap = cap;
    p.own = 1;
    p.rows = 8 * c.nt;
    p.keys = keys_of(D);
    p.wide = p.rows;
    p.cost = p.wide_cost = 1;
    p.extra = kTileExtra;
    p.lanes = 1;
    p.by_group = div_by(group);
    p.by_per_seq = div_by(own_tiles_of_rows(p));
    const long long segs = all_segs(p), most = segs * ceil_div(cap, p.keys);
    if (most + segs * p.extra > 0x7fffffffLL || segs > 0x3fffffffLL) c.fits = false;
    int per_sm = 1;
    with_kernel(D, MQ_F16, c.nt, [&](auto, int, int n) { return per_sm = n; });
    const long long held = (long long)mq::num_sms() * per_sm;
    p.G = (int)(most < held ? most : held);
    const size_t places = (size_t)p.G + (size_t)segs;
    c.o = 0;
    c.ml = up16(places * p.rows * D * sizeof(float));
    c.info = c.ml + up16(places * p.rows * sizeof(float2));
    c.bytes = c.info + up16((size_t)segs * sizeof(int2));
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
        mq::rows_meet(out, 1, out_bytes, out_bytes, cache->pages, cache->page_stride * cache->n_pages))
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
            rc = kv4::launch_read(&part, len + b, &kv, stream);
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
        rc = with_kernel(D, type, c.nt, [&](auto kern, int smem, int) {
            if (!mq::allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
            return mq::launch_pdl(kern, dim3(c.plan.G), dim3(32), smem, stream, f);
        });
        if (rc != MQ_OK) return rc;
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
