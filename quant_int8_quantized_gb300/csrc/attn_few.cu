// Attention pieces for few query rows per key head (up to 16 a segment): every key and value is
// read once and used for a handful of rows, so HBM bounds and the matrix products only have to keep
// out of the way. They run as warp-wide 16 x 8 x 16 products in registers.
//
// A block is one warp with a run of its own, eight of them per SM, and nothing waits for anything else: the
// warp copies tiles of 16 keys and values into its ring of stages (TMA: one lane issues a tile's few boxes, where
// 16-byte copies of all lanes kept the warp busy and no more than some 60 bytes a ns on their way into an SM), keeps
// running maximum, sum and output in registers and leaves the piece in the workspace. The copies run ahead
// across the ends of pieces. The products q k^T come out in the layout that the second product takes as its
// left operand, so probabilities stay in registers. The boxes' swizzle puts eight rows of an 8 x 8 matrix load into
// eight different groups of banks. Value rows past a cache's length are zeroed in the stage: whatever lies there
// must not reach a sum.
// Measured: the own caches of 64 sequences (17 to 2048 rows, 8 key heads of 128, 268 MB) in 49 us, 5.4 TB/s; one sequence on a
// prefix of 512 in 6.4 us, which is latency.

#include <type_traits>

#include "attn_few.cuh"
#include "attn_maps.cuh"

namespace attn {
namespace {

__device__ unsigned int g_few_error;   // bit 0: a bounded wait gave up
#ifdef MQ_TEST_INJECT
__device__ int g_test_skip_tile;       // test builds only: block 0 leaves out its first tile
#endif

constexpr int kThreads = 32;
constexpr int kKeys = kFewKeys;

template <int D>
struct Cfg {
    static constexpr int kDims = D % 64 == 0 ? 64 : 32;       // of a box
    static constexpr int kRow = kDims * 2;                    // bytes of a row of it
    static constexpr int kUnits = kDims / 8;                  // 16-byte units of that
    static constexpr int kBoxes = D / kDims;
    static constexpr int kBoxBytes = kKeys * kRow;
    static constexpr int kTileBytes = kBoxes * kBoxBytes;     // of keys, or of values
    static constexpr int kStageBytes = 2 * kTileBytes;        // keys, then values
    // 16 KB or so of stages: with 24 (measured) an SM no longer holds eight blocks together with what each has beside
    // them, and the last ones start when the first have ended
    static constexpr int kStages = D <= 64 ? 4 : D <= 96 ? 3 : 2;
    static constexpr int kSmem = 1024 + kStages * kStageBytes;
    // what the swizzle adds (xor) to the units of a row
    __device__ static __forceinline__ int twist(int row) { return kDims == 64 ? row & 7 : (row >> 1) & 3; }
};

// A piece as the copying side hands it to the multiplying side. n == 0: the run is over.
struct Piece {
    int n, key0;         // tiles, first key
    int seg, head;
    int b, r0;           // sequence (prefix: 0), first row
    int rows, len;
    int prefix;
};

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2^x within 2 ulp; 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kNone = -INFINITY;
// A row's reference follows its maximum, so its weights are at most 2^14 in f16.
template <typename T>
constexpr int kUp = std::is_same<T, __half>::value ? 14 : 0;

template <typename T, int D, bool RAW>
__global__ void __launch_bounds__(kThreads, 8)
    attn_few_kernel(const FewArgs a, const __grid_constant__ CUtensorMap pk, const __grid_constant__ CUtensorMap pv,
                    const __grid_constant__ CUtensorMap ok, const __grid_constant__ CUtensorMap ov) {
    using C = Cfg<D>;
    extern __shared__ uint8_t s_raw[];
    __shared__ Piece s_piece[C::kStages + 1];
    __shared__ uint64_t s_full[C::kStages];
    constexpr int stages = C::kStages;
    mq_grid_release();
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) tc::mbar_init(&s_full[i], 1);
        tc::fence_mbar_init();
        tc::prefetch_tensormap(&pk);
        tc::prefetch_tensormap(&pv);
        tc::prefetch_tensormap(&ok);
        tc::prefetch_tensormap(&ov);
    }
    if (!a.beside) mq_grid_wait();
    const Plan& p = a.plan;
    const int lane = threadIdx.x;
    const int tg = p.T * p.group, per_seq = own_tiles_of_rows(p);
    const uint32_t ring = (tc::smem_u32(s_raw) + 1023) & ~1023u;
    const int g = lane >> 2, t2 = (lane & 3) * 2;   // this thread's rows g, g + 8 and columns t2, t2 + 1

    // ---------------------------------------------------------------- copies, stages - 1 tiles ahead
    Cursor c = find_run<kThreads>(p, a.len);
    advance(p, a.len, c, 0);
    int left = 0, handed = 0, key = 0, in_slot = 0;    // tiles of the copied piece left, pieces handed over
    int head = 0, seq = 0, issued = 0;
    bool shared = false;
    auto copy = [&] {
        if (left == 0) {
            Piece q;
            q.n = 0;
            if (c.more()) {
                q.n = piece_tiles(p, c);
                q.key0 = c.in * kKeys;
                q.seg = c.seg;
                q.head = c.head;
                q.prefix = c.prefix;
                q.b = c.prefix ? 0 : p.by_per_seq.of(c.unit);
                q.r0 = (c.prefix ? c.unit : c.unit - q.b * per_seq) * kFewRows;
                q.rows = min(kFewRows, (c.prefix ? p.prefix_rows : tg) - q.r0);
                q.len = c.prefix ? p.prefix_keys : own_len_of(p, a.len, q.b);
                if (lane == 0 && c.in == 0) a.out.info[c.seg] = blocks_of(p, c);
                head = c.head;
                seq = q.b;
                shared = c.prefix;
                key = q.key0;
                left = q.n;
                advance(p, a.len, c, q.n);
            }
            __syncwarp();
            if (lane == 0) s_piece[handed] = q;
            __syncwarp();
            if (++handed == stages + 1) handed = 0;
        }
        if (left > 0) {
#ifdef MQ_TEST_INJECT
            const bool skip = g_test_skip_tile && blockIdx.x == 0 && issued == 0;
#else
            constexpr bool skip = false;
#endif
            if (!skip && lane == 0) {
                const uint32_t st = ring + in_slot * C::kStageBytes;
                const CUtensorMap *km = shared ? &pk : &ok, *vm = shared ? &pv : &ov;
                tc::mbar_arrive_expect_tx(&s_full[in_slot], C::kStageBytes);
#pragma unroll
                for (int i = 0; i < C::kBoxes; ++i) {
                    tma_load_4d(st + i * C::kBoxBytes, km, i * C::kDims, head, key, seq, &s_full[in_slot]);
                    tma_load_4d(st + C::kTileBytes + i * C::kBoxBytes, vm, i * C::kDims, head, key, seq, &s_full[in_slot]);
                }
            }
            ++issued;
            key += kKeys;
            --left;
            if (++in_slot == stages) in_slot = 0;
        }
    };
#pragma unroll 1
    for (int t = 0; t < stages - 1; ++t) copy();

    // ---------------------------------------------------------------- products
    // Byte of this lane's row and unit in a box, for the loads of keys (rows of eight keys, 8 dims side by side) and of
    // values (transposed); unit 2 i of the row is this xor 32 i.
    const int k_row = (lane >> 4) * 8 + (lane & 7), v_row = ((lane >> 3) & 1) * 8 + (lane & 7);
    const uint32_t k_at = k_row * C::kRow + ((((lane >> 3) & 1) ^ C::twist(k_row)) << 4);
    const uint32_t v_at = C::kTileBytes + v_row * C::kRow + (((lane >> 4) ^ C::twist(v_row)) << 4);
    constexpr int kPairs = C::kUnits / 2;   // 16 dims each
    int taken = 0, slot = 0, taken_tiles = 0;
    uint32_t phase = 0;
    bool alive = true;
    while (alive) {
        const Piece w = s_piece[taken];
        if (w.n == 0) break;
        if (++taken == stages + 1) taken = 0;
        // query rows g and g + 8 (zeros past the last), as left operands; the keys that each sees
        uint32_t qf[D / 16][4];
        int seen[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = w.r0 + g + 8 * u;
            const bool live = g + 8 * u < w.rows;
            const int t = p.by_group.of(r), h = w.head * p.group + r - t * p.group;   // prefix: t is b T + t
            seen[u] = w.prefix ? w.len : w.len - p.T + 1 + t;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) +
                                                                  (live ? ((long long)w.b * p.T + t) * a.q_stride + h * D : 0));
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][u] = live ? __ldca(q + (k * 16 + t2) / 2) : 0u;
                qf[k][u + 2] = live ? __ldca(q + (k * 16 + 8 + t2) / 2) : 0u;
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};   // references and sums
        float* const raw_row = RAW ? a.raw + (((long long)w.b * p.Hkv + w.head) * tg + w.r0) * p.own_cap : nullptr;

#pragma unroll 1
        for (int t = 0; t < w.n; ++t) {
            copy();
            if (!(alive = __all_sync(0xffffffffu, mbar_ready(&s_full[slot], phase) ||
                                                      tc::mbar_wait(&s_full[slot], phase, kWaitLimitNs))))
                break;
            const uint32_t st = ring + slot * C::kStageBytes;
            const int k0 = w.key0 + t * kKeys;
            if (!w.prefix && k0 + kKeys > w.len) {   // (of the prefix what lies past the end reads as zeros)
                for (int u = (w.len - k0) * C::kUnits + lane; u < kKeys * C::kUnits; u += 32)
#pragma unroll
                    for (int i = 0; i < C::kBoxes; ++i)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(st + C::kTileBytes + i * C::kBoxBytes + u * 16),
                                     "r"(0)
                                     : "memory");
                tc::fence_proxy_async_smem();
                __syncwarp();
            }
            ++taken_tiles;
            if (++slot == stages) {
                slot = 0;
                phase ^= 1;
            }
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t kf[4];
                ldm4(st + k / kPairs * C::kBoxBytes + (k_at ^ (k % kPairs * 32)), kf);
                mma<T>(s[0], qf[k], kf[0], kf[1]);
                mma<T>(s[1], qf[k], kf[2], kf[3]);
            }
            float mx[2] = {kNone, kNone};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key_at = k0 + j * 8 + t2 + (e & 1);
                    s[j][e] = key_at < seen[e >> 1] ? s[j][e] * a.scale_log2 : kNone;
                    mx[e >> 1] = fmaxf(mx[e >> 1], s[j][e]);
                }
            if constexpr (RAW) {
                if (!w.prefix) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (g + 8 * u < w.rows) {
                            float* raw = raw_row + (g + 8 * u) * (long long)p.own_cap + k0 + t2;
                            if (k0 + kKeys <= w.len && !(p.own_cap & 1)) {
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    *reinterpret_cast<float2*>(raw + j * 8) = make_float2(s[j][2 * u], s[j][2 * u + 1]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 2; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (k0 + j * 8 + t2 + e < w.len) raw[j * 8 + e] = s[j][2 * u + e];
                            }
                        }
                }
            }
            float alpha[2];
            bool grew = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
                mx[u] = fmaxf(m[u], reference<kUp<T>>(mx[u]));
                grew |= mx[u] != m[u];
                const float safe = mx[u] == kNone ? 0.0f : mx[u];
                alpha[u] = exp2_fast(m[u] - safe);
                m[u] = mx[u];
                mx[u] = safe;
            }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int u = 0; u < 2; ++u) l[u] *= alpha[u];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= alpha[0], o[i][1] *= alpha[0];
                    o[i][2] *= alpha[1], o[i][3] *= alpha[1];
                }
            }
            uint32_t pf[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float e0 = exp2_fast(s[j][2 * u] - mx[u]), e1 = exp2_fast(s[j][2 * u + 1] - mx[u]);
                    l[u] += e0 + e1;
                    pf[j * 2 + u] = mq_pack2<T>(e0, e1);
                }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t vf[4];
                ldm4t(st + i / kPairs * C::kBoxBytes + (v_at ^ (i % kPairs * 32)), vf);
                mma<T>(o[2 * i], pf, vf[0], vf[1]);
                mma<T>(o[2 * i + 1], pf, vf[2], vf[3]);
            }
            __syncwarp();   // the stage may be written again
        }
        if (!alive) break;
        const long long place = ((long long)blockIdx.x + w.seg) * kFewRows;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
            const int r = g + 8 * u;
            if (r < w.rows) {
                if ((lane & 3) == 0) a.out.ml[place + r] = make_float2(m[u], l[u]);
                float* to = a.out.o + (place + r) * D + t2;   // a quad writes whole 32-byte sectors
#pragma unroll
                for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][2 * u], o[i][2 * u + 1]);
            }
        }
    }
    if (!alive) {   // a copy never came: recorded; those still in flight must land before the block leaves
        if (lane == 0) atomicOr(&g_few_error, 1u);
        for (int i = taken_tiles; i < issued; ++i) {
            tc::mbar_wait(&s_full[slot], phase, kWaitLimitNs);
            if (++slot == stages) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
    // what follows counts on attn_many too: the last block, and with it this kernel, ends after it (the others make
    // room for more)
    if (a.beside && blockIdx.x == gridDim.x - 1) mq_grid_wait();
}

template <typename T, int D, bool RAW>
auto few_kernel() {
    return attn_few_kernel<T, D, RAW>;
}

template <typename F>
int with_kernel(int D, int type, bool raw, F f) {
    auto go = [&](auto t) {
        using T = decltype(t);
        switch (D) {
            case 64: return f(raw ? few_kernel<T, 64, true>() : few_kernel<T, 64, false>(), Cfg<64>::kSmem);
            case 96: return f(raw ? few_kernel<T, 96, true>() : few_kernel<T, 96, false>(), Cfg<96>::kSmem);
            case 128: return f(raw ? few_kernel<T, 128, true>() : few_kernel<T, 128, false>(), Cfg<128>::kSmem);
            default: return f(raw ? few_kernel<T, 256, true>() : few_kernel<T, 256, false>(), Cfg<256>::kSmem);
        }
    };
    return type == MQ_F16 ? go(__half()) : go(__nv_bfloat16());
}

}  // namespace

int launch_few(const FewArgs& a, const mq_kv* prefix, const mq_kv* own, int D, int type, cudaStream_t stream) {
    CUtensorMap pk, pv, ok, ov;
    const mq_kv* p = prefix ? prefix : own;   // a part that is not there is never read
    const mq_kv* o = own ? own : prefix;
    const int dims = D % 64 == 0 ? 64 : 32;
    if (!kv_map(&pk, p, p->k, type, dims, kKeys) || !kv_map(&pv, p, p->v, type, dims, kKeys) || !kv_map(&ok, o, o->k, type, dims, kKeys) ||
        !kv_map(&ov, o, o->v, type, dims, kKeys))
        return MQ_ERR_LAUNCH;
    return with_kernel(D, type, a.raw != nullptr, [&](auto kern, int smem) {
        if (!mq::allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3(a.plan.G), dim3(kThreads), smem, stream, a, pk, pv, ok, ov);
    });
}

#ifdef MQ_TEST_INJECT
bool test_skip_few(int on) { return cudaMemcpyToSymbol(g_test_skip_tile, &on, sizeof(on)) == cudaSuccess; }
#endif

int take_few_error(unsigned* code) {
    if (cudaMemcpyFromSymbol(code, g_few_error, sizeof(*code)) != cudaSuccess) return MQ_ERR_LAUNCH;
    const unsigned zero = 0;
    return *code && cudaMemcpyToSymbol(g_few_error, &zero, sizeof(zero)) != cudaSuccess ? MQ_ERR_LAUNCH : MQ_OK;
}

}  // namespace attn
