// Attention pieces for few query rows per key head (up to 16 a segment): every key and value is
// read once and used for a handful of rows, so HBM bounds and the matrix products only have to keep
// out of the way. They run as warp-wide 16 x 8 x 16 products in registers.
//
// Four warps share a tile of 64 keys, 16 each, and never wait for one another: a warp copies its own
// keys and values into its own ring of stages (asynchronous 16-byte copies, rows past the end filled
// with zeros, so nothing that lies there can reach a sum), multiplies, keeps its own running
// maximum, sum and output, and the four are joined at the end of the piece. The products q k^T come out
// in the layout that the second product takes as its left operand, so probabilities stay in registers.
// Rows of a stage are padded by 16 bytes: eight rows of an 8 x 8 matrix load then fall into eight
// different groups of banks.

#include "attn_few.cuh"
#include "tc.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 16;              // keys per warp and tile
constexpr int kTile = kWarps * kKeys;

template <int D>
struct Cfg {
    static constexpr int kPitch = D * 2 + 16;                 // bytes of a row of a stage
    static constexpr int kStageBytes = 2 * kKeys * kPitch;    // keys, then values
    static constexpr int kStages = D <= 128 ? 3 : 2;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // the ring's memory takes the warps' outputs at the end of a piece
    static constexpr int kJoin = kWarps * kFewRows * D * 4;
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
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

template <typename T, int D, bool RAW>
__global__ void __launch_bounds__(kThreads) attn_few_kernel(const FewArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ float2 s_ml[kWarps][kFewRows];
    mq_grid_release();
    mq_grid_wait();
    const Plan& p = a.plan;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int tg = p.T * p.group;
    Cursor c = find_run<kThreads>(p, a.len);
    const uint32_t ring = tc::smem_u32(s_ring) + wid * (C::kStages * C::kStageBytes);
    const int g = lane >> 2, t2 = (lane & 3) * 2;   // this thread's rows g, g + 8 and columns t2, t2 + 1

    advance(p, a.len, c, 0);
    while (c.more()) {
        const int nt = piece_tiles(p, c);
        const int key0 = c.in * kTile;
        // the segment's rows and keys
        const int per_seq = own_tiles_of_rows(p);
        const int b = c.prefix ? 0 : p.by_per_seq.of(c.unit);
        const int r0 = (c.prefix ? c.unit : c.unit - b * per_seq) * kFewRows;
        const int nrows = min(kFewRows, (c.prefix ? p.prefix_rows : tg) - r0);
        const int len = c.prefix ? p.prefix_keys : own_len_of(p, a.len, b);
        const long long row_stride = c.prefix ? a.p_row : a.o_row;
        const long long base = c.prefix ? c.head * a.p_head : b * a.o_seq + c.head * a.o_head;
        const T* K = static_cast<const T*>(c.prefix ? a.pk : a.ok) + base;
        const T* V = static_cast<const T*>(c.prefix ? a.pv : a.ov) + base;
        if (tid == 0 && c.in == 0)
            a.out.info[c.seg] = blocks_of(p, c);

        auto copy = [&](int t) {   // tile t of the piece into its stage
            if (t < nt) {
                const uint32_t st = ring + (t % C::kStages) * C::kStageBytes;
                const int k0 = key0 + t * kTile + wid * kKeys;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int ch = i * 32 + lane, kr = ch / (D / 8), kc = ch % (D / 8);
                    const bool in = k0 + kr < len;
                    const long long off = (in ? k0 + kr : 0) * row_stride + kc * 8;
                    tc::cp_async16_zfill(st + kr * C::kPitch + kc * 16, K + off, in ? 16 : 0);
                    tc::cp_async16_zfill(st + (kKeys + kr) * C::kPitch + kc * 16, V + off, in ? 16 : 0);
                }
            }
            tc::cp_async_commit();
        };
#pragma unroll
        for (int t = 0; t < C::kStages - 1; ++t) copy(t);

        // query rows g and g + 8 (zeros past the last), as left operands; the keys that each sees
        uint32_t qf[D / 16][4];
        int seen[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = r0 + g + 8 * u;
            const bool live = g + 8 * u < nrows;
            const int t = p.by_group.of(r), h = c.head * p.group + r - t * p.group;   // prefix: t is b T + t
            seen[u] = c.prefix ? len : len - p.T + 1 + t;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) +
                                                                  (live ? ((long long)b * p.T + t) * a.q_stride + h * D : 0));
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][u] = live ? __ldca(q + (k * 16 + t2) / 2) : 0u;
                qf[k][u + 2] = live ? __ldca(q + (k * 16 + 8 + t2) / 2) : 0u;
            }
        }
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};

        for (int t = 0; t < nt; ++t) {
            copy(t + C::kStages - 1);
            tc::cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t st = ring + (t % C::kStages) * C::kStageBytes;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t kf[4];
                ldm4(st + ((lane >> 4) * 8 + (lane & 7)) * C::kPitch + (k * 16 + ((lane >> 3) & 1) * 8) * 2, kf);
                mma<T>(s[0], qf[k], kf[0], kf[1]);
                mma<T>(s[1], qf[k], kf[2], kf[3]);
            }
            const int k0 = key0 + t * kTile + wid * kKeys;
            float mx[2] = {m[0], m[1]};
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + j * 8 + t2 + (e & 1);
                    s[j][e] = key < seen[e >> 1] ? s[j][e] * a.scale_log2 : kNone;
                    mx[e >> 1] = fmaxf(mx[e >> 1], s[j][e]);
                }
            if constexpr (RAW) {
                if (!c.prefix) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (g + 8 * u < nrows) {
                            float* raw = a.raw + (((long long)b * p.Hkv + c.head) * tg + r0 + g + 8 * u) * p.own_cap;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (k0 + j * 8 + t2 + e < len) raw[k0 + j * 8 + t2 + e] = s[j][2 * u + e];
                        }
                }
            }
            float alpha[2];
            bool grew = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
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
                ldm4t(st + (kKeys + ((lane >> 3) & 1) * 8 + (lane & 7)) * C::kPitch + (i * 16 + (lane >> 4) * 8) * 2, vf);
                mma<T>(o[2 * i], pf, vf[0], vf[1]);
                mma<T>(o[2 * i + 1], pf, vf[2], vf[3]);
            }
            __syncwarp();   // the stage may be written again
        }
        tc::cp_async_wait<0>();
        // join the four warps
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
            l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
            if ((lane & 3) == 0) s_ml[wid][g + 8 * u] = make_float2(m[u], l[u]);
        }
        __syncthreads();
        float* join = reinterpret_cast<float*>(s_ring);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float mm = kNone;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][g + 8 * u].x);
            const float f = exp2_fast(m[u] - (mm == kNone ? 0.0f : mm));
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2*>(join + (wid * kFewRows + g + 8 * u) * D + i * 8 + t2) =
                    make_float2(o[i][2 * u] * f, o[i][2 * u + 1] * f);
        }
        __syncthreads();
        const long long place = (long long)blockIdx.x + c.seg;
        for (int i = tid; i < nrows * (D / 4); i += kThreads) {
            float4 sum = *reinterpret_cast<const float4*>(join + i * 4);
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(join + w * kFewRows * D + i * 4);
                sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
            }
            *reinterpret_cast<float4*>(a.out.o + place * kFewRows * D + i * 4) = sum;
        }
        if (tid < nrows) {
            float mm = kNone, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][tid].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) ll += s_ml[w][tid].y * exp2_fast(s_ml[w][tid].x - (mm == kNone ? 0.0f : mm));
            a.out.ml[place * kFewRows + tid] = make_float2(mm, ll);
        }
        __syncthreads();   // s_ml and the ring are free again
        advance(p, a.len, c, nt);
    }
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

int few_tile_keys(int) { return kTile; }

int few_blocks(int D, int type) {
    return with_kernel(D, type, false, [](auto kern, int smem) {
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return mq::num_sms();
        return mq::num_sms() * mq::resident_blocks(reinterpret_cast<const void*>(kern), kThreads, smem);
    });
}

int launch_few(const FewArgs& a, int D, int type, cudaStream_t stream) {
    return with_kernel(D, type, a.raw != nullptr, [&](auto kern, int smem) {
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3(a.plan.G), dim3(kThreads), smem, stream, a);
    });
}

}  // namespace attn
