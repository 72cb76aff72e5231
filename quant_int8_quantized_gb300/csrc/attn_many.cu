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
// products. The maximum that the exponents are taken against is renewed only when a row passes it by 2^8
// (the sums are the same in any scale, and 2^8 does not bring a 16-bit value near its end), so O in
// tensor memory is hardly ever scaled again.
//
// 384 threads, one block per SM: warps 0-3 and 4-7 the rows of the halves, warp 8 TMA, warp 9 the
// products; the register file is shared out again to give a row's thread its 128 products. Shared memory: Q (64 KB at D = 128) and a ring of K and V tiles (32 KB each).
// Waits are bounded; a wait that runs out is recorded (mq_device_status), the block drains its own copies
// and products, frees tensor memory and returns.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <map>
#include <mutex>
#include <type_traits>

#include "attn_many.cuh"
#include "tc.cuh"

namespace attn {
namespace {

__device__ unsigned int g_attn_error;   // bit 0: a bounded wait gave up

#ifndef MQ_WAIT_LIMIT_NS
#define MQ_WAIT_LIMIT_NS 2000000000ull   // test builds may shorten it
#endif
constexpr uint64_t kWaitLimitNs = MQ_WAIT_LIMIT_NS;

constexpr int kThreads = 384;
// Registers a thread: what the launch gives to 384 threads, and after sharing out again (2 x 208 + 88 = 3 x 168).
constexpr int kLaunchRegs = 168, kRowRegs = 208, kOtherRegs = 88;
constexpr int kHalf = 128;
constexpr int kKeys = kManyKeys;
constexpr uint32_t kTmemCols = 512;
constexpr float kGrow = 8.0f;           // powers of two by which a row may pass its maximum

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;                       // 128-byte columns of a row
    static constexpr int kChunkBytes = 128 * 128;                // 128 rows of one
    static constexpr int kTileBytes = kChunks * kChunkBytes;     // a K or V tile, a half of Q
    static constexpr int kRing = D == 128 ? 5 : 10;
    static constexpr int kSmem = 1024 + (2 + kRing) * kTileBytes;
};

struct Bars {
    uint64_t full[10], empty[10];
    uint64_t q_ready[2], s_full[2], p_ready[2], pv_done[2];
    uint64_t drained;
    uint32_t tmem;
    int abort;
};

// Whole warp, or any set of threads of one whose outcome need not be uniform with the others.
__device__ bool wait(Bars& b, uint64_t* bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
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
    return __all_sync(0xffffffffu, wait(b, bar, parity));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(tc::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
        : "memory");
}

// 128-byte swizzle, the other axis contiguous: rows of 64 elements (128 bytes) are steps of the product's K axis;
// 8 rows are an atom of 1024 bytes, `lbo` bytes lie between chunks of 64 elements.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// What a role keeps of the segment that its cursor is in.
struct Seg {
    int b, r0, rows, len, halves;
};
__device__ __forceinline__ Seg segment_of(const Plan& p, const int32_t* len, const Cursor& c) {
    Seg s;
    const int per_seq = own_tiles_of_rows(p);
    s.b = c.prefix ? 0 : c.unit / per_seq;
    s.r0 = (c.prefix ? c.unit : c.unit - s.b * per_seq) * kManyRows;
    s.rows = min(kManyRows, (c.prefix ? p.prefix_rows : p.T * p.group) - s.r0);
    s.len = c.prefix ? p.prefix_keys : own_len_of(p, len, s.b);
    s.halves = s.rows > kHalf ? 2 : 1;
    return s;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_many_kernel(const ManyArgs a, const __grid_constant__ CUtensorMap pk, const __grid_constant__ CUtensorMap pv,
                     const __grid_constant__ CUtensorMap ok, const __grid_constant__ CUtensorMap ov) {
    using C = Cfg<D>;
    extern __shared__ uint8_t s_raw[];
    __shared__ Bars s_bars;
    Bars& bars = s_bars;
    uint8_t* smem = s_raw + ((1024 - (tc::smem_u32(s_raw) & 1023)) & 1023);
    uint8_t* s_q = smem;                            // two halves
    uint8_t* s_ring = smem + 2 * C::kTileBytes;
    const Plan& p = a.plan;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;

    mq_grid_release();
    if (tid == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            tc::mbar_init(&bars.full[i], 1);
            tc::mbar_init(&bars.empty[i], 1);
        }
        for (int h = 0; h < 2; ++h) {
            tc::mbar_init(&bars.q_ready[h], kHalf);
            tc::mbar_init(&bars.s_full[h], 1);
            tc::mbar_init(&bars.p_ready[h], kHalf);
            tc::mbar_init(&bars.pv_done[h], 1);
        }
        tc::mbar_init(&bars.drained, 1);
        bars.abort = 0;
        tc::fence_mbar_init();
    }
    if (wid == 9) tc::tmem_alloc(&bars.tmem, kTmemCols);
    if (wid == 8 && lane == 0) {
        tc::prefetch_tensormap(&pk);
        tc::prefetch_tensormap(&pv);
        tc::prefetch_tensormap(&ok);
        tc::prefetch_tensormap(&ov);
    }
    mq_grid_wait();
    tc::tc_fence_before();
    Cursor c = find_run<kThreads>(p, a.len);   // holds block barriers
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (wid < 8) {
        tc::setmaxnreg_inc<kRowRegs>();
        // ---------------------------------------------------------------- rows: a thread each
        const int h = wid >> 2, row = (wid & 3) * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(wid & 3) * 32 << 16);
        const uint32_t s_col = lane_base + h * 128, o_col = lane_base + 256 + h * 128;
        uint32_t s_phase = 0, pv_phase = 0;
        bool alive = true;
        while (alive && c.tile < c.end) {
            const int nt = (int)min((long long)(c.seg_tiles - c.in), c.end - c.tile);
            const Seg g = segment_of(p, a.len, c);
            if (tid == 0 && c.in == 0)
                a.out.info[c.seg] = make_int2(blockIdx.x, block_of(c.tile + c.seg_tiles - 1, c.total, c.blocks));
            const bool mine = h < g.halves;
            const int r = g.r0 + h * kHalf + row;            // row of the segment's row space
            const bool live = h * kHalf + row < g.rows;
            // the row of Q into shared memory, as TMA would lay it (16-byte units xor row % 8)
            if (mine) {
                const int q_row = r / p.group, q_in = r - q_row * p.group;   // b T + t (own: t), head in the group
                const uint4* q = reinterpret_cast<const uint4*>(
                    static_cast<const T*>(a.q) +
                    (live ? ((long long)q_row + (c.prefix ? 0 : (long long)g.b * p.T)) * a.q_stride +
                                (long long)(c.head * p.group + q_in) * D
                          : 0));
                uint8_t* dst = s_q + h * C::kTileBytes + row * 128;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 x = live ? __ldca(q + i) : make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(dst + (i / 8) * C::kChunkBytes + (((i & 7) ^ (row & 7)) << 4)) = x;
                }
                tc::fence_proxy_async_smem();
                tc::mbar_arrive(&bars.q_ready[h]);
            }
            const int seen = c.prefix ? g.len : g.len - p.T + 1 + r / p.group;
            float m = -INFINITY, l = 0.0f;                    // base 2, scaled
            if (mine) {
                for (int j = 0; j < nt; ++j) {
                    if (!(alive = wwait(bars, &bars.s_full[h], s_phase))) break;
                    s_phase ^= 1;
                    tc::tc_fence_after();
                    uint32_t s[4][32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc::tmem_ld32(s_col + k * 32, s[k]);
                    tc::tmem_ld_wait();
                    const int k0 = (c.in + j) * kKeys;
                    if (__any_sync(0xffffffffu, k0 + kKeys > seen)) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (k0 + k * 32 + i >= seen) s[k][i] = 0xff800000u;   // -infinity
                    }
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(s[k][i]));
                    mx *= a.scale_log2;
                    const bool grew = mx > m + kGrow;          // true for the first key that a row sees
                    if (j == 0) {
                        m = mx;
                    } else if (__any_sync(0xffffffffu, grew)) {
                        const float now = fmaxf(m, mx);
                        const float f = now == -INFINITY ? 1.0f : exp2_fast(m - now);
                        m = now;
                        l *= f;
                        // the product before this one must be done with O
                        if (!(alive = wwait(bars, &bars.pv_done[h], pv_phase ^ 1))) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            uint32_t o[32];
                            tc::tmem_ld32(o_col + k * 32, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc::tmem_st32(o_col + k * 32, o);
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : m;
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pr[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = f2_fma(make_float2(__uint_as_float(s[k][2 * i]), __uint_as_float(s[k][2 * i + 1])),
                                                    f2_dup(a.scale_log2), f2_dup(-base));
                            const float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
                            sum[0] += e0;
                            sum[1] += e1;
                            pr[i] = mq_pack2<T>(e0, e1);
                        }
                        tc::tmem_st16(s_col + k * 16, pr);
                    }
                    l += sum[0] + sum[1];
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars.p_ready[h]);
                    pv_phase ^= 1;
                }
                if (alive) alive = wwait(bars, &bars.pv_done[h], pv_phase ^ 1);
                if (alive) {
                    tc::tc_fence_after();
                    const long long place = (long long)blockIdx.x + c.seg;
                    const long long at = place * kManyRows + h * kHalf + row;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t o[32];
                        tc::tmem_ld32(o_col + k * 32, o);
                        tc::tmem_ld_wait();
                        if (live) {
                            float4* to = reinterpret_cast<float4*>(a.out.o + at * D + k * 32);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                to[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                    __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                        }
                    }
                    tc::tc_fence_before();
                    if (live) a.out.ml[at] = make_float2(m, l);
                }
            }
            c.tile += nt;
            if (c.tile < c.end) next_segment(p, a.len, c);
        }
    } else {
        tc::setmaxnreg_dec<kOtherRegs>();
        if (wid == 8) {
        // ---------------------------------------------------------------- TMA
        int slot = 0, issued = 0;
        uint32_t phase = 0;
        bool alive = true;
        while (alive && c.tile < c.end) {
            const int nt = (int)min((long long)(c.seg_tiles - c.in), c.end - c.tile);
            const Seg g = segment_of(p, a.len, c);
            for (int j = 0; alive && j < nt; ++j)
                for (int kv = 0; kv < 2; ++kv) {
                    if (!(alive = wwait(bars, &bars.empty[slot], phase ^ 1))) break;
                    if (tc::elect_one()) {
                        const CUtensorMap* map = c.prefix ? (kv ? &pv : &pk) : (kv ? &ov : &ok);
                        tc::mbar_arrive_expect_tx(&bars.full[slot], C::kTileBytes);
#pragma unroll
                        for (int k = 0; k < C::kChunks; ++k)
                            tma_load_4d(s_ring + slot * C::kTileBytes + k * C::kChunkBytes, map, k * 64, c.head,
                                        (c.in + j) * kKeys, g.b, &bars.full[slot]);
                    }
                    __syncwarp();
                    ++issued;
                    if (++slot == C::kRing) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            c.tile += nt;
            if (c.tile < c.end) next_segment(p, a.len, c);
        }
        if (!alive) {   // copies in flight must land before the block leaves
            for (int i = 0; i < C::kRing && i < issued; ++i) {
                if (--slot < 0) {
                    slot = C::kRing - 1;
                    phase ^= 1;
                }
                tc::mbar_wait(&bars.full[slot], phase, kWaitLimitNs);
            }
        }
        } else if (wid == 9) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        const uint32_t idesc_qk = tc::instr_desc(kHalf, kKeys, fmt) | (a.negative ? 1u << 13 : 0u);
        const uint32_t idesc_pv = tc::instr_desc(kHalf, D, fmt) | 1u << 16;   // V: the N axis contiguous
        const uint32_t q_addr = tc::smem_u32(s_q), ring = tc::smem_u32(s_ring);
        int slot = 0;
        uint32_t phase = 0, q_phase = 0, p_phase = 0;   // q, p: a bit per half
        bool alive = true;
        auto next_slot = [&] {
            if (++slot == C::kRing) {
                slot = 0;
                phase ^= 1;
            }
        };
        while (alive && c.tile < c.end) {
            const int nt = (int)min((long long)(c.seg_tiles - c.in), c.end - c.tile);
            const Seg g = segment_of(p, a.len, c);
            for (int h = 0; alive && h < g.halves; ++h) alive = wwait(bars, &bars.q_ready[h], q_phase >> h & 1);
            if (!alive) break;
            const uint32_t both = g.halves == 2 ? 3 : 1;
            q_phase ^= both;
            auto qk = [&](int h, int k_slot) {
                if (tc::elect_one()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k / 4) * C::kChunkBytes + (k % 4) * 32;
                        tc::mma_f16(tmem + h * 128, tc::smem_desc_sw128(q_addr + h * C::kTileBytes + off),
                                    tc::smem_desc_sw128(ring + k_slot * C::kTileBytes + off), idesc_qk, k > 0);
                    }
                    tc::mma_commit(&bars.s_full[h]);
                    if (h == g.halves - 1) tc::mma_commit(&bars.empty[k_slot]);
                }
                __syncwarp();
            };
            if (!(alive = wwait(bars, &bars.full[slot], phase))) break;
            tc::tc_fence_after();
            for (int h = 0; h < g.halves; ++h) qk(h, slot);
            next_slot();
            for (int j = 0; alive && j < nt; ++j) {
                if (!(alive = wwait(bars, &bars.full[slot], phase))) break;
                const int v_slot = slot;
                next_slot();
                const int k0 = (c.in + j) * kKeys;
                if (k0 + kKeys > g.len && !c.prefix) {
                    // rows past the length may hold anything: zeros times a probability of zero
                    for (int i = lane; i < (k0 + kKeys - g.len) * 8; i += 32)
#pragma unroll
                        for (int k = 0; k < C::kChunks; ++k)
                            *reinterpret_cast<uint4*>(s_ring + v_slot * C::kTileBytes + k * C::kChunkBytes +
                                                      (g.len - k0) * 128 + i * 16) = make_uint4(0, 0, 0, 0);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                for (int h = 0; h < g.halves; ++h) {
                    if (!(alive = wwait(bars, &bars.p_ready[h], p_phase >> h & 1))) break;
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            tc::mma_f16_ts(tmem + 256 + h * 128, tmem + h * 128 + k * 8,
                                           smem_desc_sw128_mn(ring + v_slot * C::kTileBytes + k * 2048, C::kChunkBytes),
                                           idesc_pv, j > 0 || k > 0);
                        tc::mma_commit(&bars.pv_done[h]);
                        if (h == g.halves - 1) tc::mma_commit(&bars.empty[v_slot]);
                    }
                    __syncwarp();
                    if (j + 1 < nt) {
                        if (h == 0 && !(alive = wwait(bars, &bars.full[slot], phase))) break;
                        qk(h, slot);
                        if (h == g.halves - 1) next_slot();
                    }
                }
                p_phase ^= both;
            }
            c.tile += nt;
            if (c.tile < c.end) next_segment(p, a.len, c);
        }
        if (tc::elect_one()) tc::mma_commit(&bars.drained);
        __syncwarp();
        tc::mbar_wait(&bars.drained, 0, kWaitLimitNs);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (wid == 9) tc::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

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

// [n][cap][heads][dim] of k or v as (dim, head, row, sequence); rows past the cap read as zeros.
bool kv_map(CUtensorMap* map, const mq_kv* c, const void* base) {
    auto fn = encode_fn();
    if (!fn) return false;
    auto stride = [](long long s) { return (cuuint64_t)(s > 0 ? s * 2 : 16); };   // an axis of one step may have none
    const cuuint64_t dims[4] = {(cuuint64_t)c->dim, (cuuint64_t)c->heads, (cuuint64_t)c->cap, (cuuint64_t)c->n};
    const cuuint64_t strides[3] = {stride(c->head_stride), stride(c->row_stride), stride(c->seq_stride)};
    const cuuint32_t box[4] = {64, 1, kManyKeys, 1}, step[4] = {1, 1, 1, 1};
    return fn(map, c->type == MQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
              const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_many(const ManyArgs& a, const mq_kv* prefix, const mq_kv* own, int D, int type, cudaStream_t stream) {
    CUtensorMap pk, pv, ok, ov;
    const mq_kv* p = prefix ? prefix : own;   // a part that is not there is never read
    const mq_kv* o = own ? own : prefix;
    if (!kv_map(&pk, p, p->k) || !kv_map(&pv, p, p->v) || !kv_map(&ok, o, o->k) || !kv_map(&ov, o, o->v))
        return MQ_ERR_LAUNCH;
    auto go = [&](auto kern, int smem) {
        if (!regs_as_planned(reinterpret_cast<const void*>(kern))) return (int)MQ_ERR_LAUNCH;
        if (!allow_smem(reinterpret_cast<const void*>(kern), smem)) return (int)MQ_ERR_LAUNCH;
        return mq::launch_pdl(kern, dim3(a.plan.G), dim3(kThreads), smem, stream, a, pk, pv, ok, ov);
    };
    if (type == MQ_F16)
        return D == 64 ? go(attn_many_kernel<__half, 64>, Cfg<64>::kSmem) : go(attn_many_kernel<__half, 128>, Cfg<128>::kSmem);
    return D == 64 ? go(attn_many_kernel<__nv_bfloat16, 64>, Cfg<64>::kSmem)
                   : go(attn_many_kernel<__nv_bfloat16, 128>, Cfg<128>::kSmem);
}

}  // namespace attn

namespace mq {
int take_attn_device_error(cudaStream_t stream, unsigned* code) {
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MQ_ERR_LAUNCH;
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, attn::g_attn_error, sizeof(v)) != cudaSuccess) return MQ_ERR_LAUNCH;
    if (v) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(attn::g_attn_error, &zero, sizeof(zero)) != cudaSuccess) return MQ_ERR_LAUNCH;
    }
    *code = v;
    return MQ_OK;
}
}  // namespace mq
