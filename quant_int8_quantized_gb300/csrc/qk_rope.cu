// Per-head RMS norm of queries and keys with their rotation, and the write of keys and values
// into a cache, in one pass over the f32 projections.
//
// A pair (a, b) of a head is turned by t = pos * inv_freq: (a cos t - b sin t, a sin t + b cos t).
// A thread holds four pairs (two float4: both halves of the head, or eight neighbours), so a
// head is D / 8 lanes of one aligned group of 8, 16 or 32, the sum of squares a few xor shuffles,
// and no value passes through shared memory. Values (v) and dims that are not rotated are the
// same eight numbers a thread, turned by nothing. cos t and sin t depend on token and pair only:
// a block computes them once for all heads of its token, in shared memory, while its first
// heads are on their way.
//
// Bound: HBM, 4 bytes read and 2 written an element (M = 1: latency). Measured: 16384 tokens of 56 heads of 128, 110 us,
// 6.4 TB/s; 3314 tokens of 36, 20.4 us, 4.5 TB/s; one token of 56, 2.6 us.

#include "heads.cuh"

namespace {

constexpr int kThreads = 128;

struct Args {
    const float* x[3];          // q, k, v (NULL: left out)
    long long stride[3];
    const float* w[2];
    const float* inv_freq;
    const uint8_t* axis;
    const int32_t* pos;
    const int32_t* slot;
    void* q_out;
    void* kv[2];
    long long seq_stride, row_stride, head_stride, slots;
    int M, D, n_pairs, n_axes, cap;
    int h0, h1, h2;             // rows of a token: [0, h0) q, [h0, h1) k, [h1, h2) v
    float eps;
};

// cos and sin of pos * freq. The turn is taken out in 64 bits: the product of an int32 and an
// f32 has 55 bits, so no int32 position loses accuracy (in f32 the angle of position 100000 would be
// off by up to 4e-3).
__device__ __forceinline__ float2 turn(int pos, float freq) {
    const double t = (double)pos * (double)freq * 0.31830988618379067154;   // in half turns
    float s, c;
    sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ float dot8(const float (&v)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaf(v[i], v[i], a);
    return a;
}

// LG lanes a head. VEC: pairs come in fours (n_pairs % 4 == 0); otherwise each of a thread's
// four pairs or eight plain numbers is placed by itself.
template <typename T, int LG, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const Args a) {
    extern __shared__ float2 s_turn[];   // [n_pairs]
    mq_grid_release();
    mq_grid_wait();
    const int m = blockIdx.x;            // the token
    const int lane = threadIdx.x % LG;
    const int D = a.D, n = a.n_pairs;
    const int rows = a.h2;
    const int r_first = blockIdx.y * (kThreads / LG) + threadIdx.x / LG, r_step = gridDim.y * (kThreads / LG);

    // a row: which projection and head it is, and this thread's eight numbers of it
    struct Row {
        int what, h, np;
        float v[8];
    };
    // Without VEC, element i of this thread is pair p's (i & 1) member for p = 4 lane + i / 2 < np, and a plain number
    // past that.
    auto place = [&](int np, int i) {
        const int p = lane * 4 + i / 2;
        if (p >= np) return lane * 8 + i;
        return INTER ? 2 * p + (i & 1) : p + (i & 1) * np;
    };
    // With VEC, elements 0 .. 3 lie at low(np), 4 .. 7 at high(np).
    auto low = [&](int np) { return INTER || lane * 4 >= np ? lane * 8 : lane * 4; };
    auto high = [&](int np) { return INTER || lane * 4 >= np ? lane * 8 + 4 : np + lane * 4; };
    auto fetch = [&](int r, Row& x) {
        const bool live = r < rows && lane * 8 < D;
        const int hr = live ? r : 0;
        x.what = hr < a.h0 ? 0 : hr < a.h1 ? 1 : 2;
        x.h = hr - (x.what == 0 ? 0 : x.what == 1 ? a.h0 : a.h1);
        x.np = x.what == 2 ? 0 : n;
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] = 0.0f;
        if (!live) return;
        const float* p = a.x[x.what] + (long long)m * a.stride[x.what] + (long long)x.h * D;
        if constexpr (VEC) {
            const float4 u0 = __ldcs(reinterpret_cast<const float4*>(p + low(x.np)));
            const float4 u1 = __ldcs(reinterpret_cast<const float4*>(p + high(x.np)));
            x.v[0] = u0.x, x.v[1] = u0.y, x.v[2] = u0.z, x.v[3] = u0.w;
            x.v[4] = u1.x, x.v[5] = u1.y, x.v[6] = u1.z, x.v[7] = u1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.v[i] = __ldcs(p + place(x.np, i));
        }
    };
    Row now;
    fetch(r_first, now);             // on its way while the turns are computed

    for (int p = threadIdx.x; p < n; p += kThreads) {
        const int ax = a.axis ? min((int)a.axis[p], a.n_axes - 1) : 0;
        s_turn[p] = turn(a.pos[(long long)ax * a.M + m], a.inv_freq[p]);
    }
    __syncthreads();
    for (int r = r_first; r - (int)(threadIdx.x / LG) < rows; r += r_step) {
        Row next;
        fetch(r + r_step, next);     // (past the last row: nothing)
        const bool live = r < rows && lane * 8 < D;
        const int what = now.what, h = now.h, np = now.np;
        const int lo = low(np), hi = high(np);
        const bool rot = lane * 4 < np;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = now.v[i];
        now = next;
        const float* w = what == 2 ? nullptr : a.w[what];
        float ss = dot8(v);
#pragma unroll
        for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!live) continue;
        if (w) {
            const float sc = 1.0f / sqrtf(ss / (float)D + a.eps);
            if constexpr (VEC) {
                const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + lo));
                const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + hi));
                v[0] *= sc * w0.x, v[1] *= sc * w0.y, v[2] *= sc * w0.z, v[3] *= sc * w0.w;
                v[4] *= sc * w1.x, v[5] *= sc * w1.y, v[6] *= sc * w1.z, v[7] *= sc * w1.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= sc * __ldg(w + place(np, i));
            }
        }
        const float2* tt = s_turn;
        auto rotate = [](float& p, float& q, float2 t) {
            const float u = p * t.x - q * t.y;
            q = p * t.y + q * t.x;
            p = u;
        };
        if constexpr (VEC) {
            if (rot) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (INTER) rotate(v[2 * i], v[2 * i + 1], tt[lane * 4 + i]);
                    else rotate(v[i], v[4 + i], tt[lane * 4 + i]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane * 4 + i < np) rotate(v[2 * i], v[2 * i + 1], tt[lane * 4 + i]);
        }
        T* y;
        if (what == 0) {
            y = reinterpret_cast<T*>(a.q_out) + ((long long)m * a.h0 + h) * D;
        } else {
            const long long s = a.slot ? (long long)a.slot[m] : (long long)m;
            if (s < 0 || s >= a.slots) continue;
            const long long seq = s / a.cap;
            y = reinterpret_cast<T*>(a.kv[what - 1]) + seq * a.seq_stride + (s - seq * a.cap) * a.row_stride +
                h * a.head_stride;
        }
        if constexpr (VEC) {
            const uint2 y0 = make_uint2(mq_pack2<T>(v[0], v[1]), mq_pack2<T>(v[2], v[3]));
            const uint2 y1 = make_uint2(mq_pack2<T>(v[4], v[5]), mq_pack2<T>(v[6], v[7]));
            if (INTER || !rot) {
                *reinterpret_cast<uint4*>(y + lo) = make_uint4(y0.x, y0.y, y1.x, y1.y);
            } else {
                *reinterpret_cast<uint2*>(y + lo) = y0;
                *reinterpret_cast<uint2*>(y + hi) = y1;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[place(np, i)] = T(v[i]);
        }
    }
}

template <typename T, int LG>
int launch(const Args& a, bool inter, dim3 grid, size_t smem, cudaStream_t stream) {
    const bool vec = a.n_pairs % 4 == 0;
    auto kern = vec ? (inter ? qk_norm_rope_kernel<T, LG, true, true> : qk_norm_rope_kernel<T, LG, false, true>)
                    : (inter ? qk_norm_rope_kernel<T, LG, true, false> : qk_norm_rope_kernel<T, LG, false, false>);
    return mq::launch_pdl(kern, grid, dim3(kThreads), smem, stream, a);
}

}  // namespace

extern "C" int mq_qk_norm_rope(const mq_qkv* x, void* q_out, const mq_kv* cache, const int32_t* slot,
                               cudaStream_t stream) {
    if (!x) return MQ_ERR_NULL;
    int rc = mq::check_kv(cache, false);
    if (rc != MQ_OK) return rc;
    const int D = cache->dim, Hkv = cache->heads;
    if (x->M < 0 || x->Hq < 0 || x->n_pairs < 0 || 2 * x->n_pairs > D) return MQ_ERR_SHAPE;
    if (x->n_pairs > 0 && (x->n_axes < 1 || x->n_axes > 8)) return MQ_ERR_SHAPE;
    const long long slots = (long long)cache->n * cache->cap;
    if (x->M == 0) return MQ_OK;
    const bool cached = x->k || x->v;
    if (cached && !slot && x->M > slots) return MQ_ERR_SHAPE;
    const float* src[3] = {x->q, x->k, x->v};
    const long long st[3] = {x->q_stride, x->k_stride, x->v_stride};
    const int heads[3] = {x->q ? x->Hq : 0, x->k ? Hkv : 0, x->v ? Hkv : 0};
    for (int i = 0; i < 3; ++i)
        if (src[i]) {
            if (st[i] < (long long)heads[i] * D || st[i] % 4 != 0 || (x->M > 1 && st[i] > mq::kTokenStrideMost)) return MQ_ERR_SHAPE;
            if (!mq::aligned16(src[i])) return MQ_ERR_ALIGN;
        }
    if (x->n_pairs > 0 && (!x->inv_freq || !x->pos)) return MQ_ERR_NULL;
    if ((heads[0] > 0 && !q_out) || (x->k && slots > 0 && !cache->k) || (x->v && slots > 0 && !cache->v))
        return MQ_ERR_NULL;
    if (!mq::aligned16(q_out) || !mq::aligned16(cache->k) || !mq::aligned16(cache->v) || !mq::aligned16(x->wq) ||
        !mq::aligned16(x->wk) || !mq::aligned16(x->inv_freq) || !mq::aligned16(x->axis) || !mq::aligned16(x->pos) ||
        !mq::aligned16(slot))
        return MQ_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)   // a block's output rows would lie over what others have yet to read
        if (mq::rows_meet(src[i], x->M, 4 * st[i], 4LL * heads[i] * D, q_out, 2LL * x->M * heads[0] * D)) return MQ_ERR_SHAPE;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    Args a;
    for (int i = 0; i < 3; ++i) {
        a.x[i] = src[i];
        a.stride[i] = st[i];
    }
    a.w[0] = x->wq;
    a.w[1] = x->wk;
    a.inv_freq = x->inv_freq;
    a.axis = x->axis;
    a.pos = x->pos;
    a.slot = slot;
    a.q_out = q_out;
    a.kv[0] = cache->k;
    a.kv[1] = cache->v;
    a.seq_stride = cache->seq_stride;
    a.row_stride = cache->row_stride;
    a.head_stride = cache->head_stride;
    a.slots = slots;
    a.M = x->M;
    a.D = D;
    a.n_pairs = x->n_pairs;
    a.n_axes = x->n_axes;
    a.cap = cache->cap > 0 ? cache->cap : 1;
    a.h0 = heads[0];
    a.h1 = a.h0 + heads[1];
    a.h2 = a.h1 + heads[2];
    a.eps = x->eps;
    if (a.h2 == 0) return MQ_OK;
    const int lg = D <= 64 ? 8 : D <= 128 ? 16 : 32, per = kThreads / lg;
    // A block takes a token, all its heads (measured at 3314 tokens of 36 heads of 128: 20.4 us; 256 threads with 1, 2, 3, 4
    // and 5 tokens: 26.2, 23.6, 23.1, 23.0 and 25.6); the heads of a few tokens are spread over blocks of one pass each.
    const int passes = (a.h2 + per - 1) / per;
    const dim3 grid(x->M, x->M >= 2 * mq::num_sms() ? 1 : passes < 65535 ? passes : 65535);
    const size_t smem = (size_t)a.n_pairs * sizeof(float2);
    const bool inter = x->interleaved != 0;
    auto go = [&](auto t) {
        using T = decltype(t);
        return lg == 8 ? launch<T, 8>(a, inter, grid, smem, stream)
               : lg == 16 ? launch<T, 16>(a, inter, grid, smem, stream)
                          : launch<T, 32>(a, inter, grid, smem, stream);
    };
    return cache->type == MQ_F16 ? go(__half()) : go(__nv_bfloat16());
}
