// How a row's pieces (attn.cuh) are added up and the row is written, by one warp.
#pragma once

#include "attn.cuh"

namespace attn {

// Pieces of a row: `count` of them, `stride` rows apart, the first at row `first` of the pieces.
struct Run {
    const Pieces* p;
    long long first, stride;
    int count;
};

// Pieces of row `in` of a segment whose blocks are f.x .. f.y; none where these are no blocks (a kernel that gave up on
// a wait leaves entries unwritten).
__device__ __forceinline__ Run run_of(const Part& p, int seg, int2 f, int in) {
    const bool ok = f.x >= 0 && f.y >= f.x && f.y < p.plan.G / p.plan.lanes;
    return Run{&p.p, ok ? (long long)place_of(p.plan, f.x, seg) * p.rows + in : 0, p.rows, ok ? f.y - f.x + 1 : 0};
}

// A lane's part of a row of D floats: V floats at V (lane + 32 k), k < W.
template <int D>
struct Lane {
    static constexpr int V = D >= 128 ? 4 : 2, W = (D + 32 * V - 1) / (32 * V);
};
// Maximum, sum and (this lane's part of the) output of some pieces of a row.
template <int D>
struct Sum {
    float m, l, o[Lane<D>::W][Lane<D>::V];
};

// One warp adds up pieces i0 .. i1 - 1 of a row, counted over run 0 and then run 1: their common maximum, then
// outputs weighted and added in order. Lane i holds place, maximum and sum of piece i of 32; the outputs' loads do
// not depend on one another, kAtOnce (a divisor of 32) are asked for at once.
template <int D, int kAtOnce>
__device__ __forceinline__ Sum<D> add_pieces(const Run& r0, const Run& r1, int i0, int i1) {
    constexpr int V = Lane<D>::V, W = Lane<D>::W;
    const int lane = threadIdx.x & 31;
    Sum<D> s = {-INFINITY, 0.0f, {}};
#pragma unroll 1
    for (; i0 < i1; i0 += 32) {
        const int n = min(32, i1 - i0), i = i0 + lane;
        const bool second = i >= r0.count;
        const Run& r = second ? r1 : r0;
        const long long at = r.first + (second ? i - r0.count : i) * r.stride;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (lane < n) ml = __ldca(r.p->ml + at);
        const unsigned long long from = reinterpret_cast<unsigned long long>(lane < n ? r.p->o + at * D : nullptr);
        float now = fmaxf(s.m, ml.x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
        const float safe = now == -INFINITY ? 0.0f : now;
        const float back = exp2f(s.m - safe), f = exp2f(ml.x - safe);
        s.m = now;
        float sum = ml.y == 0.0f ? 0.0f : ml.y * f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s.l = s.l * back + sum;
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) s.o[k][e] *= back;
#pragma unroll 1
        for (int j0 = 0; j0 < n; j0 += kAtOnce) {
            float x[kAtOnce][W][V], g[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                g[j] = __shfl_sync(0xffffffffu, f, j0 + j);
                const float* oi = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, from, j0 + j));
#pragma unroll
                for (int k = 0; k < W; ++k) {
#pragma unroll
                    for (int e = 0; e < V; ++e) x[j][k][e] = 0.0f;
                    if (j0 + j < n && V * (k * 32 + lane) < D) {
                        if constexpr (V == 4) {
                            const float4 v = __ldca(reinterpret_cast<const float4*>(oi) + k * 32 + lane);
                            x[j][k][0] = v.x, x[j][k][1] = v.y, x[j][k][2] = v.z, x[j][k][3] = v.w;
                        } else {
                            const float2 v = __ldca(reinterpret_cast<const float2*>(oi) + k * 32 + lane);
                            x[j][k][0] = v.x, x[j][k][1] = v.y;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
                if (j0 + j < n)
#pragma unroll
                    for (int k = 0; k < W; ++k)
#pragma unroll
                        for (int e = 0; e < V; ++e) s.o[k][e] = fmaf(x[j][k][e], g[j], s.o[k][e]);
        }
    }
    return s;
}

// The finished row out, by one warp.
template <typename O, int D>
__device__ __forceinline__ void write_row(const Sum<D>& s, const Out& fin, float* lse2, long long row) {
    constexpr int V = Lane<D>::V, W = Lane<D>::W;
    const int lane = threadIdx.x & 31;
    const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;   // l == 0: no key seen (a NaN or infinite l stays one)
#pragma unroll
    for (int k = 0; k < W; ++k)
        if (V * (k * 32 + lane) < D) {
            const long long at = row * (D / V) + k * 32 + lane;
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = s.o[k][e] * inv;
            if constexpr (sizeof(O) == 4) {
                if constexpr (V == 4) reinterpret_cast<float4*>(fin.out)[at] = make_float4(y[0], y[1], y[2], y[3]);
                else reinterpret_cast<float2*>(fin.out)[at] = make_float2(y[0], y[1]);
            } else {
                if constexpr (V == 4)
                    reinterpret_cast<uint2*>(fin.out)[at] = make_uint2(mq_pack2<O>(y[0], y[1]), mq_pack2<O>(y[2], y[3]));
                else
                    reinterpret_cast<uint32_t*>(fin.out)[at] = mq_pack2<O>(y[0], y[1]);
            }
        }
    if (lane == 0) {
        if (fin.lse) fin.lse[row] = s.l == 0.0f ? -INFINITY : s.m * kLn2 + logf(s.l);
        if (lse2) lse2[row] = s.l == 0.0f ? -INFINITY : s.m + log2f(s.l);
    }
}

}  // namespace attn
