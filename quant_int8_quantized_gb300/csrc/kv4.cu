// Rows of a 4-bit cache (kv4.cuh): head norms and rotation of a layer's projections with the keys and values rounded
// to 4 bits in the same pass, and rows read back in 16 bits.
//
// Writing. As in qk_rope.cu a thread holds four pairs of a head, a head is D / 8 lanes of an aligned group of 8, 16 or 32, and
// cos and sin come once per token out of shared memory. Keys and values then change hands through shared memory so that a
// lane has the eight dims of one word of the page, four lanes a block of 32 dims: two shuffles find its largest
// magnitude a, the scale is the least one with 7 d >= a, the numbers are rint(y / d).
// That rounding is decided for y as the formula has it, not as 32 bits do. In units of u = 2^-24: a cosine or sine is off by the angle's
// rounding (1.6), the function's (1) and rot_scale's product (0.5); a pair's product with them by sqrt(2) 3.1 and its own two
// roundings, 6.4 of the pair's length, which is sqrt(2) times the head's largest magnitude at most: 9.1 u of it. A norm's factor
// is off by half of the sum's 9 (two roundings, two levels of additions, up to five of shuffles) and by six more roundings' 5: 9.5
// of the pair's length besides, 22.5 u in all. Where a border lies within that of y or of the block's largest, the row
// goes to a list, and the block computes those rows again in 64 bits at its end, a thread a pair (in the warps that met them, all
// heads of a warp at once, they held up 16384 tokens for 60 us of 164). So the bytes do not depend on how 32-bit sums are ordered.
// Values are the inputs themselves: 32 bits tell on which side of a border they lie.
// Bound: HBM, 4 bytes read an element, 2 written (q) or 17/32. Measured: 16384 tokens of 40 + 8 heads of 128, 115 us, 5.4 TB/s; 3314 of
// 28 + 4, 27 us; one token, 3 us.

#include <cmath>

#include "kv4.cuh"

namespace kv4 {
namespace {

constexpr int kThreads = 128, kList = 64;
constexpr float kOffNorm = 24.5f * 5.9604644775390625e-08f, kOffTurn = 9.6f * 5.9604644775390625e-08f;   // see above

struct FillArgs {
    const float* x[3];          // q, k, v (NULL: left out)
    long long stride[3];
    const float* w[2];
    const float* inv_freq;
    const uint8_t* axis;
    const int32_t* pos;
    const int32_t* seq;
    const int32_t* row;
    void* q_out;
    Cache c;
    int M, D, n_pairs, n_axes;
    int h0, h1, h2;             // rows of a token: [0, h0) q, [h0, h1) k, [h1, h2) v
    float eps, rot_scale;
};

// cos and sin of pos * freq, times `by`; the turn is taken out in 64 bits (qk_rope.cu).
__device__ __forceinline__ float2 turn(int pos, float freq, float by) {
    const double t = (double)pos * (double)freq * 0.31830988618379067154;   // in half turns
    float s, c;
    sincospif((float)(t - 2.0 * rint(0.5 * t)), &s, &c);
    return make_float2(c * by, s * by);
}

// sin and cos of pi t for |t| <= 1 by their power series, to 2^-51.
__device__ __forceinline__ void sincos_pi(double t, double& s, double& c) {
    const double k = rint(2.0 * t), x = fma(-0.5, k, t) * 3.14159265358979323846, z = x * x;   // |x| <= pi / 4
    double u = 1.0 / 1307674368000.0, v = 1.0 / 20922789888000.0;
    u = fma(u, -z, 1.0 / 6227020800.0), v = fma(v, -z, 1.0 / 87178291200.0);
    u = fma(u, -z, 1.0 / 39916800.0), v = fma(v, -z, 1.0 / 479001600.0);
    u = fma(u, -z, 1.0 / 362880.0), v = fma(v, -z, 1.0 / 3628800.0);
    u = fma(u, -z, 1.0 / 5040.0), v = fma(v, -z, 1.0 / 40320.0);
    u = fma(u, -z, 1.0 / 120.0), v = fma(v, -z, 1.0 / 720.0);
    u = fma(u, -z, 1.0 / 6.0), v = fma(v, -z, 1.0 / 24.0);
    u = fma(u, -z, 1.0), v = fma(v, -z, 0.5);
    u *= x, v = fma(v, -z, 1.0);
    const int q = (int)k & 3;
    s = q & 1 ? v : u;
    c = q & 1 ? u : v;
    if (q >= 2) s = -s;
    if (q == 1 || q == 2) c = -c;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if one of them is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// The least code whose 7 d is `a` or more.
__device__ __forceinline__ int code_of(float a) {
    if (!(a < 3360.0f)) return kMostCode;
    const float t = a * (1.0f / 7.0f);
    int c = t < 6.103515625e-05f ? (int)ceilf(t * 131072.0f) : (int)((__float_as_uint(t) + 0xfffffu) >> 20) - 896;
    if (c > 0 && 7.0f * scale_of(c - 1) >= a) --c;
    else if (7.0f * scale_of(c) < a) ++c;
    return c;
}
__device__ __forceinline__ int code_of(double a) {
    if (!(a < 3360.0)) return kMostCode;
    int c = code_of((float)a);
    if (c > 0 && 7.0 * (double)scale_of(c - 1) >= a) --c;
    else if (7.0 * (double)scale_of(c) < a && c < kMostCode) ++c;
    return c;
}

// rint(y / d) within -7 .. 7, ties to even, exactly (binary32: y - n d has few bits, and is no longer than y).
template <typename F>
__device__ __forceinline__ float nearest(F y, float d, float inv) {
    float k = fminf(fmaxf(rintf((float)y * inv), -8.0f), 8.0f);
    const F rest = fma(-(F)k, (F)d, y), over = 2 * fabs(rest);
    if (over > d || (over == d && ((int)k & 1))) k += rest < 0 ? -1.0f : 1.0f;
    return fminf(fmaxf(k, -7.0f), 7.0f);
}

// LG lanes a head. VEC: pairs come in fours (n_pairs % 4 == 0); otherwise each of a thread's
// four pairs or eight plain numbers is placed by itself.
template <typename T, int LG, bool INTER, bool VEC>
__global__ void __launch_bounds__(kThreads) fill_kernel(const FillArgs a) {
    extern __shared__ float2 s_turn[];                 // [4][n_pairs / 4]: pair 4 i + k at [k][i], a thread's four in four rows of banks
    __shared__ float s_row[kThreads / LG][LG * 8 + 16]; // a head's row on its way from pairs to words (heads in other banks)
    __shared__ int s_list[kList], s_n;                 // rows that want 64 bits
    mq_grid_release();
    mq_grid_wait();
    const int m = blockIdx.x;                          // the token
    const int lane = threadIdx.x % LG, group = threadIdx.x / LG;
    const int D = a.D, n = a.n_pairs, quarter = (n + 3) / 4;
    const int rows = a.h2;
    const int r_first = blockIdx.y * (kThreads / LG) + group, r_step = gridDim.y * (kThreads / LG);

    struct Row {
        int what, h, np;
        float v[8];
    };
    // Where element i of this thread lies (VEC: 0 .. 3 from low(np) on, 4 .. 7 from high(np); see qk_rope.cu).
    auto place = [&](int np, int i) {
        const int p = lane * 4 + i / 2;
        if (p >= np) return lane * 8 + i;
        return INTER ? 2 * p + (i & 1) : p + (i & 1) * np;
    };
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
            const float4 u0 = __ldca(reinterpret_cast<const float4*>(p + low(x.np)));
            const float4 u1 = __ldca(reinterpret_cast<const float4*>(p + high(x.np)));
            x.v[0] = u0.x, x.v[1] = u0.y, x.v[2] = u0.z, x.v[3] = u0.w;
            x.v[4] = u1.x, x.v[5] = u1.y, x.v[6] = u1.z, x.v[7] = u1.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.v[i] = __ldca(p + place(x.np, i));
        }
    };
    Row now;
    fetch(r_first, now);             // on its way while the turns are computed

    auto angle = [&](int p, float& freq) {
        const int ax = a.axis ? min((int)a.axis[p], a.n_axes - 1) : 0;
        freq = a.inv_freq[p];
        return a.pos[(long long)ax * a.M + m];
    };
    for (int p = threadIdx.x; p < n; p += kThreads) {
        float freq;
        const int pos = angle(p, freq);
        s_turn[(p & 3) * quarter + (p >> 2)] = turn(pos, freq, a.rot_scale);
    }
    int page = -1, row = -1;
    if (a.h2 > a.h0) {
        const int seq = a.seq ? __ldca(a.seq + m) : 0;
        row = __ldca(a.row + m);
        if ((unsigned)seq < (unsigned)a.c.n && row >= 0 && row >> a.c.shift < a.c.width) page = a.c.page(seq, row);
    }
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    for (int r = r_first; r - group < rows; r += r_step) {
        Row next;
        fetch(r + r_step, next);     // (past the last row: nothing)
        const bool live = r < rows && lane * 8 < D;
        const int what = r < rows ? now.what : 0, h = now.h, np = now.np;
        const int lo = low(np), hi = high(np);
        const bool rot = lane * 4 < np;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = now.v[i];
        now = next;
        const float* w = what == 2 ? nullptr : a.w[what];
        float ss = 0.0f, mean = 1.0f;
        if (a.w[0] || a.w[1]) {
            float pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = fmaf(v[2 * i], v[2 * i], v[2 * i + 1] * v[2 * i + 1]);
            ss = (pr[0] + pr[1]) + (pr[2] + pr[3]);
#pragma unroll
            for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        }
        if (w && live) mean = ss / (float)D + a.eps;
        const bool lost = !(mean > 1e-30f && mean < 3e38f);                 // a mean square that 32 bits do not hold
        if (__any_sync(0xffffffffu, lost)) {                                // taken by a power of two that brings them next to 1
            float top = sqrtf(a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
            for (int o = LG / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float by = lost ? __uint_as_float(max(1, 253 - (int)(__float_as_uint(top) >> 23)) << 23) : 1.0f;
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] *= by;
                ss = fmaf(v[i], v[i], ss);
            }
#pragma unroll
            for (int o = LG / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lost) mean = ss / (float)D + a.eps * by * by;
        }
        if (w && live) {
            const float sc = 1.0f / sqrtf(mean);
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
        auto rotate = [](float& p, float& q, float2 t) {
            const float u = p * t.x - q * t.y;
            q = p * t.y + q * t.x;
            p = u;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane * 4 + i < np) {
                if constexpr (VEC && !INTER) rotate(v[i], v[4 + i], s_turn[i * quarter + lane]);
                else rotate(v[2 * i], v[2 * i + 1], s_turn[i * quarter + lane]);
            }
        if (live && what == 0) {
            T* y = reinterpret_cast<T*>(a.q_out) + ((long long)m * a.h0 + h) * D;
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
        if (__all_sync(0xffffffffu, what == 0) || page < 0) continue;      // (the page is the token's: the same for all)

        // ------------------------------------------------------------ keys and values to words and scales
        if constexpr (!(INTER && VEC)) {               // (neighbours and values lie as they will be packed)
            float* row32 = s_row[group];
            if (live && what == 1) {
                if constexpr (VEC) {
                    *reinterpret_cast<float4*>(row32 + lo) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4*>(row32 + hi) = make_float4(v[4], v[5], v[6], v[7]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) row32[place(np, i)] = v[i];
                }
            }
            __syncwarp();
            if (live && what == 1) {
                const float4 u0 = *reinterpret_cast<const float4*>(row32 + lane * 8);
                const float4 u1 = *reinterpret_cast<const float4*>(row32 + lane * 8 + 4);
                v[0] = u0.x, v[1] = u0.y, v[2] = u0.z, v[3] = u0.w;
                v[4] = u1.x, v[5] = u1.y, v[6] = u1.z, v[7] = u1.w;
            }
            __syncwarp();
        }
        float most;                                                         // of the block of 32 dims; NaN where one of them is
        auto find_most = [&] {
            most = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max_nan(most, fabsf(v[i]));
            most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
        };
        find_most();
        float all = most;
#pragma unroll
        for (int o = 4; o < LG; o <<= 1) all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, o));
        if (__any_sync(0xffffffffu, !(most <= 3360.0f))) {
            // past 7 d of the largest scale: as 7 d (an infinity has no rest); no number: 0. (A head that this changes, and that is not to be
            // rounded as it is, goes to the list by `all`.)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -3360.0f), 3360.0f) : 0.0f;
            find_most();
        }
        const bool exact = what != 1 || (!w && n == 0);                     // v is what there is to round
        const float off = exact ? 0.0f : all * (w ? kOffNorm : kOffTurn);
        int code = code_of(most);
        const float d = scale_of(code);
        const float inv = d > 0.0f ? __frcp_rn(d) : 0.0f;
        // rint(v / d) + 8 in the last bits of v / d + 1.5 2^23 + 8, ties to even. The quotient is the correctly rounded one (a step
        // from the product with the rounded reciprocal by the exact rest), and that is a tie only where v / d is: d has four bits, so
        // another v / d lies more than half a unit away.
        float quot[8], far = 0.0f;
        uint32_t num[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = v[i] * inv;
            quot[i] = fmaf(fmaf(-q, d, v[i]), inv, q);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float m = quot[i] + 12582920.0f;
            far = fmaxf(far, fabsf(quot[i] - (m - 12582920.0f)));
            num[i] = __float_as_uint(m);
        }
        // (a rotated or normed v is off by `off`: what lies next to a border goes to the list, and what 32 bits have no room for)
        const bool near = !exact && (lost || !(far < 0.5f - 1e-6f - off * inv) || !(all < 3360.0f - off) ||
                          (most > 0.0f && (7.0f * d < most + off || (code > 0 && 7.0f * scale_of(code - 1) >= most - off))));
        const uint32_t again = __ballot_sync(0xffffffffu, near && live) >> (threadIdx.x & 31 & ~(LG - 1)) &
                               (LG == 32 ? ~0u : (1u << (LG & 31)) - 1);
        if (again) {                                   // (all of a head's lanes)
            if (lane == 0) {
                const int k = atomicAdd(&s_n, 1);
                if (k < kList) s_list[k] = r;
            }
            continue;
        }
        if (!live || what == 0) continue;
        // four numbers, and what lies above their four bits (a constant, or nothing), as one sum
        auto four = [&](int i0, int step) { return num[i0] + 16u * num[i0 + step] + 256u * num[i0 + 2 * step] + 4096u * num[i0 + 3 * step]; };
        const int nb = D / 32, b = lane / 4, t = lane % 4, in = row & (kBlockRows - 1);
        uint8_t* block = a.c.block(page, h, row, block_bytes(D));
        if (what == 1) {
            reinterpret_cast<uint32_t*>(block)[(4 * in + t) * nb + b] = __byte_perm(four(0, 2), four(1, 2), 0x5410);
        } else {
            uint16_t* half = reinterpret_cast<uint16_t*>(block + value_at(D));
            const int p = in >> 3, tt = (in >> 1) & 3, c = in & 1;
#pragma unroll
            for (int k = 0; k < 2; ++k) half[2 * (((8 * p + 2 * t + k) * 4 + tt) * nb + b) + c] = (uint16_t)four(4 * k, 1);
        }
        if (t == 0) block[what == 1 ? key_scale_at(D) + in * nb + b : value_scale_at(D) + (in >> 1) * 2 * nb + 2 * b + (in & 1)] = (uint8_t)code;
    }

    // ---------------------------------------------------------------- rows next to a border, in 64 bits: a thread a pair
    __syncthreads();
    if (s_n == 0) return;
    __shared__ double s_y[256], s_part[kThreads / 32];
    const float* const w = a.w[1];
    const int nb = D / 32, in = row & (kBlockRows - 1), tid = threadIdx.x, wl = tid & 31, wid = tid >> 5;
    const bool every = s_n > kList;                    // more than the list holds: all keys of this block
    const int k_first = every ? (int)blockIdx.y * (kThreads / LG) : 0, k_end = every ? a.h1 : s_n;
    for (int k = k_first; k < k_end; ++k) {
        int r = k;
        if (!every) r = s_list[k];
        else if (k < a.h0 || (k / (kThreads / LG)) % (int)gridDim.y != (int)blockIdx.y) continue;
        const int h = r - a.h0;
        const float* x = a.x[1] + (long long)m * a.stride[1] + (long long)h * D;
        double by = 1.0;
        if (w) {
            double sum = 0.0;
            for (int i = tid; i < D; i += kThreads) sum = fma((double)x[i], (double)x[i], sum);
#pragma unroll 1
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (wl == 0) s_part[wid] = sum;
            __syncthreads();
            by = 1.0 / sqrt((s_part[0] + s_part[1] + s_part[2] + s_part[3]) / D + (double)a.eps);
        }
        auto normed = [&](int i) { return w ? (double)x[i] * by * (double)w[i] : (double)x[i]; };
        for (int p = tid; p < n; p += kThreads) {
            float freq;
            const int pos = angle(p, freq);
            const double t = (double)pos * (double)freq * 0.31830988618379067154;
            double sn, cs;
            sincos_pi(t - 2.0 * rint(0.5 * t), sn, cs);
            cs *= (double)a.rot_scale;
            sn *= (double)a.rot_scale;
            const int i0 = INTER ? 2 * p : p, i1 = INTER ? 2 * p + 1 : p + n;
            const double u = normed(i0), q = normed(i1);
            s_y[i0] = u * cs - q * sn;
            s_y[i1] = u * sn + q * cs;
        }
        for (int i = 2 * n + tid; i < D; i += kThreads) s_y[i] = normed(i);
        __syncthreads();
        uint8_t* block = a.c.block(page, h, row, block_bytes(D));
        for (int b = wid; b < nb; b += kThreads / 32) {
            double y = s_y[32 * b + wl];
            if (y != y) y = 0.0;
            long long top = __double_as_longlong(y) & 0x7fffffffffffffffLL;   // (numbers without their sign are in the order of their bits)
#pragma unroll 1
            for (int o = 16; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int code = code_of(__longlong_as_double(top));
            const float d = scale_of(code);
            uint32_t word = (8u + (int)nearest(y, d, d > 0.0f ? 1.0f / d : 0.0f)) << (16 * (wl & 1) + 4 * ((wl & 7) >> 1));
#pragma unroll
            for (int o = 4; o >= 1; o >>= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
            if ((wl & 7) == 0) reinterpret_cast<uint32_t*>(block)[(4 * in + (wl >> 3)) * nb + b] = word;
            if (wl == 0) block[key_scale_at(D) + in * nb + b] = (uint8_t)code;
        }
        __syncthreads();
    }
}

template <typename T, int LG>
int launch_fill(const FillArgs& a, bool inter, dim3 grid, size_t smem, cudaStream_t stream) {
    const bool vec = a.n_pairs % 4 == 0;
    auto kern = vec ? (inter ? fill_kernel<T, LG, true, true> : fill_kernel<T, LG, false, true>)
                    : (inter ? fill_kernel<T, LG, true, false> : fill_kernel<T, LG, false, false>);
    return mq::launch_pdl(kern, grid, dim3(kThreads), smem, stream, a);
}

// ---------------------------------------------------------------------------------------------- rows in 16 bits

struct ReadArgs {
    Cache c;
    const int32_t* len;
    void* k;
    void* v;
    long long seq_stride, row_stride, head_stride;
    int cap, chunks;        // rows at most of a sequence; chunks of kChunk blocks of them
    long long units;        // sequences x heads x chunks
};
constexpr int kChunk = 2, kReadWarps = 4;

// A warp takes 32 rows of a head, 16 at a time: the words that a lane loads are those that the products' operands are
// made of, so eight lanes' stores fill a row's 64 bytes.
template <typename T, typename V, int D>
__global__ void __launch_bounds__(32 * kReadWarps) read_kernel(const ReadArgs a) {
    constexpr int nb = D / 32;
    mq_grid_release();
    mq_grid_wait();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long warps = (long long)gridDim.x * kReadWarps;
    for (long long unit = (long long)blockIdx.x * kReadWarps + (threadIdx.x >> 5); unit < a.units; unit += warps) {
        const long long sh = unit / a.chunks;
        const int chunk = (int)(unit - sh * a.chunks), seq = (int)(sh / a.c.heads), h = (int)(sh - (long long)seq * a.c.heads);
        const int len = min(max(__ldca(a.len + seq), 0), a.cap);
        T* k_to = reinterpret_cast<T*>(a.k) + seq * a.seq_stride + h * a.head_stride;
        V* v_to = reinterpret_cast<V*>(a.v) + seq * a.seq_stride + h * a.head_stride;
#pragma unroll 1
        for (int i = 0; i < kChunk; ++i) {
            const int row0 = (chunk * kChunk + i) * kBlockRows;
            if (row0 >= len) break;
            const int page = a.c.page(seq, row0);
            uint32_t kw[2][nb], vw[2][nb], ks[2][(nb + 3) / 4], vs[2][nb / 2 + nb % 2];
            if (page >= 0) {
                const uint8_t* block = a.c.block(page, h, row0, block_bytes(D));
                auto from = [](const uint8_t* p) {
                    return [p](auto type, int i) { return __ldca(reinterpret_cast<const decltype(type)*>(p) + i); };
                };
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    words<nb>(from(block + (p * 32 + lane) * nb * 4), kw[p]);
                    words<nb>(from(block + value_at(D) + (p * 32 + lane) * nb * 4), vw[p]);
                    bytes<nb>(from(block + key_scale_at(D) + (g + 8 * p) * nb), ks[p]);
                    bytes<2 * nb>(from(block + value_scale_at(D) + (4 * p + t) * 2 * nb), vs[p]);
                }
            } else {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int b = 0; b < nb; ++b) kw[p][b] = vw[p][b] = 0;
#pragma unroll
                    for (int b = 0; b < (nb + 3) / 4; ++b) ks[p][b] = 0;
#pragma unroll
                    for (int b = 0; b < nb / 2 + nb % 2; ++b) vs[p][b] = 0;
                }
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int kr = row0 + g + 8 * p, vr = row0 + 8 * p + 2 * t;
#pragma unroll
                for (int b = 0; b < nb; ++b) {
                    uint32_t x[4];
                    numbers(kw[p][b], Scale<T>::of(twice(ks[p], b)), x);
                    if (kr < len)
                        *reinterpret_cast<uint4*>(k_to + kr * a.row_stride + 32 * b + 8 * t) = make_uint4(x[0], x[1], x[2], x[3]);
                    numbers(vw[p][b], Scale<V>::of(both(vs[p], b)), x);
                    V* to = v_to + vr * a.row_stride + 32 * b + 4 * g;
                    if (vr < len)
                        *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
                    if (vr + 1 < len)
                        *reinterpret_cast<uint2*>(to + a.row_stride) =
                            make_uint2(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
                }
            }
        }
    }
}

}  // namespace

int launch_read(const mq_kv4* src, const int32_t* len, const mq_kv* dst, int v_type, cudaStream_t stream) {
    ReadArgs a;
    a.c = cache_of(src);
    a.len = len;
    a.k = dst->k;
    a.v = dst->v;
    a.seq_stride = dst->seq_stride;
    a.row_stride = dst->row_stride;
    a.head_stride = dst->head_stride;
    const int held = src->width * src->page_rows;
    a.cap = dst->cap < held ? dst->cap : held;
    a.chunks = (a.cap + kChunk * kBlockRows - 1) / (kChunk * kBlockRows);
    a.units = (long long)src->n * src->heads * a.chunks;
    if (a.units == 0) return MQ_OK;
    const long long blocks = (a.units + kReadWarps - 1) / kReadWarps, most = 16LL * mq::num_sms();
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    auto go = [&](auto t, auto v) {
        using T = decltype(t);
        using V = decltype(v);
        auto kern = src->dim == 64 ? read_kernel<T, V, 64> : src->dim == 96 ? read_kernel<T, V, 96>
                    : src->dim == 128 ? read_kernel<T, V, 128> : read_kernel<T, V, 256>;
        return mq::launch_pdl(kern, grid, dim3(32 * kReadWarps), 0, stream, a);
    };
    if (dst->type == MQ_F16) return go(__half(), __half());
    return v_type == MQ_F16 ? go(__nv_bfloat16(), __half()) : go(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace kv4

extern "C" size_t mq_kv4_page_bytes(int page_rows, int heads, int dim) {
    if (!kv4::valid_rows(page_rows) || !kv4::valid_dim(dim) || heads < 1) return 0;
    return (size_t)(page_rows / 16) * heads * kv4::block_bytes(dim);
}

extern "C" int mq_qk_norm_rope_kv4(const mq_qkv* x, int type, float rot_scale, void* q_out, const mq_kv4* cache,
                                   const int32_t* seq, const int32_t* row, cudaStream_t stream) {
    using namespace kv4;
    if (!x) return MQ_ERR_NULL;
    int rc = check(cache, false);
    if (rc != MQ_OK) return rc;
    if (type != MQ_F16 && type != MQ_BF16) return MQ_ERR_TYPE;
    const int D = cache->dim, Hkv = cache->heads;
    if (x->M < 0 || x->Hq < 0 || x->n_pairs < 0 || 2 * x->n_pairs > D || !std::isfinite(rot_scale)) return MQ_ERR_SHAPE;
    if (x->n_pairs > 0 && (x->n_axes < 1 || x->n_axes > 8)) return MQ_ERR_SHAPE;
    if (x->M == 0) return MQ_OK;
    const bool cached = x->k || x->v;
    const float* src[3] = {x->q, x->k, x->v};
    const long long st[3] = {x->q_stride, x->k_stride, x->v_stride};
    const int heads[3] = {x->q ? x->Hq : 0, x->k ? Hkv : 0, x->v ? Hkv : 0};
    if ((long long)heads[0] + heads[1] + heads[2] > 0x7fffff) return MQ_ERR_SHAPE;
    for (int i = 0; i < 3; ++i)
        if (src[i]) {
            if (st[i] < (long long)heads[i] * D || st[i] % 4 != 0 || (x->M > 1 && st[i] > mq::kTokenStrideMost)) return MQ_ERR_SHAPE;
            if (!mq::aligned16(src[i])) return MQ_ERR_ALIGN;
        }
    if (x->n_pairs > 0 && (!x->inv_freq || !x->pos)) return MQ_ERR_NULL;
    if ((heads[0] > 0 && !q_out) || (cached && !row)) return MQ_ERR_NULL;
    if (cached) {
        rc = check(cache, true);
        if (rc != MQ_OK) return rc;
    }
    if (!mq::aligned16(q_out) || !mq::aligned16(x->wq) || !mq::aligned16(x->wk) || !mq::aligned16(x->inv_freq) ||
        !mq::aligned16(x->axis) || !mq::aligned16(x->pos) || !mq::aligned16(seq) || !mq::aligned16(row))
        return MQ_ERR_ALIGN;
    const long long q_bytes = 2LL * x->M * heads[0] * D;
    for (int i = 0; i < 3; ++i)   // a block's output rows would lie over what others have yet to read
        if (mq::rows_meet(src[i], x->M, 4 * st[i], 4LL * heads[i] * D, q_out, q_bytes) ||
            (cached && mq::rows_meet(src[i], x->M, 4 * st[i], 4LL * heads[i] * D, cache->pages, pool_span(cache))))
            return MQ_ERR_SHAPE;
    if (cached && meets_pages(cache, q_out, q_bytes)) return MQ_ERR_SHAPE;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    FillArgs a;
    for (int i = 0; i < 3; ++i) {
        a.x[i] = src[i];
        a.stride[i] = st[i];
    }
    a.w[0] = x->wq;
    a.w[1] = x->wk;
    a.inv_freq = x->inv_freq;
    a.axis = x->axis;
    a.pos = x->pos;
    a.seq = seq;
    a.row = row;
    a.q_out = q_out;
    a.c = cache_of(cache);
    a.M = x->M;
    a.D = D;
    a.n_pairs = x->n_pairs;
    a.n_axes = x->n_axes;
    a.h0 = heads[0];
    a.h1 = a.h0 + heads[1];
    a.h2 = a.h1 + heads[2];
    a.eps = x->eps;
    a.rot_scale = rot_scale;
    if (a.h2 == 0) return MQ_OK;
    const int lg = D <= 64 ? 8 : D <= 128 ? 16 : 32, per = kThreads / lg;
    const int passes = (a.h2 + per - 1) / per;
    const dim3 grid(x->M, x->M >= 2 * mq::num_sms() ? 1 : passes < 65535 ? passes : 65535);
    const size_t smem = (size_t)((a.n_pairs + 3) / 4) * 4 * sizeof(float2);
    const bool inter = x->interleaved != 0;
    auto go = [&](auto t) {
        using T = decltype(t);
        return lg == 8 ? launch_fill<T, 8>(a, inter, grid, smem, stream)
               : lg == 16 ? launch_fill<T, 16>(a, inter, grid, smem, stream)
                          : launch_fill<T, 32>(a, inter, grid, smem, stream);
    };
    return type == MQ_F16 ? go(__half()) : go(__nv_bfloat16());
}

extern "C" int mq_kv4_read(const mq_kv4* src, const int32_t* len, const mq_kv* dst, cudaStream_t stream) {
    using namespace kv4;
    int rc = check(src, true);
    if (rc == MQ_OK) rc = mq::check_kv(dst, true);
    if (rc != MQ_OK) return rc;
    if (dst->n != src->n || dst->heads != src->heads || dst->dim != src->dim) return MQ_ERR_SHAPE;
    if (src->n == 0 || src->width == 0 || dst->cap == 0) return MQ_OK;
    if (!len) return MQ_ERR_NULL;
    if (!mq::aligned16(len)) return MQ_ERR_ALIGN;
    const long long span = 2 * mq::kv_span(dst);
    if (meets_pages(src, dst->k, span) || meets_pages(src, dst->v, span)) return MQ_ERR_SHAPE;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    return launch_read(src, len, dst, dst->type, stream);
}
