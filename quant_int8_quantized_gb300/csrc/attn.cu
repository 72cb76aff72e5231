// Attention over a shared prefix and each sequence's own cache: arguments, workspace, and the kernels
// that join the pieces (attn.cuh) into outputs and add up attention weights.

#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "attn_few.cuh"
#include "attn_many.cuh"

namespace attn {

bool allow_smem(const void* kern, int bytes) {
    static std::mutex mu;
    static std::map<std::pair<const void*, int>, bool> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lk(mu);
    const auto key = std::make_pair(kern, dev);
    const auto it = done.find(key);
    if (it != done.end()) return it->second;
    const bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    if (!ok) cudaGetLastError();
    done.emplace(key, ok);
    return ok;
}

namespace {

constexpr int kMaxPerSm = 4;   // blocks of a piece kernel per SM, at most
constexpr float kLn2 = 0.6931471805599453f;

// One part of the keys, as the joining kernel sees it.
struct Part {
    Pieces p;
    int rows;      // per segment; 0: no such part
};

struct JoinArgs {
    Part prefix, own;
    const int32_t* len;
    int B, T, Hq, Hkv, group, own_cap, seg0;   // seg0: the own part's first segment
    void* out;
    float* lse;    // natural, or nullptr
    float* lse2;   // base 2, or nullptr
};

__device__ __forceinline__ float exp2_acc(float x) { return exp2f(x); }

// A warp per query row: the pieces' common maximum, then their outputs weighted and added in key order.
template <typename O, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const JoinArgs a) {
    constexpr int N = (D + 63) / 64;
    mq_grid_release();
    mq_grid_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);   // (b T + t) Hq + h
    if (row >= (long long)a.B * a.T * a.Hq) return;
    const int h = (int)(row % a.Hq);
    const long long bt = row / a.Hq;
    const int t = (int)(bt % a.T), b = (int)(bt / a.T);
    const int hk = h / a.group;
    const int r_own = t * a.group + h - hk * a.group;
    float m = -INFINITY;
    // the row's pieces: prefix segment, own segment; [first place, count, row in the segment]
    long long place[2] = {0, 0};
    int count[2] = {0, 0}, in[2] = {0, 0};
    if (a.prefix.rows > 0) {
        const int r = b * a.T * a.group + r_own;
        const int seg = r / a.prefix.rows * a.Hkv + hk;
        in[0] = r % a.prefix.rows;
        const int2 f = __ldca(a.prefix.p.info + seg);
        place[0] = (long long)f.x + seg;
        count[0] = f.y - f.x + 1;
    }
    if (a.own.rows > 0) {
        const int rt = r_own / a.own.rows, tg = a.T * a.group;
        const int last = min((rt + 1) * a.own.rows, tg) - 1;
        if (min(max(__ldca(a.len + b), 0), a.own_cap) - a.T + 1 + last / a.group > 0) {
            const int seg = a.seg0 + (b * ceil_div(tg, a.own.rows) + rt) * a.Hkv + hk;
            in[1] = r_own % a.own.rows;
            const int2 f = __ldca(a.own.p.info + seg);
            place[1] = (long long)f.x + seg;
            count[1] = f.y - f.x + 1;
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const Part& p = w ? a.own : a.prefix;
        for (int i = lane; i < count[w]; i += 32) m = fmaxf(m, __ldca(&p.p.ml[(place[w] + i) * p.rows + in[w]].x));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float safe = m == -INFINITY ? 0.0f : m;
    float l = 0.0f;
    float2 acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const Part& p = w ? a.own : a.prefix;
#pragma unroll 4
        for (int i = 0; i < count[w]; ++i) {
            const long long at = (place[w] + i) * p.rows + in[w];
            const float2 ml = __ldca(p.p.ml + at);
            const float f = exp2_acc(ml.x - safe);
            l += ml.y * f;
            const float2* o = reinterpret_cast<const float2*>(p.p.o + at * D);
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k * 32 + lane < D / 2) {
                    const float2 x = __ldca(o + k * 32 + lane);
                    acc[k].x = fmaf(x.x, f, acc[k].x);
                    acc[k].y = fmaf(x.y, f, acc[k].y);
                }
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // l == 0: no key seen (a NaN or infinite l stays one)
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k * 32 + lane < D / 2) {
            const float x = acc[k].x * inv, y = acc[k].y * inv;
            if constexpr (sizeof(O) == 4)
                reinterpret_cast<float2*>(a.out)[row * (D / 2) + k * 32 + lane] = make_float2(x, y);
            else
                reinterpret_cast<uint32_t*>(a.out)[row * (D / 2) + k * 32 + lane] = mq_pack2<O>(x, y);
        }
    if (lane == 0) {
        const float l2 = l == 0.0f ? -INFINITY : safe + log2f(l);
        if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : safe * kLn2 + logf(l);
        if (a.lse2) a.lse2[row] = l2;
    }
}

// score_out = score + sum over the rows of 2^(raw - lse2), one thread a key.
__global__ void __launch_bounds__(256) attn_score_kernel(const float* raw, const float* lse2, const int32_t* len,
                                                         const float* score, float* score_out, int T, int Hq, int Hkv,
                                                         int cap) {
    mq_grid_release();
    mq_grid_wait();
    const int b = blockIdx.y / Hkv, hk = blockIdx.y - b * Hkv;
    const int n = min(max(__ldca(len + b), 0), cap);
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= n) return;
    const int group = Hq / Hkv, tg = T * group;
    const float* s = raw + (long long)blockIdx.y * tg * cap + j;
    float w = 0.0f;
#pragma unroll 4
    for (int r = 0; r < tg; ++r) {
        const int t = r / group;
        if (j >= n - T + 1 + t) continue;   // not seen; the first kernel left nothing there
        const float l2 = __ldca(lse2 + ((long long)b * T + t) * Hq + hk * group + r - t * group);
        const float x = __ldca(s + (long long)r * cap);
        w += x == -INFINITY ? 0.0f : exp2f(x - l2);
    }
    const long long at = (long long)blockIdx.y * cap + j;
    score_out[at] = __ldca(score + at) + w;
}

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

// Query rows per key head from which the tensor-core kernel takes a part.
constexpr int kManyFrom = 33;

// How a call is cut: the part of each kernel, and where the workspace holds what.
struct Cut {
    Plan few, many;
    bool prefix_many, own_many;
    size_t few_o, few_ml, few_info, many_o, many_ml, many_info, lse2, raw, bytes;
};

Cut cut_of(int B, int T, int Hq, int Hkv, int D, int prefix_keys, int own_cap, bool scores) {
    Cut c;
    const int group = Hq / Hkv;
    c.prefix_many = prefix_keys > 0 && many_takes(D) && (long long)B * T * group >= kManyFrom;
    // the weights' raw products come from the kernel for few rows
    c.own_many = own_cap > 0 && many_takes(D) && !scores && (long long)T * group >= kManyFrom;
    size_t at = 0;
    auto plan = [&](bool many, size_t* o, size_t* ml, size_t* info) {
        Plan p;
        p.B = B;
        p.T = T;
        p.Hq = Hq;
        p.Hkv = Hkv;
        p.group = group;
        p.prefix_rows = B * T * group;
        p.prefix_keys = c.prefix_many == many ? prefix_keys : 0;
        p.own_cap = c.own_many == many ? own_cap : 0;
        p.rows = many ? kManyRows : kFewRows;
        p.keys = many ? kManyKeys : few_tile_keys(D);
        const long long segs = all_segs(p);
        const long long most = (long long)prefix_segs(p) * ceil_div(p.prefix_keys, p.keys) +
                               (segs - prefix_segs(p)) * ceil_div(p.own_cap, p.keys);
        const long long held = (long long)mq::num_sms() * (many ? 1 : kMaxPerSm);
        p.G = (int)(most < held ? most : held);
        const size_t places = segs > 0 ? (size_t)p.G + (size_t)segs : 0;
        *o = at;
        at += up16(places * p.rows * D * sizeof(float));
        *ml = at;
        at += up16(places * p.rows * sizeof(float2));
        *info = at;
        at += up16((size_t)segs * sizeof(int2));
        return p;
    };
    c.few = plan(false, &c.few_o, &c.few_ml, &c.few_info);
    c.many = plan(true, &c.many_o, &c.many_ml, &c.many_info);
    const size_t rows = (size_t)B * T * Hq;
    c.lse2 = at;
    at += scores ? up16(rows * sizeof(float)) : 0;
    c.raw = at;
    at += scores ? up16(rows * own_cap * sizeof(float)) : 0;
    c.bytes = at;
    return c;
}

bool valid_heads(int Hq, int Hkv, int D) {
    return Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && (D == 64 || D == 96 || D == 128 || D == 256);
}

// Rows, segments and places are counted in int32.
bool valid_counts(long long B, long long T, long long Hq) { return B * T * Hq <= 0x3fffffffLL; }

}  // namespace
}  // namespace attn

extern "C" size_t mq_attn_ws_bytes(int B, int T, int Hq, int Hkv, int D, int prefix_cap, int own_cap, int scores) {
    using namespace attn;
    if (B <= 0 || T <= 0 || prefix_cap < 0 || own_cap < 0 || !valid_heads(Hq, Hkv, D) || !valid_counts(B, T, Hq)) return 0;
    return cut_of(B, T, Hq, Hkv, D, prefix_cap, own_cap, scores != 0).bytes;
}

extern "C" int mq_attn_prefix(const void* q, long long q_stride, int B, int T, int Hq, const mq_kv* prefix,
                              const mq_kv* own, const int32_t* own_len, float scale, void* out, int out_type,
                              float* lse, const float* score, float* score_out, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
    using namespace attn;
    if (B < 0 || T < 0) return MQ_ERR_SHAPE;
    const mq_kv* any = own ? own : prefix;
    if (!any) return MQ_ERR_NULL;
    int rc = MQ_OK;
    if (prefix) rc = mq::check_kv(prefix, true);
    if (rc == MQ_OK && own) rc = mq::check_kv(own, true);
    if (rc != MQ_OK) return rc;
    const int Hkv = any->heads, D = any->dim, type = any->type;
    if (prefix && own && (prefix->heads != Hkv || prefix->dim != D)) return MQ_ERR_SHAPE;
    if (prefix && prefix->type != type) return MQ_ERR_TYPE;
    if (out_type != type && out_type != MQ_F32) return MQ_ERR_TYPE;
    if (!valid_heads(Hq, Hkv, D) || (prefix && prefix->n != 1) || (own && own->n != B)) return MQ_ERR_SHAPE;
    if (B == 0 || T == 0) return MQ_OK;
    if (!valid_counts(B, T, Hq) || q_stride < (long long)Hq * D || q_stride % 8 != 0 || !std::isfinite(scale))
        return MQ_ERR_SHAPE;
    const int P = prefix ? prefix->cap : 0, cap = own ? own->cap : 0;
    if (!q || !out || !ws || (own && !own_len) || (score == nullptr) != (score_out == nullptr)) return MQ_ERR_NULL;
    if (!mq::aligned16(q) || !mq::aligned16(out) || !mq::aligned16(ws) || !mq::aligned16(own_len) ||
        !mq::aligned16(lse) || !mq::aligned16(score) || !mq::aligned16(score_out))
        return MQ_ERR_ALIGN;
    const bool scores = score_out && cap > 0;
    Cut c = cut_of(B, T, Hq, Hkv, D, P, cap, scores);
    if (all_segs(c.few) > 0x3fffffffLL || (long long)B * Hkv > 65535) return MQ_ERR_SHAPE;
    if (ws_bytes < c.bytes) return MQ_ERR_SCRATCH;
    rc = mq::check_arch();
    if (rc != MQ_OK) return rc;
    uint8_t* base = static_cast<uint8_t*>(ws);
    auto pieces = [&](size_t o, size_t ml, size_t info) {
        return Pieces{reinterpret_cast<float*>(base + o), reinterpret_cast<float2*>(base + ml),
                      reinterpret_cast<int2*>(base + info)};
    };
    const Pieces few = pieces(c.few_o, c.few_ml, c.few_info), many = pieces(c.many_o, c.many_ml, c.many_info);
    float* lse2 = scores ? reinterpret_cast<float*>(base + c.lse2) : nullptr;
    float* raw = scores ? reinterpret_cast<float*>(base + c.raw) : nullptr;
    constexpr float kLog2e = 1.4426950408889634f;

    if (all_segs(c.many) > 0) {
        ManyArgs m;
        m.plan = c.many;
        m.q = q;
        m.q_stride = q_stride;
        m.len = own_len;
        // a scale of next to nothing keeps masked products (-infinity) masked where zero would not
        m.scale_log2 = std::fmax(std::fabs(scale) * kLog2e, 1e-30f);
        m.negative = scale < 0.0f;
        m.out = many;
        rc = launch_many(m, c.prefix_many ? prefix : nullptr, c.own_many ? own : nullptr, D, type, stream);
        if (rc != MQ_OK) return rc;
    }
    if (all_segs(c.few) > 0) {
        FewArgs f;
        f.plan = c.few;
        f.q = q;
        f.q_stride = q_stride;
        f.pk = P > 0 ? prefix->k : nullptr;
        f.pv = P > 0 ? prefix->v : nullptr;
        f.p_row = P > 0 ? prefix->row_stride : 0;
        f.p_head = P > 0 ? prefix->head_stride : 0;
        f.ok = cap > 0 ? own->k : nullptr;
        f.ov = cap > 0 ? own->v : nullptr;
        f.o_seq = cap > 0 ? own->seq_stride : 0;
        f.o_row = cap > 0 ? own->row_stride : 0;
        f.o_head = cap > 0 ? own->head_stride : 0;
        f.len = own_len;
        f.scale_log2 = scale * kLog2e;
        f.out = few;
        f.raw = raw;
        const int held = few_blocks(D, type);
        if (f.plan.G > held) f.plan.G = held;
        rc = launch_few(f, D, type, stream);
        if (rc != MQ_OK) return rc;
    }
    JoinArgs j;
    j.prefix = {c.prefix_many ? many : few, P > 0 ? (c.prefix_many ? kManyRows : kFewRows) : 0};
    j.own = {c.own_many ? many : few, cap > 0 ? (c.own_many ? kManyRows : kFewRows) : 0};
    j.len = own_len;
    j.B = B;
    j.T = T;
    j.Hq = Hq;
    j.Hkv = Hkv;
    j.group = Hq / Hkv;
    j.own_cap = cap;
    j.seg0 = prefix_segs(c.own_many ? c.many : c.few);
    j.out = out;
    j.lse = lse;
    j.lse2 = lse2;
    const dim3 grid((unsigned)(((long long)B * T * Hq + 7) / 8));
    auto join = [&](auto o) {
        using O = decltype(o);
        auto kern = D == 64 ? attn_join_kernel<O, 64> : D == 96 ? attn_join_kernel<O, 96>
                    : D == 128 ? attn_join_kernel<O, 128> : attn_join_kernel<O, 256>;
        return mq::launch_pdl(kern, grid, dim3(256), 0, stream, j);
    };
    rc = out_type == MQ_F32 ? join(float()) : out_type == MQ_F16 ? join(__half()) : join(__nv_bfloat16());
    if (rc != MQ_OK || !scores) return rc;
    return mq::launch_pdl(attn_score_kernel, dim3((cap + 255) / 256, B * Hkv), dim3(256), 0, stream, raw, lse2, own_len,
                          score, score_out, T, Hq, Hkv, cap);
}
