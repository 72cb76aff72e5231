// Caches in 4 bits on pages (include/mq.h, mq_kv4): where rows lie, and their scales.
//
// A page holds page_rows rows of every key head, head by head, each head as blocks of 16 rows. A block is
//     16 D / 2 bytes of the keys' numbers, as many of the values', 16 D / 32 bytes of the keys' scales, as many of the
//     values',
// so a run of rows of one head is one contiguous copy, and every lane of a warp finds its operands of the 16 x 8 x 16
// products in consecutive bytes (nb = D / 32 scales a row):
//   keys:   row r, dims 32 b + 8 t + 2 j + h (t, j < 4; h < 2): bits 16 h + 4 j of 32-bit word (4 r + t) nb + b;
//   values: row 8 p + 2 t + c, dim 32 u + 4 g + i (p, c < 2; t, i < 4; g < 8): bits 16 c + 4 i of word ((8 p + g) 4 + t) nb + u;
//   scales: byte r nb + b for the keys' dims 32 b .., byte (r / 2) 2 nb + 2 b + r % 2 for the values'.
// A number is n = nibble - 8; the writer makes -7 .. 7. A scale byte c is the top of a binary16 without its sign: c << 7 are that
// number's bits, so four significant bits and five of exponent. n has three, so n d is exact in binary16 and in
// bfloat16 alike, and whoever reads a row in either has it without a rounding.
#pragma once

#include "heads.cuh"

namespace kv4 {

constexpr int kBlockRows = 16;
constexpr int kMostCode = 191;        // d = 480: 7 d and what the readers' arithmetic makes of d (72 d) stay in binary16's range

__host__ __device__ constexpr int block_bytes(int D) { return 16 * (D + D / 16); }
__host__ __device__ constexpr int value_at(int D) { return 8 * D; }           // of a block's bytes
__host__ __device__ constexpr int key_scale_at(int D) { return 16 * D; }
__host__ __device__ constexpr int value_scale_at(int D) { return 16 * D + D / 2; }

// A cache as kernels see it.
struct Cache {
    uint8_t* pages;
    const int32_t* table;
    long long page_stride, table_stride;
    int n, width, n_pages, heads;
    int shift;                         // log2 of the rows of a page
    int head_bytes;                    // of a page's head

    // The page of row `row` of sequence `seq`; -1: none (an entry outside the pool).
    __device__ __forceinline__ int page(int seq, int row) const {
        const int p = __ldca(table + seq * table_stride + (row >> shift));
        return (unsigned)p < (unsigned)n_pages ? p : -1;
    }
    // The block that holds row `row` of its page.
    __device__ __forceinline__ uint8_t* block(int page, int head, int row, int bytes) const {
        return pages + page * page_stride + (long long)head * head_bytes + ((row & ((1 << shift) - 1)) / kBlockRows) * bytes;
    }
};

inline bool valid_dim(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }
inline bool valid_rows(int r) { return r >= 16 && r <= 1024 && (r & (r - 1)) == 0; }

// Bytes of a page that are used; of the pool from its first page to the end of its last.
inline long long page_used(const mq_kv4* c) { return (long long)c->page_rows / 16 * block_bytes(c->dim) * c->heads; }
inline long long pool_span(const mq_kv4* c) { return c->n_pages > 0 ? c->page_stride * (c->n_pages - 1) + page_used(c) : 0; }
// Whether a page and the `bytes` from b on have a byte in common (between pages may lie other things: other layers' pages).
inline bool meets_pages(const mq_kv4* c, const void* b, long long bytes) {
    return mq::rows_meet(c->pages, c->n_pages, c->page_stride, page_used(c), b, bytes);
}

// Sizes, then (with `pointers`) pointers.
inline int check(const mq_kv4* c, bool pointers) {
    if (!c) return MQ_ERR_NULL;
    if (c->n < 0 || c->width < 0 || c->n_pages < 0 || c->heads < 1 || c->heads > 65535 || !valid_dim(c->dim) || !valid_rows(c->page_rows))
        return MQ_ERR_SHAPE;
    if (c->page_stride < page_used(c) || c->page_stride % 16 != 0 || c->page_stride > (1LL << 40)) return MQ_ERR_SHAPE;
    if ((long long)c->width * c->page_rows > 0x7fffffffLL - 255) return MQ_ERR_SHAPE;
    if (c->n > 1 && (c->table_stride < c->width || c->table_stride > (1LL << 40))) return MQ_ERR_SHAPE;
    if (pointers && c->n > 0 && c->width > 0) {
        if (!c->table || (c->n_pages > 0 && !c->pages)) return MQ_ERR_NULL;
        if (!mq::aligned16(c->table) || !mq::aligned16(c->pages)) return MQ_ERR_ALIGN;
    }
    return MQ_OK;
}

inline Cache cache_of(const mq_kv4* c) {
    Cache k;
    k.pages = static_cast<uint8_t*>(c->pages);
    k.table = c->table;
    k.page_stride = c->page_stride;
    k.table_stride = c->n > 1 ? c->table_stride : 0;
    k.n = c->n;
    k.width = c->width;
    k.n_pages = c->n_pages;
    k.heads = c->heads;
    k.shift = 0;
    while ((1 << k.shift) < c->page_rows) ++k.shift;
    k.head_bytes = c->page_rows / 16 * block_bytes(c->dim);
    return k;
}

// The scale that a byte stands for: (8 + c % 8) 2^(c / 8 - 18), c 2^-17 below 8. As binary32: the byte's bits at the
// place of binary32's exponent are off by 2^112, subnormal ones too.
__device__ __forceinline__ float scale_of(int c) { return __uint_as_float((uint32_t)c << 20) * 5.192296858534828e33f; }

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
template <typename V>
__device__ __forceinline__ uint32_t as_word(const V& v) { return *reinterpret_cast<const uint32_t*>(&v); }

__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t mask, uint32_t bits) {   // (x & mask) | bits
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
    return y;
}

// A word's nibbles as four pairs of 16-bit numbers n d, exact: out[i] those of the nibbles i of both halves, with a
// pair of scales that came as bytes in the upper halves of two 16-bit words. A bit operation puts a nibble under an exponent, a fused
// multiply-add takes out what that added:
// bf16: 0x4300 | nibble is 128 + nibble, times d less 136 d (17 d: four bits by five, exact in bfloat16's eight).
// f16: 0x6400 | nibble << 4 is 16 (64 + nibble), times d / 16 less 72 d (9 d; below 2^16 up to d = 909).
template <typename T>
struct Scale;
template <>
struct Scale<__half> {
    __half2 mul, off;
    __device__ __forceinline__ static Scale of(uint32_t high_bytes) {
        const __half2 d = as_half2(high_bytes >> 1);
        return {__hmul2(d, __float2half2_rn(0.0625f)), __hmul2(d, __float2half2_rn(-72.0f))};
    }
};
template <>
struct Scale<__nv_bfloat16> {
    __nv_bfloat162 mul, off;
    __device__ __forceinline__ static Scale of(uint32_t high_bytes) {
        const __nv_bfloat162 d = __hmul2(as_bf162(high_bytes >> 4), __float2bfloat162_rn(5.192296858534828e33f));
        return {d, __hmul2(d, __float2bfloat162_rn(-136.0f))};
    }
    // One of the two scales for both numbers (an operand's half: no instruction).
    __device__ __forceinline__ Scale half(int e) const {
        return e ? Scale{__high2bfloat162(mul), __high2bfloat162(off)} : Scale{__low2bfloat162(mul), __low2bfloat162(off)};
    }
};
__device__ __forceinline__ void numbers(uint32_t w, const Scale<__half>& s, uint32_t (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = as_word(__hfma2(as_half2(mask_or(i == 0 ? w << 4 : w >> (4 * i - 4), 0x00f000f0u, 0x64006400u)), s.mul, s.off));
}
__device__ __forceinline__ void numbers(uint32_t w, const Scale<__nv_bfloat16>& s, uint32_t (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = as_word(__hfma2(as_bf162(mask_or(w >> (4 * i), 0x000f000fu, 0x43004300u)), s.mul, s.off));
}

// In f16, an eighth of them, with one shift instead of three for two more multiplications a scale: 0x6400 | nibble is 1024 + nibble, times
// d / 8 less 129 d; as above, times d / 128 less 9 d. 129 d stays below 2^16 up to d = 508 and has eight bits by four, d / 128 of the
// least scale is binary16's least number: all exact. (An eighth, because 1032 d would leave the range from d = 64 on.)
struct Eighth {
    static constexpr int kWords = 4;
    __half2 mul0, off0, mul1, off1;
    __device__ __forceinline__ static Eighth of(uint32_t high_bytes) {
        const __half2 d = as_half2(high_bytes >> 1);
        return {__hmul2(d, __float2half2_rn(0.125f)), __hmul2(d, __float2half2_rn(-129.0f)),
                __hmul2(d, __float2half2_rn(0.0078125f)), __hmul2(d, __float2half2_rn(-9.0f))};
    }
    __device__ __forceinline__ static Eighth from(const uint32_t* w) { return {as_half2(w[0]), as_half2(w[1]), as_half2(w[2]), as_half2(w[3])}; }
    __device__ __forceinline__ void to(uint32_t* w) const {
        w[0] = as_word(mul0), w[1] = as_word(off0), w[2] = as_word(mul1), w[3] = as_word(off1);
    }
    __device__ __forceinline__ Eighth half(int e) const {
        return e ? Eighth{__high2half2(mul0), __high2half2(off0), __high2half2(mul1), __high2half2(off1)}
                 : Eighth{__low2half2(mul0), __low2half2(off0), __low2half2(mul1), __low2half2(off1)};
    }
};
__device__ __forceinline__ void numbers(uint32_t w, const Eighth& s, uint32_t (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? w >> 8 : w;
        out[2 * i] = as_word(__hfma2(as_half2(mask_or(x, 0x000f000fu, 0x64006400u)), s.mul0, s.off0));
        out[2 * i + 1] = as_word(__hfma2(as_half2(mask_or(x, 0x00f000f0u, 0x64006400u)), s.mul1, s.off1));
    }
}

// nb consecutive words (or bytes), aligned as far as nb allows.
template <int nb, typename P>
__device__ __forceinline__ void words(P load, uint32_t (&w)[nb]) {
    if constexpr (nb % 4 == 0) {
#pragma unroll
        for (int i = 0; i < nb / 4; ++i) {
            const uint4 v = load(uint4(), i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if constexpr (nb == 2) {
        const uint2 v = load(uint2(), 0);
        w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < nb; ++i) w[i] = load(uint32_t(), i);
    }
}
// nb scale bytes as words of four.
template <int nb, typename P>
__device__ __forceinline__ void bytes(P load, uint32_t (&w)[(nb + 3) / 4]) {
    if constexpr (nb % 4 == 0) {
        words<nb / 4>(load, w);
    } else if constexpr (nb == 2) {
        w[0] = load(uint16_t(), 0);
    } else if constexpr (nb == 6) {
        w[0] = load(uint16_t(), 0) | (uint32_t)load(uint16_t(), 1) << 16;
        w[1] = load(uint16_t(), 2);
    } else {
        static_assert(nb == 3, "64, 96, 128 and 256 dims");
        w[0] = load(uint8_t(), 0) | (uint32_t)load(uint8_t(), 1) << 8 | (uint32_t)load(uint8_t(), 2) << 16;
    }
}
// Byte i of w in the upper halves of two 16-bit words; bytes 2 i and 2 i + 1.
template <int n>
__device__ __forceinline__ uint32_t twice(const uint32_t (&w)[n], int i) {
    return __byte_perm(w[i / 4], 0, 0x0404 + (i % 4) * 0x1010);
}
template <int n>
__device__ __forceinline__ uint32_t both(const uint32_t (&w)[n], int i) {
    return __byte_perm(w[i / 2], 0, i % 2 ? 0x3424 : 0x1404);
}

}  // namespace kv4
