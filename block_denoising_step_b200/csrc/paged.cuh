// The paged KV cache: what its kernels share.
//
// Keys and values live in pages of `page` positions, [n_pages][Hkv][page][hd]
// each; table[b][p] names the page that holds positions p * page .. of sequence
// b, and kv_len[b] counts its positions, the new tokens of a call included.  So
// the n_b new tokens of sequence b sit at positions kv_len[b] - n_b + i.  Rows
// of one KV head within a page are contiguous: a tile of keys is a few long
// runs of memory whatever the page size.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace dgen {
namespace paged {

constexpr uint32_t kNoRow = 0xFFFFFFFFu;

struct CacheView {
    uint8_t* k;
    uint8_t* v;
    const float* k_scale;  // [Hkv], E4M3 only
    const float* v_scale;
    const int* table;
    const int* kv_len;
    const int* cu;  // [B + 1] first token row of each sequence, or null: n_uniform rows each
    int n_pages, Hkv, page, B, table_stride, table_pages;
    int n_tokens, n_uniform;
    uint32_t page_mul, page_shift;  // pos / page = pos * page_mul >> page_shift for pos < 2^30

    __device__ __forceinline__ int page_of(int pos) const {
        return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(pos)) * page_mul >> page_shift);
    }
};

struct RowsView {  // [tokens][heads][hd], strides in elements
    uint8_t* p;
    long long ts, hs;
};

// Token rows [first, first + n) of sequence b, clamped to the token array.
__device__ __forceinline__ void seq_tokens(const CacheView& c, int b, int& first, int& n) {
    if (c.cu == nullptr) {
        first = b * c.n_uniform;
        n = c.n_uniform;
        return;
    }
    first = min(max(__ldg(c.cu + b), 0), c.n_tokens);
    n = max(min(__ldg(c.cu + b + 1), c.n_tokens) - first, 0);
}

// Cache row (one position of one KV head) of position pos of sequence b, or
// kNoRow when the table has no page for it.  Rows fit 32 bits: a row is at
// least 64 bytes.
__device__ __forceinline__ int page_entry(const CacheView& c, int b, int pidx) {
    return pidx < c.table_pages ? __ldg(c.table + static_cast<size_t>(b) * c.table_stride + pidx) : -1;
}
__device__ __forceinline__ uint32_t row_in_page(const CacheView& c, int id, int h, int off) {
    return static_cast<uint32_t>(id) < static_cast<uint32_t>(c.n_pages)
               ? (static_cast<uint32_t>(id) * c.Hkv + h) * c.page + off
               : kNoRow;
}

// Keys the query at position p sees, as [lo, hi): all of [0, len), cut by the
// causal order and by the window |p - j| < w.
__device__ __forceinline__ void visible(int p, int len, int causal, int window, int& lo, int& hi) {
    lo = window > 0 && p >= window ? p - window + 1 : 0;
    hi = causal ? min(len, p + 1) : (window > 0 && window < len - p ? p + window : len);
    hi = max(hi, lo);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF>
struct Half2;
template <>
struct Half2<true> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack2_bf16(a, b); }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
};
template <>
struct Half2<false> {
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
};

}  // namespace paged
}  // namespace dgen
