// Appending new tokens to the paged cache, with the rotation on the way.
//
//   y_j = x_j cos a_j - x_{j+hd/2} sin a_j,   y_{j+hd/2} = x_{j+hd/2} cos a_j + x_j sin a_j,
//   a_j = pos * base^(-2j/hd)
//
// for the query and key rows of each token; values are copied.  Keys and values
// go to their page (bf16 / fp16, or x / scale[head] as E4M3), rotated queries to
// q_out.  The rotation is computed in fp32 and rounded once.
//
// The angle is taken in double as turns, t = pos * (base^(-2j/hd) / 2 pi), of
// which only the fraction enters the fp32 sine and cosine: positions in the
// millions keep 1e-7 of absolute accuracy without a table.  Each block computes
// the hd/2 frequencies once and its tokens' sines once, for all heads.
//
// Memory-bound: every row is read and written once, 16 bytes per access.  A
// block takes up to kTokens tokens (one warp each finds its token's sequence
// and page), then all threads sweep (row, 8 + 8 elements) items, kUnroll loads
// in flight each.
#pragma once

#include "paged.cuh"

namespace dgen {
namespace paged {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;  // tokens per block at most (one warp each)

struct AppendArgs {
    CacheView c;
    RowsView q, k, v, q_out;
    int Hq;            // 0: no queries
    double log2_base;  // log2 of the rotation's base
    int rotate;
};

// The sequence that owns token row tok (32-ary search over cu), or -1.
__device__ __forceinline__ int find_sequence(const CacheView& c, int tok, int lane) {
    if (c.cu == nullptr) return tok / c.n_uniform < c.B ? tok / c.n_uniform : -1;
    int lo = 0, hi = c.B + 1;  // the answer + 1 = number of entries <= tok, in [lo, hi]
    while (hi > lo) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && __ldg(c.cu + at) <= tok;
        const int n = __popc(__ballot_sync(0xffffffffu, le));
        if (n == 0) return lo - 1;
        const int last = lo + (n - 1) * step;  // entry `last` <= tok, the next probe is not
        hi = min(hi, last + step);
        lo = last + 1;
    }
    const int b = lo - 1;
    return b < c.B ? b : -1;
}

template <int HD, bool BF, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a, int tokens_per_block) {
    constexpr int HALF = HD / 2;
    constexpr int CH = HALF / 8;  // items per row: 8 elements of each half
    __shared__ double freq[HALF];
    __shared__ float2 cs[kAppendTokens][HALF];
    __shared__ int s_pos[kAppendTokens], s_page[kAppendTokens], s_off[kAppendTokens];
    using H2 = Half2<BF>;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok0 = blockIdx.x * tokens_per_block;
    const int nt = min(tokens_per_block, a.c.n_tokens - tok0);
    if (a.rotate)
        for (int j = threadIdx.x; j < HALF; j += kAppendThreads)
            freq[j] = exp2(-a.log2_base * j / HALF) * 0.15915494309189533577;  // turns per position
    if (warp < nt) {
        const int tok = tok0 + warp;
        const int b = find_sequence(a.c, tok, lane);
        int pos = -1, id = -1, off = 0;
        if (b >= 0) {
            int first, n;
            seq_tokens(a.c, b, first, n);
            if (tok - first < n) pos = max(__ldg(a.c.kv_len + b), 0) - n + (tok - first);
            if (pos >= 0) {
                const int pg = pos < (1 << 30) ? a.c.page_of(pos) : a.c.table_pages;  // (the table ends at 2^30)
                id = page_entry(a.c, b, pg);
                off = pos - pg * a.c.page;
            }
        }
        if (lane == 0) {
            s_pos[warp] = pos;
            s_page[warp] = id;
            s_off[warp] = off;
        }
    }
    __syncthreads();
    if (a.rotate) {
        for (int i = threadIdx.x; i < nt * HALF; i += kAppendThreads) {
            const int t = i / HALF, j = i % HALF;
            const double turns = freq[j] * s_pos[t];
            float s, co;
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &co);
            cs[t][j] = make_float2(co, s);
        }
        __syncthreads();
    }
    const int rows = a.Hq + 2 * a.c.Hkv;
    const int items = nt * rows * CH;
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < items; i0 += U * kAppendThreads) {
        uint4 lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kAppendThreads;
            if (i < items) {
                const int c = i % CH, row = (i / CH) % rows, tok = tok0 + i / (CH * rows);
                const RowsView& src = row < a.Hq ? a.q : (row < a.Hq + a.c.Hkv ? a.k : a.v);
                const int h = row < a.Hq ? row : (row - a.Hq) % a.c.Hkv;
                const uint4* p = reinterpret_cast<const uint4*>(src.p + (tok * src.ts + h * src.hs + c * 8) * 2);
                lo[u] = *p;
                hi[u] = *(p + HALF / 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kAppendThreads;
            if (i >= items) break;
            const int c = i % CH, row = (i / CH) % rows, t = i / (CH * rows);
            if (s_pos[t] < 0) continue;
            const bool is_q = row < a.Hq, is_v = row >= a.Hq + a.c.Hkv;
            const int h = is_q ? row : (row - a.Hq) % a.c.Hkv;
            if (!is_q && static_cast<uint32_t>(s_page[t]) >= static_cast<uint32_t>(a.c.n_pages)) continue;
            uint32_t* L = reinterpret_cast<uint32_t*>(&lo[u]);
            uint32_t* H = reinterpret_cast<uint32_t*>(&hi[u]);
            float2 x[4], y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = H2::unpack(L[e]);
                y[e] = H2::unpack(H[e]);
            }
            if (a.rotate && !is_v) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 c0 = cs[t][c * 8 + 2 * e], c1 = cs[t][c * 8 + 2 * e + 1];
                    const float2 p = x[e], r = y[e];
                    x[e] = make_float2(p.x * c0.x - r.x * c0.y, p.y * c1.x - r.y * c1.y);
                    y[e] = make_float2(r.x * c0.x + p.x * c0.y, r.y * c1.x + p.y * c1.y);
                }
            }
            if (E4M3 && !is_q) {
                const float s = __ldg((is_v ? a.c.v_scale : a.c.k_scale) + h);
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[e] = pack2_e4m3(x[2 * e].x / s, x[2 * e].y / s) |
                           (static_cast<uint32_t>(pack2_e4m3(x[2 * e + 1].x / s, x[2 * e + 1].y / s)) << 16);
                    o[2 + e] = pack2_e4m3(y[2 * e].x / s, y[2 * e].y / s) |
                               (static_cast<uint32_t>(pack2_e4m3(y[2 * e + 1].x / s, y[2 * e + 1].y / s)) << 16);
                }
                uint8_t* base = (is_v ? a.c.v : a.c.k) +
                                static_cast<size_t>(row_in_page(a.c, s_page[t], h, s_off[t])) * HD + c * 8;
                *reinterpret_cast<uint2*>(base) = make_uint2(o[0], o[1]);
                *reinterpret_cast<uint2*>(base + HALF) = make_uint2(o[2], o[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    L[e] = H2::pack(x[e].x, x[e].y);
                    H[e] = H2::pack(y[e].x, y[e].y);
                }
                uint8_t* base =
                    is_q ? a.q_out.p + ((tok0 + t) * a.q_out.ts + h * a.q_out.hs + c * 8) * 2
                         : (is_v ? a.c.v : a.c.k) +
                               (static_cast<size_t>(row_in_page(a.c, s_page[t], h, s_off[t])) * HD + c * 8) * 2;
                *reinterpret_cast<uint4*>(base) = lo[u];
                *reinterpret_cast<uint4*>(base + HD) = hi[u];
            }
        }
    }
}

}  // namespace paged
}  // namespace dgen
