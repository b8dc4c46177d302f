// Appending new tokens to the paged cache, with the rotation on the way.
//
//   y_j = x_j cos a_j - x_{j+hd/2} sin a_j,   y_{j+hd/2} = x_{j+hd/2} cos a_j + x_j sin a_j,
//   a_j = pos * base^(-2j/hd)
//
// for the query and key rows of each token; values are copied.  Keys and values
// go to their page (bf16 / fp16, or x / scale[head] as E4M3), rotated queries to
// q_out.  The rotation is computed in fp32 and rounded once.
//
// The angle is taken in double as turns, t = pos * (base^(-2j/hd) / 2 pi), and so are
// the sine and cosine of its fraction, rounded to fp32 once: positions in the
// millions are as exact as small ones, without a table.  A block computes the hd/2
// frequencies once and its tokens' sines once, for all heads.
//
// Memory-bound: every row is read and written once, 16 bytes per access.  A
// block takes up to kAppendTokens tokens (one warp each finds its token's sequence
// and page), then all threads sweep (row, 8 + 8 elements) items.  A thread's next
// items are on their way while it writes the current ones, the first ones already
// while the pages are looked up, which their addresses do not need.
//
// Measured on a B200 (device time of a replayed graph): prompts of up to 4,096 tokens in 16
// sequences, 32 query heads on 8 of 128 into E4M3 pages, 160 us (5.1 TB/s); eight canvases of
// 256 tokens, 16 heads on 8 of 256, 16 us (4.2 TB/s); one token 3.0 us (launch latency).
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

// Whether q = x * (1 / s) may round to another E4M3 value than x / s does.  Both are within 2 steps of fp32 of the
// exact quotient, so they can differ only within as many of a midpoint of E4M3 (for normal numbers: 20 zero bits
// behind a one behind the 3 kept ones); the coarser midpoints of its subnormals are not looked at one by one.
__device__ __forceinline__ bool near_midpoint(float q) {
    const uint32_t u = __float_as_uint(q);
    return (u & 0xFFFFFu) - 0x7FFF8u <= 16u || fabsf(q) < 0x1p-6f;
}

template <int HD, bool BF, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, E4M3 ? 3 : 4) paged_append_kernel(const AppendArgs a, int tokens_per_block) {
    constexpr int HALF = HD / 2;
    constexpr int CH = HALF / 8;  // items per row: 8 elements of each half
    constexpr int STEP = kAppendThreads / CH;  // rows between a thread's items
    constexpr int U = 2;                       // items in flight besides the ones at hand
    __shared__ double freq[HALF];
    __shared__ __align__(16) float2 cs[kAppendTokens][HALF];  // (read 16 bytes at a time)
    __shared__ int s_pos[kAppendTokens], s_page[kAppendTokens], s_off[kAppendTokens];
    using H2 = Half2<BF>;
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tok0 = blockIdx.x * tokens_per_block;
    const int nt = min(tokens_per_block, a.c.n_tokens - tok0);
    const int rows = a.Hq + 2 * a.c.Hkv, c = threadIdx.x % CH;
    // the items of this thread: (token t, row), always the same chunk
    int lt = 0, lrow = threadIdx.x / CH;  // the next item to load
    auto settle = [&](int& t, int& row) {
        while (row >= rows) {
            row -= rows;
            ++t;
        }
    };
    uint4 lo[U], hi[U];
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            settle(lt, lrow);
            if (lt < nt) {
                const RowsView& src = lrow < a.Hq ? a.q : (lrow < a.Hq + a.c.Hkv ? a.k : a.v);
                const int h = lrow < a.Hq ? lrow : lrow - a.Hq - (lrow < a.Hq + a.c.Hkv ? 0 : a.c.Hkv);
                const uint4* p = reinterpret_cast<const uint4*>(src.p + ((tok0 + lt) * src.ts + h * src.hs + c * 8) * 2);
                lo[u] = *p;
                hi[u] = *(p + HALF / 8);
            }
            lrow += STEP;
        }
    };
    load();
    if (a.rotate)
        for (int j = threadIdx.x; j < HALF; j += kAppendThreads)
            freq[j] = exp2(-a.log2_base * j / HALF) * 0.15915494309189533577;  // turns per position
    if (warp < nt) {
        const int tok = tok0 + warp;
        const int b = find_sequence(a.c, tok, lane);
        int pos = -1, id = -1, off = 0;
        if (b >= 0) {
            int first, n;
            const int len = max(__ldg(a.c.kv_len + b), 0);
            seq_tokens(a.c, b, first, n);
            if (tok - first < n) pos = len - n + (tok - first);
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
            double s, co;
            sincospi(2.0 * (turns - rint(turns)), &s, &co);
            cs[t][j] = make_float2(static_cast<float>(co), static_cast<float>(s));
        }
        __syncthreads();
    }
    int t = 0, row = threadIdx.x / CH;
    settle(t, row);
    while (t < nt) {
        uint4 xl[U], xh[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xl[u] = lo[u];
            xh[u] = hi[u];
        }
        load();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            settle(t, row);
            const int tt = t, rr = row;
            row += STEP;
            if (tt >= nt || s_pos[tt] < 0) continue;
            const bool is_q = rr < a.Hq, is_v = rr >= a.Hq + a.c.Hkv;
            const int h = is_q ? rr : rr - a.Hq - (is_v ? a.c.Hkv : 0);
            if (!is_q && static_cast<uint32_t>(s_page[tt]) >= static_cast<uint32_t>(a.c.n_pages)) continue;
            uint32_t* L = reinterpret_cast<uint32_t*>(&xl[u]);
            uint32_t* H = reinterpret_cast<uint32_t*>(&xh[u]);
            const bool turn = a.rotate && !is_v;
            float2 x[4], y[4];
            if (turn || (E4M3 && !is_q)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = H2::unpack(L[e]);
                    y[e] = H2::unpack(H[e]);
                }
            }
            if (turn) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 w = *reinterpret_cast<const float4*>(&cs[tt][c * 8 + 2 * e]);  // cos, sin, cos, sin
                    const float2 p = x[e], r = y[e];
                    x[e] = make_float2(p.x * w.x - r.x * w.y, p.y * w.z - r.y * w.w);
                    y[e] = make_float2(r.x * w.x + p.x * w.y, r.y * w.z + p.y * w.w);
                }
            }
            if (E4M3 && !is_q) {
                const float s = __ldg((is_v ? a.c.v_scale : a.c.k_scale) + h), inv = 1.f / s;
                uint32_t o[4];
                auto pack4 = [&](float2 p, float2 r) -> uint32_t {
                    return pack2_e4m3(p.x, p.y) | (static_cast<uint32_t>(pack2_e4m3(r.x, r.y)) << 16);
                };
                // the division where it matters: 1 / s of an extreme scale, quotients near a midpoint
                bool divide = !(s > 0x1p-100f && s < 0x1p100f);
                float2 qx[4], qy[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    qx[e] = make_float2(x[e].x * inv, x[e].y * inv);
                    qy[e] = make_float2(y[e].x * inv, y[e].y * inv);
                    divide |= near_midpoint(qx[e].x) || near_midpoint(qx[e].y) || near_midpoint(qy[e].x) || near_midpoint(qy[e].y);
                }
                if (divide) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        qx[e] = make_float2(x[e].x / s, x[e].y / s);
                        qy[e] = make_float2(y[e].x / s, y[e].y / s);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[e] = pack4(qx[2 * e], qx[2 * e + 1]);
                    o[2 + e] = pack4(qy[2 * e], qy[2 * e + 1]);
                }
                uint8_t* base = (is_v ? a.c.v : a.c.k) +
                                static_cast<size_t>(row_in_page(a.c, s_page[tt], h, s_off[tt])) * HD + c * 8;
                *reinterpret_cast<uint2*>(base) = make_uint2(o[0], o[1]);
                *reinterpret_cast<uint2*>(base + HALF) = make_uint2(o[2], o[3]);
            } else {
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        L[e] = H2::pack(x[e].x, x[e].y);
                        H[e] = H2::pack(y[e].x, y[e].y);
                    }
                }
                uint8_t* base =
                    is_q ? a.q_out.p + ((tok0 + tt) * a.q_out.ts + h * a.q_out.hs + c * 8) * 2
                         : (is_v ? a.c.v : a.c.k) +
                               (static_cast<size_t>(row_in_page(a.c, s_page[tt], h, s_off[tt])) * HD + c * 8) * 2;
                *reinterpret_cast<uint4*>(base) = xl[u];
                *reinterpret_cast<uint4*>(base + HD) = xh[u];
            }
        }
        settle(t, row);
    }
}

}  // namespace paged
}  // namespace dgen
