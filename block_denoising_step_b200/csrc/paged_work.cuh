// How the attention kernels over the paged cache divide a batch of unequal
// sequences, without the host knowing their lengths.
//
// A unit is one row tile (up to R of the n_b * G query rows that share a KV
// head) of one sequence and KV head; its keys are dealt in blocks of KB.  All
// units' blocks, in unit order, form one line of T blocks, which is cut into
// equal pieces, one per CTA: each CTA finds T and its first unit by scanning the
// lengths (32 sequences per step).  A unit cut by a piece's end is finished by
// the CTA that completes last, from the partial results (O, m, l) of all pieces,
// added in piece order: which CTA does it does not change the result.
#pragma once

#include "paged.cuh"

namespace dgen {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescale = 8.f;  // a running maximum moves only when it grows by more than 2^8

struct SeqInfo {
    int first, n;      // token rows
    int len;           // keys (kv_len, at most what the table can hold)
    int pos0;          // position of the first new token
    int lo, hi;        // keys any of its queries sees
    int tiles;         // row tiles
    int blocks;        // key blocks per unit
    int b;
    long long end;     // T of all sequences up to and including this one
};

struct Partition {
    int G, R, KB, align, causal, window;  // align: blocks start at multiples of it (a power of two)
    int rows_min, rows_max;  // query rows per KV head of the sequences this launch takes
};

__device__ __forceinline__ long long warp_inclusive(long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Lane's sequence of the 32 starting at base; .end = `before` + inclusive prefix.
__device__ __forceinline__ SeqInfo load_chunk(const CacheView& c, const Partition& p, int base, long long before,
                                              int lane) {
    SeqInfo s{};
    s.b = base + lane;
    long long w = 0;
    if (s.b < c.B) {
        seq_tokens(c, s.b, s.first, s.n);
        const int full = max(__ldg(c.kv_len + s.b), 0);
        s.pos0 = full - s.n;
        const long long cap = static_cast<long long>(c.table_pages) * c.page;
        s.len = full < cap ? full : static_cast<int>(cap);
        const int rows = s.n * p.G;
        if (rows >= p.rows_min && rows <= p.rows_max && rows > 0) {
            int lo1, hi0;
            visible(s.pos0, s.len, p.causal, p.window, s.lo, hi0);
            visible(s.pos0 + s.n - 1, s.len, p.causal, p.window, lo1, s.hi);
            s.lo &= ~(p.align - 1);
            s.hi = max(s.hi, s.lo);
            s.tiles = (rows + p.R - 1) / p.R;
            s.blocks = max(1, (s.hi - s.lo + p.KB - 1) / p.KB);  // no key: one block that writes zeros
            w = static_cast<long long>(s.tiles) * c.Hkv * s.blocks;
        }
    }
    s.end = before + warp_inclusive(w, lane);
    return s;
}

__device__ __forceinline__ SeqInfo pick(const SeqInfo& s, int src) {
    SeqInfo r;
    const unsigned f = 0xffffffffu;
    r.first = __shfl_sync(f, s.first, src);
    r.n = __shfl_sync(f, s.n, src);
    r.len = __shfl_sync(f, s.len, src);
    r.pos0 = __shfl_sync(f, s.pos0, src);
    r.lo = __shfl_sync(f, s.lo, src);
    r.hi = __shfl_sync(f, s.hi, src);
    r.tiles = __shfl_sync(f, s.tiles, src);
    r.blocks = __shfl_sync(f, s.blocks, src);
    r.b = __shfl_sync(f, s.b, src);
    r.end = __shfl_sync(f, s.end, src);
    return r;
}

// A warp's walk over the units of its CTA's piece.
struct Walk {
    SeqInfo mine;            // this lane's sequence of the current chunk
    int base;                // first sequence of the chunk
    long long total, per, t, t_end;

    __device__ __forceinline__ void start(const CacheView& c, const Partition& p, int lane, int min_blocks) {
        long long before = 0;
        for (base = 0;; base += 32) {
            mine = load_chunk(c, p, base, before, lane);
            before = __shfl_sync(0xffffffffu, mine.end, 31);
            if (base + 32 >= c.B) break;
        }
        total = before;
        per = (total + gridDim.x - 1) / gridDim.x;
        if (per < min_blocks) per = min_blocks;
        t = per * blockIdx.x;
        t_end = t + per < total ? t + per : total;
        if (base > 0) {
            base = 0;
            mine = load_chunk(c, p, 0, 0, lane);
        }
    }
    // The unit at t: its sequence, unit number within the sequence and blocks
    // [b0, b1); false when the piece is done.  u0 is the unit's first block on
    // the line.
    __device__ __forceinline__ bool next(const CacheView& c, const Partition& p, int lane, SeqInfo& s, int& unit,
                                         int& b0, int& b1, long long& u0) {
        if (t >= t_end) return false;
        long long chunk_end = __shfl_sync(0xffffffffu, mine.end, 31);
        while (t >= chunk_end) {
            base += 32;
            mine = load_chunk(c, p, base, chunk_end, lane);
            chunk_end = __shfl_sync(0xffffffffu, mine.end, 31);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, t < mine.end)) - 1;
        s = pick(mine, src);
        const long long seq0 = s.end - static_cast<long long>(s.tiles) * c.Hkv * s.blocks;
        unit = static_cast<int>((t - seq0) / s.blocks);
        u0 = seq0 + static_cast<long long>(unit) * s.blocks;
        b0 = static_cast<int>(t - u0);
        const long long left = t_end - u0;
        b1 = left < s.blocks ? static_cast<int>(left) : s.blocks;
        t = u0 + b1;
        return true;
    }
};

struct AttendArgs {
    CacheView c;
    RowsView q, out;
    Partition p;
    float* lse;  // [tokens][Hq] or null
    int Hq;
    float scale, cap;
    int q_bf16;
    unsigned int* counters;  // [grid]
    float* parts;            // [2 grid][R][HD] then [2 grid][R][2]
    int min_blocks;
};

// log2(e) cap tanh(s / cap) from x = 2 log2(e) s / cap, with tanh y = 1 - 2 / (1 + e^2y)
__device__ __forceinline__ float capped_log2(float x, float cap) {
    return kLog2e * cap * (1.f - __fdividef(2.f, 1.f + exp2f(x)));
}

// One row tile: where its rows' outputs go.
struct Tile {
    int first, row0, rows, h;  // first token of the sequence, first and number of query rows, KV head
};

// Four columns of a row: v / l (times the values' scale) rounded to the output
// type; the row's log-sum-exp goes with column 0.  l = 0: no key seen.
__device__ __forceinline__ void store4(const AttendArgs& a, const Tile& t, bool bf, float vscale, int r, int col,
                                       float4 v, float m, float l) {
    const int tok = t.first + (t.row0 + r) / a.p.G, head = t.h * a.p.G + (t.row0 + r) % a.p.G;
    const float inv = l > 0.f || l != l ? vscale / l : 0.f;
    uint2 w;
    if (bf)
        w = make_uint2(Half2<true>::pack(v.x * inv, v.y * inv), Half2<true>::pack(v.z * inv, v.w * inv));
    else
        w = make_uint2(Half2<false>::pack(v.x * inv, v.y * inv), Half2<false>::pack(v.z * inv, v.w * inv));
    *reinterpret_cast<uint2*>(a.out.p + (tok * a.out.ts + head * a.out.hs + col) * 2) = w;
    if (a.lse != nullptr && col == 0)
        a.lse[static_cast<size_t>(tok) * a.Hq + head] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Partial results: slot 2 c + 1 holds the piece that starts a unit in CTA c,
// slot 2 c the one that continues it there.  O is relative to 2^m, not divided by l.
__device__ __forceinline__ float* part_o(const AttendArgs& a, int hd, size_t slot, int r) {
    return a.parts + (slot * a.p.R + r) * hd;
}
__device__ __forceinline__ float* part_ml(const AttendArgs& a, int hd, size_t slot, int r) {
    return a.parts + 2 * static_cast<size_t>(gridDim.x) * a.p.R * hd + (slot * a.p.R + r) * 2;
}

// Adds the pieces of a unit cut over CTAs c_first .. c_last, in that order, by
// `threads` threads; all of them are in memory.
template <int HD>
__device__ __forceinline__ void join_pieces(const AttendArgs& a, const Tile& t, bool bf, float vscale, int c_first,
                                            int c_last, int tid, int threads) {
    for (int i = tid; i < t.rows * (HD / 4); i += threads) {
        const int r = i / (HD / 4), col = (i % (HD / 4)) * 4;
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = c_first; k <= c_last; ++k) {
            const size_t slot = 2 * static_cast<size_t>(k) + (k == c_first ? 1 : 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml(a, HD, slot, r)));
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part_o(a, HD, slot, r) + col));
            const float mn = fmaxf(m, ml.x);
            // (a piece without a maximum holds zeros, or NaN from NaN scores alone)
            const float fo = m == -INFINITY ? 1.f : exp2f(m - mn), fn = ml.x == -INFINITY ? 1.f : exp2f(ml.x - mn);
            v.x = v.x * fo + x.x * fn, v.y = v.y * fo + x.y * fn;
            v.z = v.z * fo + x.z * fn, v.w = v.w * fo + x.w * fn;
            l = l * fo + ml.y * fn;
            m = mn;
        }
        store4(a, t, bf, vscale, r, col, v, m, l);
    }
}

}  // namespace paged
}  // namespace dgen
