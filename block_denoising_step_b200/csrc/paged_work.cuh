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
    int G, R, KB, causal, window;
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

}  // namespace paged
}  // namespace dgen
