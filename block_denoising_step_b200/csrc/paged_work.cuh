// How the attention kernels over the paged cache divide a batch of unequal
// sequences, without the host knowing their lengths.
//
// The n_b * G query rows that share a KV head of a sequence are cut into row tiles
// of R; TS neighbouring row tiles form a unit (sequence, KV head, super tile), whose
// keys are dealt in blocks of KB.  All units' blocks, in unit order, form one line
// of T blocks, cut into equal pieces, one per team of TS CTAs (where units are
// few or short, each is cut by itself or not at all); member m of a team
// computes row tile m of each unit, so that the team reads the same keys at the same
// time and all but one member find them in L2 (separate units per CTA read them from
// HBM once per row tile: 1.2 GB instead of 0.3 for eight canvases over 4096 tokens).
// A unit counts the blocks its own rows see (causal order, window), so a prompt's
// first rows weigh little.  Each warp finds T and its piece by scanning the lengths,
// 32 sequences per step; the prefix sums over a sequence's units have a closed form.
// A unit cut by a piece's end is joined from its pieces' partial results (O, m, l),
// added in piece order: which CTA or thread does it does not change the result.
#pragma once

#include "paged.cuh"

namespace dgen {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescale = 8.f;  // a running maximum moves only when it grows by more than 2^8
// Weights in fp16 are 2^kHalfLift times those relative to the running maximum: up to 2^15, below fp16's largest, so
// that they keep their 11 bits down to 2^-21 of it and lose 2^-32 of it at most below (without, keys at 2^-18 of
// the maximum were 0.8 % off, and those at 2^-25 gone).  Their sums are relative to m - kHalfLift alike; bf16 has
// fp32's range.
constexpr float kHalfLift = 7.f;

struct SeqInfo {
    int first, n;      // token rows
    int len;           // keys (kv_len, at most what the table can hold)
    int pos0;          // position of the first new token
    int tiles;         // super tiles
    int lo, blocks;    // irregular: first key and blocks of every unit
    int regular;       // units have ranges of their own (prefix_blocks)
    int b;
    int head;          // length of one KV head's super tiles on the line, in blocks or in pieces
    int end;           // blocks of all sequences up to and including this one (the host keeps T below 2^31)
};

struct Partition {
    int G, R, TS, KB, log2_kb, causal, window;
    int tokens;              // of a super tile: R / G * TS
    int unit_cost;           // blocks that starting and ending a unit takes the time of
    int align;               // blocks start at multiples of it: KB, or 1 where sequences have one tile
    int rows_min, rows_max;  // query rows per KV head of the sequences this launch takes
};

// sum over i < n of floor((a i + b) / m) (Euclid's scheme on the lattice points
// below the line); a n + b below 2^31
__host__ __device__ inline long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long sum = 0;
    while (n > 0) {
        const uint32_t qa = a / m, qb = b / m;
        sum += static_cast<long long>(n) * (n - 1) / 2 * qa + static_cast<long long>(n) * qb;
        a -= qa * m;
        b -= qb * m;
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y - n * m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// Blocks of the super tiles before number k of a regular sequence (pos0 >= 0,
// len = pos0 + n): tile i holds the tokens i T .. (T = tokens of a super tile) and
// sees blocks floor(lo / KB) .. ceil(hi / KB) - 1.  (Positions are below 2^30, and
// so is every sum of blocks here: the host bounds the line.)
// (Not inlined: a launch's first pass over any code waits for it, and this is long.)
__host__ __device__ __noinline__ static int prefix_masked(int n, int len, int pos0, int tiles, int T, int KB, int whole,
                                                          int causal, int window, int k) {
    int up;  // sum of ceil(hi / KB)
    if (causal) {
        const int m = k < tiles ? k : tiles - 1;  // the last tile may be short
        up = static_cast<int>(floor_sum(m, KB, T, pos0 + T + KB - 1)) + (k - m) * whole;
    } else {  // hi = min(len, pos0 + (i + 1) T - 1 + w): reaches len from tile r on
        const long long d = static_cast<long long>(n) + 1 - window;
        int r = d <= 0 ? 0 : (static_cast<int>(d) + T - 1) / T - 1;
        r = r < 0 ? 0 : r > tiles - 1 ? tiles - 1 : r;
        const int m = k < r ? k : r;
        up = (m > 0 ? static_cast<int>(floor_sum(m, KB, T, pos0 + T - 1 + window + KB - 1)) : 0) + (k - m) * whole;
    }
    if (window == 0) return up;
    // lo = max(0, pos0 + i T - w + 1): positive from tile r on
    const int d = window - 1 - pos0;
    const int r = d <= 0 ? 0 : d > (1 << 30) ? k : (d + T - 1) / T;
    return up - (k > r ? static_cast<int>(floor_sum(k - r, KB, T, pos0 + r * T - window + 1)) : 0);
}
__host__ __device__ inline int prefix_blocks(const SeqInfo& s, const Partition& p, int k) {
    const int whole = (s.len + p.KB - 1) >> p.log2_kb;
    return !p.causal && p.window == 0 ? k * whole
                                      : prefix_masked(s.n, s.len, s.pos0, s.tiles, p.tokens, p.KB, whole, p.causal,
                                                      p.window, k);
}

// Blocks by which a CTA may take longer with whole units than with cut ones: the
// join costs about as much (2 us against 1 us a block).
constexpr int kWholeSlack = 2;

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Lane's sequence of the 32 starting at base.
__device__ __forceinline__ SeqInfo load_chunk(const CacheView& c, const Partition& p, int base, int lane) {
    SeqInfo s{};
    s.b = base + lane;
    if (s.b < c.B) {
        const int full = max(__ldg(c.kv_len + s.b), 0);
        seq_tokens(c, s.b, s.first, s.n);
        s.pos0 = full - s.n;
        const long long cap = static_cast<long long>(c.table_pages) * c.page;
        s.len = full < cap ? full : static_cast<int>(cap);
        const int rows = s.n * p.G;
        if (rows >= p.rows_min && rows <= p.rows_max && rows > 0) {
            s.tiles = rows <= p.R * p.TS ? 1 : (rows + p.R * p.TS - 1) / (p.R * p.TS);
            s.regular = s.tiles > 1 && p.align == p.KB && s.pos0 >= 0 && s.len == full;
            int hi, x;
            visible(s.pos0, s.len, p.causal, p.window, s.lo, x);
            visible(s.pos0 + s.n - 1, s.len, p.causal, p.window, x, hi);
            s.lo &= ~(p.align - 1);
            s.blocks = max(1, (hi - s.lo + p.KB - 1) >> p.log2_kb);  // no key: one block that writes zeros
        }
    }
    return s;
}
// Its length on the line, and the line's up to it (`before` the chunk).  cut > 0:
// the line counts pieces of `cut` blocks of each unit, else blocks, with unit_cost
// empty ones before each unit's (CTAs with many short units took up to 1.5 times as
// long without: a ragged batch of prompt chunks 397 us instead of 286, 1,536 windows
// of 1,024 keys 90 us instead of 74).
__device__ __forceinline__ void place(SeqInfo& s, const CacheView& c, const Partition& p, int cut, int before, int lane) {
    if (cut > 0)
        s.head = s.tiles * (s.blocks <= cut ? 1 : (s.blocks + cut - 1) / cut);
    else
        s.head = (s.regular ? prefix_blocks(s, p, s.tiles) : s.tiles * s.blocks) + s.tiles * p.unit_cost;
    s.end = before + warp_inclusive(s.head * c.Hkv, lane);
}

__device__ __forceinline__ SeqInfo pick(const SeqInfo& s, int src) {
    SeqInfo r;
    const unsigned f = 0xffffffffu;
    r.first = __shfl_sync(f, s.first, src);
    r.n = __shfl_sync(f, s.n, src);
    r.len = __shfl_sync(f, s.len, src);
    r.pos0 = __shfl_sync(f, s.pos0, src);
    r.tiles = __shfl_sync(f, s.tiles, src);
    r.lo = __shfl_sync(f, s.lo, src);
    r.blocks = __shfl_sync(f, s.blocks, src);
    r.regular = __shfl_sync(f, s.regular, src);
    r.b = __shfl_sync(f, s.b, src);
    r.head = __shfl_sync(f, s.head, src);
    r.end = __shfl_sync(f, s.end, src);
    return r;
}

// First key of a regular sequence's super tile k, where its blocks start.
__device__ __forceinline__ int first_key(const SeqInfo& s, const Partition& p, int k) {
    const int p0 = s.pos0 + k * p.tokens;
    return p.window > 0 && p0 >= p.window ? (p0 - p.window + 1) & ~(p.KB - 1) : 0;
}

// A piece of a unit, as one member of the team sees it.
struct Piece {
    int end;             // no piece: the walk is over
    int b, h;            // sequence, KV head
    int first, row0;     // first token row of the sequence, first query row of the row tile
    int rows;            // its rows (<= 0: this member has none)
    int pos0, len;
    int key0;            // first key of this member's first block
    int n;               // its blocks (0: it sees no key here)
    int hi;              // keys from here on are not seen by any of its rows
    int whole, starts;   // the piece is the whole unit / holds the unit's first block
    int t_first, t_last; // teams that hold the unit's pieces
};

// A warp's walk over the units of its team's piece of the line.
struct Walk {
    SeqInfo mine;  // this lane's sequence of the current chunk
    int base;      // first sequence of the chunk
    int member, cut;  // cut > 0: the line is made of pieces of `cut` blocks, which no unit shares
    int total, per, t, t_end;

    __device__ __forceinline__ void start(const CacheView& c, const Partition& p, int lane, int cta, int n_ctas) {
        const int log2_ts = __ffs(p.TS) - 1, teams = n_ctas >> log2_ts;  // (TS is a power of two)
        member = cta & (p.TS - 1);
        int before = 0, units = 0, most = 0, nominal = 0;  // most: blocks of the longest unit, at most
        for (base = 0;; base += 32) {
            mine = load_chunk(c, p, base, lane);
            place(mine, c, p, 0, before, lane);
            before = __shfl_sync(0xffffffffu, mine.end, 31);
            units += __reduce_add_sync(0xffffffffu, mine.tiles);
            nominal += __reduce_add_sync(0xffffffffu, mine.tiles * mine.blocks);
            most = max(most, __reduce_max_sync(0xffffffffu, mine.blocks));
            if (base + 32 >= c.B) break;
        }
        units *= c.Hkv;
        nominal *= c.Hkv;
        total = before;
        per = (total + teams - 1) / teams;
        cut = 0;
        if (units > 0 && 2 * units <= teams) {
            // fewer units than teams: each cut by itself, one piece a team.  Even lengths take all teams' share,
            // others pieces of T / (teams - units), of which there are at most T / that + units = teams.
            cut = nominal == units * most ? (most + teams / units - 1) / (teams / units)
                                          : (nominal + teams - units - 1) / (teams - units);
            if (most <= cut + kWholeSlack) cut = most;
        } else if (units > 0 && static_cast<long long>((units + teams - 1) / teams) * most <= per + kWholeSlack) {
            cut = most;  // whole units
        }
        if (cut > 0) {
            before = 0;
            for (base = 0;; base += 32) {
                if (c.B > 32) mine = load_chunk(c, p, base, lane);
                place(mine, c, p, cut, before, lane);
                before = __shfl_sync(0xffffffffu, mine.end, 31);
                if (base + 32 >= c.B) break;
            }
            total = before;
            per = (total + teams - 1) / teams;
        }
        // (per * team can pass 2^31 only behind the line's end)
        const long long at = static_cast<long long>(per) * (cta >> log2_ts);
        t = at < total ? static_cast<int>(at) : total;
        t_end = per < total - t ? t + per : total;
        if (base > 0) {
            base = 0;
            mine = load_chunk(c, p, 0, lane);
            place(mine, c, p, cut, 0, lane);
        }
    }
    // The unit at t and this team's blocks of it; false when the piece is done.
    __device__ __forceinline__ bool next(const CacheView& c, const Partition& p, int lane, Piece& q) {
        if (t >= t_end) return false;
        int chunk_end = __shfl_sync(0xffffffffu, mine.end, 31);
        while (t >= chunk_end) {
            if (base + 32 >= c.B) return false;  // (never with the lengths of start(); ends the walk if they changed since)
            base += 32;
            mine = load_chunk(c, p, base, lane);
            place(mine, c, p, cut, chunk_end, lane);
            chunk_end = __shfl_sync(0xffffffffu, mine.end, 31);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, t < mine.end)) - 1;
        const SeqInfo s = pick(mine, src);
        const int seq0 = s.end - s.head * c.Hkv;
        q.h = (t - seq0) / s.head;
        const int head0 = seq0 + q.h * s.head, x = t - head0;
        // the super tile: the last k with prefix(k) <= x
        int k, u0, blocks, lo, len;  // len: the unit's length on the line
        if (cut > 0 || !s.regular) {
            len = cut <= 0 ? s.blocks + p.unit_cost : s.blocks <= cut ? 1 : (s.blocks + cut - 1) / cut;
            k = s.tiles == 1 ? 0 : x / len;
            u0 = head0 + k * len;
            blocks = s.blocks;
            lo = s.lo;
            if (s.regular) {
                blocks = prefix_blocks(s, p, k + 1) - prefix_blocks(s, p, k);
                lo = first_key(s, p, k);
            }
        } else {
            int from = 0, to = s.tiles;  // prefix(from) <= x < prefix(to)
            while (to - from > 1) {
                const int step = (to - from + 31) / 32, at = from + lane * step;
                const bool le = at < to && prefix_blocks(s, p, at) + at * p.unit_cost <= x;
                const int cnt = __popc(__ballot_sync(0xffffffffu, le));
                from += (cnt - 1) * step;
                to = min(to, from + step);
            }
            k = from;
            const int before = prefix_blocks(s, p, k);
            u0 = head0 + before + k * p.unit_cost;
            blocks = prefix_blocks(s, p, k + 1) - before;
            len = blocks + p.unit_cost;
            lo = first_key(s, p, k);
        }
        int b0, b1;
        bool starts, ends;  // the piece has the unit's beginning, its end
        if (cut > 0) {
            b0 = min((t - u0) * cut, blocks);
            b1 = min(b0 + cut, blocks);
            starts = t == u0;
            ends = t == u0 + len - 1;
            ++t;
        } else {
            const int e0 = t - u0, e1 = min(t_end - u0, len);
            starts = e0 == 0;
            ends = e1 == len;
            b0 = max(e0 - p.unit_cost, 0);
            b1 = max(e1 - p.unit_cost, 0);
            t = u0 + e1;
        }
        q.end = 0;
        q.b = s.b;
        q.first = s.first;
        q.pos0 = s.pos0;
        q.len = s.len;
        q.row0 = (k * p.TS + member) * p.R;
        q.rows = min(p.R, s.n * p.G - q.row0);
        q.t_first = per == 1 ? u0 : u0 / per;
        q.t_last = cut > 0 && len == 1 ? q.t_first : per == 1 ? u0 + len - 1 : (u0 + len - 1) / per;
        q.whole = starts && ends;
        q.starts = starts;
        q.n = 0;
        q.hi = 0;
        q.key0 = lo;
        if (q.rows > 0) {  // this member's own range, in the unit's blocks
            int my_lo, x0;
            visible(s.pos0 + q.row0 / p.G, s.len, p.causal, p.window, my_lo, x0);
            visible(s.pos0 + (q.row0 + q.rows - 1) / p.G, s.len, p.causal, p.window, x0, q.hi);
            if (q.hi > my_lo) {
                const int j0 = max(b0, (my_lo - lo) >> p.log2_kb), j1 = min(b1, (q.hi - lo + p.KB - 1) >> p.log2_kb);
                q.n = max(0, j1 - j0);
                q.key0 = lo + j0 * p.KB;
            }
        }
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
    Piece* joins;            // [grid], block kernel
    float* parts;            // [2 n_ctas][R][HD] then [2 n_ctas][R][2]
    int n_ctas;
};

// Capped scores, log2(e) cap tanh(s / cap), from x = log2(e) s and u = s / cap.
// tanh u = u + u^3 P(u^2) for |u| <= 0.6 (a least-squares fit of four terms over
// that range, reweighted towards equal errors: 3e-8 off): scores are mostly far
// below the cap, and this needs no exponential or division, whose unit the softmax
// already fills.
constexpr float kTanhSmall = 0.6f;
__device__ constexpr float kTanhCoef[4] = {-0.333322137594223f, 0.13307641446590424f, -0.05197533965110779f,
                                           0.015294312499463558f};
__device__ __forceinline__ float capped_small(float x, float u) {
    const float z = u * u;
    float p = kTanhCoef[3];
#pragma unroll
    for (int i = 2; i >= 0; --i) p = fmaf(p, z, kTanhCoef[i]);
    return fmaf(x * z, p, x);
}
// any u: tanh u = 1 - 2 / (1 + e^2u); cap2 = log2(e) cap
__device__ __forceinline__ float capped_any(float u, float cap2) {
    return cap2 * (1.f - __fdividef(2.f, 1.f + exp2f(u * (2.f * kLog2e))));
}

// Four columns of a row: v / l (times the values' scale) rounded to the output
// type; the row's log-sum-exp goes with column 0.  l = 0: no key seen.
__device__ __forceinline__ void store4(const AttendArgs& a, const Piece& t, bool bf, float vscale, int r, int col,
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
// slot 2 c the one that continues it there.  O is relative to 2^m, not divided by l;
// a piece that saw no key has m = -inf, l = 0 and no O.
__device__ __forceinline__ float* part_o(const AttendArgs& a, int hd, size_t slot, int r) {
    return a.parts + (slot * a.p.R + r) * hd;
}
__device__ __forceinline__ float* part_ml(const AttendArgs& a, int hd, size_t slot, int r) {
    return a.parts + 2 * static_cast<size_t>(a.n_ctas) * a.p.R * hd + (slot * a.p.R + r) * 2;
}

// Adds the pieces of rows [r_begin, r_end) of a unit cut over teams t_first ..
// t_last, in that order, by `threads` threads; all pieces are in memory.
template <int HD>
__device__ __forceinline__ void join_pieces(const AttendArgs& a, const Piece& t, int member, bool bf, float vscale,
                                            int r_begin, int r_end, int tid, int threads) {
    for (int i = r_begin * (HD / 4) + tid; i < r_end * (HD / 4); i += threads) {
        const int r = i / (HD / 4), col = (i % (HD / 4)) * 4;
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = t.t_first; k <= t.t_last; ++k) {
            const size_t slot = 2 * static_cast<size_t>(k * a.p.TS + member) + (k == t.t_first ? 1 : 0);
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml(a, HD, slot, r)));
            float4 x = __ldcg(reinterpret_cast<const float4*>(part_o(a, HD, slot, r) + col));
            if (ml.x == -INFINITY && ml.y == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);
            const float mn = fmaxf(m, ml.x);
            // (a piece without a maximum holds nothing, or NaN from NaN scores alone)
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
