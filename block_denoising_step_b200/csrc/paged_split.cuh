// Attention of a few query rows per KV head over the paged cache (a sequence's
// next token, a handful of tokens, or any count where the tcgen05 kernel of
// paged_block.cuh does not apply).
//
//   o = sum_j softmax_j(f(scale q . k_j)) v_j,  f(s) = cap tanh(s / cap) or s
//
// One pass over the keys with a running maximum m and sum l per row.  The
// G query heads of a KV head (times the new tokens) are the rows; they fill the
// N side (8 per tile) of mma.sync m16n8k16 and the keys the M side, so one token
// of a group of up to 8 heads wastes nothing that matters: S^T = K Q^T
// (16 keys x 8 rows per instruction), O^T += V^T P^T.  P^T's operand layout is
// S^T's accumulator layout transposed 8 x 8 (movmatrix).  P is kept as hi + lo
// 16-bit parts (about 16 significant bits, fp16's down to 2^-16 of the largest weight), so the
// output's own rounding is the only one that shows; with an E4M3 cache and bf16 rows fp16's 11
// bits alone do (2^-11 of a weight against the output's 2^-8).
//
// Memory-bound: every visible K and V row is read once.  Each warp streams its
// own tiles of 16 or 32 keys through a private ring of shared memory (cp.async 16 bytes,
// XOR-swizzled by row; no block barrier in the loop); the page of each row is
// looked up per key, one tile ahead, so a page may end anywhere in a tile.  Rows
// outside the sequence's visible range or without a page are filled with zeros
// and masked: nothing behind a sequence's end is read.
//
// E4M3 caches: bytes are widened to fp16 (exact) in registers; queries are
// scaled by a power of two per row to the top of fp16's range; the head's scales enter
// the score factor and the output.  A pair of ldmatrix b16 lanes holds four
// bytes, so the k order within 16 elements is permuted alike in K and Q.
//
// Measured on a B200 (device time of a replayed graph): 131,071 keys of 8 heads x 128 for
// one token 89 us (6.0 TB/s); 64 tokens over up to 8,192 keys of 8 x 256 326 us (6.8 TB/s);
// 48 tokens over up to 16,384 E4M3 keys of 8 x 128 188 to 191 us (4.3 TB/s: the conversions bound it);
// 128 tokens in windows of 1,024 keys of 12 x 64 74 us (4.8 TB/s: the start and end of short
// units); one token over 301 keys 8.9 us (the chain of dependent loads and the join).
#pragma once

#include "mma_sync.cuh"
#include "paged_work.cuh"

namespace dgen {
namespace paged {

constexpr int kSplitWarps = 4;

template <int HD, int ES, int NT>
struct SplitLayout {
    static constexpr int ROWB = HD * ES;        // bytes of a cache row
    static constexpr int CH = ROWB / 16;        // 16-byte chunks of a row
    // 16-key steps per warp tile
    static constexpr int MT = NT == 1 && ROWB <= 128 ? 2 : 1;
    // CTAs per SM: short rows need more warps than long ones to keep as many bytes in flight, and a tile's chain
    // of dependent steps (scores, maximum, weights, products) overlapped
    static constexpr int CTAS = ROWB <= 128 ? (NT == 4 ? 2 : 3) : ROWB == 256 ? 2 : 1;
    static constexpr int KEYS = 16 * MT;                      // keys per warp tile
    static constexpr int BLOCK_KEYS = kSplitWarps * KEYS;     // keys per block of the line
    static constexpr int TILE = KEYS * ROWB;
    static constexpr int STAGES = NT == 1 && ROWB == 128 ? 2 : 3;
    static constexpr int RING = kSplitWarps * STAGES * 2 * TILE;
};
template <int HD, int ES, int NT>
struct SplitSmem {
    using L = SplitLayout<HD, ES, NT>;
    static constexpr int R = 8 * NT;
    static constexpr int OP = HD + 4;  // padded row of the join buffers
    static constexpr int JOIN = kSplitWarps / 2 * R * OP * 4;
    static constexpr int REST = 2 * R * HD * 2 + 2 * R * 4 + 2 * kSplitWarps * R * 4 + kSplitWarps * L::STAGES * 4 + 16 +
                                2 * 64 + 32 * static_cast<int>(sizeof(Walk));
    // The next unit's first tiles are fetched before the current one is joined, where a join buffer beside the
    // ring costs no CTA of the SM (227 KB, 1 KB each); else the join uses the ring's memory.
    static constexpr bool EARLY = L::RING + JOIN + REST <= 227 * 1024 / L::CTAS - 1024;
    static constexpr int JOIN_OFF = EARLY ? L::RING : 0;
    static constexpr int Q_OFF = EARLY ? L::RING + JOIN : (L::RING > JOIN ? L::RING : JOIN);
    static constexpr int Q_BYTES = R * HD * 2;                    // two in turn
    static constexpr int QS_OFF = Q_OFF + 2 * Q_BYTES;            // float qscale[2][R]
    static constexpr int ML_OFF = QS_OFF + 2 * R * 4;             // float m[W][R], l[W][R]
    static constexpr int MASK_OFF = ML_OFF + 2 * kSplitWarps * R * 4;  // uint32 mask[W][STAGES]
    static constexpr int FLAG_OFF = MASK_OFF + kSplitWarps * L::STAGES * 4;
    static constexpr int PIECE_OFF = FLAG_OFF + 16;                     // the current piece and the next
    static constexpr int WALK_OFF = PIECE_OFF + 2 * 64;                 // Walk[32]: warp 0's, a lane each
    static constexpr int BYTES = (WALK_OFF + 32 * static_cast<int>(sizeof(Walk)) + 15) & ~15;
    static_assert(BYTES <= 227 * 1024, "shared memory");
};

// chunk position of chunk c in row r: eight rows of one chunk column fall into
// eight different 16-byte bank groups
template <int CH>
__device__ __forceinline__ int swz_chunk(int r, int c) {
    return CH >= 8 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <bool BF>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        attn::mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two E4M3 bytes (low half of v) -> two fp16 values, exact
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// old value of *p, which goes on to old + 1, from `last` to 0
__device__ __forceinline__ unsigned inc_acq_rel(unsigned* p, unsigned last) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(last) : "memory");
    return old;
}

// HD: head size.  ES: bytes of a cache element.  BF: the products run in bf16
// (else fp16; always fp16 for E4M3 caches).  NT: tiles of 8 query rows.
template <int HD, int ES, bool BF, int NT>
__global__ void __launch_bounds__(kSplitWarps * 32, SplitLayout<HD, ES, NT>::CTAS) paged_split_kernel(const AttendArgs a) {
    using L = SplitLayout<HD, ES, NT>;
    using S = SplitSmem<HD, ES, NT>;
    using H2 = Half2<BF>;
    constexpr int R = S::R, CH = L::CH, ST = L::STAGES, QCH = HD / 8, MT = L::MT, KEYS = L::KEYS;
    constexpr float LIFT = BF ? 0.f : kHalfLift;
    constexpr uint32_t kAllKeys = KEYS == 32 ? 0xFFFFFFFFu : (1u << KEYS) - 1u;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t sbase = smem_u32(smem), ring = sbase + warp * (ST * 2 * L::TILE);
    float* s_m = reinterpret_cast<float*>(smem + S::ML_OFF);
    float* s_l = s_m + kSplitWarps * R;
    uint32_t* s_mask = reinterpret_cast<uint32_t*>(smem + S::MASK_OFF) + warp * ST;
    int* s_flag = reinterpret_cast<int*>(smem + S::FLAG_OFF);
    float* join = reinterpret_cast<float*>(smem + S::JOIN_OFF);

    pdl_enter();
    const CacheView& c = a.c;
    static_assert(sizeof(Piece) <= 64, "piece slot");
    auto slot_of = [&](int i) { return reinterpret_cast<Piece*>(smem + S::PIECE_OFF + i * 64); };
    // warp 0 walks the units; its state waits in shared memory, not in the registers of the key loop
    auto walk_on = [&](int i) {
        const volatile Walk& seen = reinterpret_cast<Walk*>(smem + S::WALK_OFF)[lane];
        if (seen.t >= seen.t_end) {
            if (lane == 0) slot_of(i)->end = 1;
            return;
        }
        Walk walk = reinterpret_cast<Walk*>(smem + S::WALK_OFF)[lane];
        Piece q{};
        q.end = !walk.next(c, a.p, lane, q);
        reinterpret_cast<Walk*>(smem + S::WALK_OFF)[lane] = walk;
        if (lane == 0) *slot_of(i) = q;
    };

    // Fetching: rows of this warp's next tile; the table entry is loaded one tile ahead.
    int key_next = 0, pg_next = 0, id_next = -1;
    const uint8_t *k_lane = c.k + lane % CH * 16, *v_lane = c.v + lane % CH * 16;
    static_assert(CH <= 32 && 32 % CH == 0, "a lane copies the same chunk of every row");
    auto fetch = [&](const Piece& p, int stage, bool live) {
        uint32_t row = kNoRow;
        if (live && key_next < p.hi) row = row_in_page(c, id_next, p.h, key_next - pg_next * c.page);
        key_next += L::BLOCK_KEYS;
        pg_next = c.page_of(key_next);
        id_next = live && key_next < p.hi ? page_entry(c, p.b, pg_next) : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, row != kNoRow) & kAllKeys;
        if (lane == 0) s_mask[stage] = mask;
        if (mask != 0) {
            const uint32_t dk = ring + stage * (2 * L::TILE), dv = dk + L::TILE;
#pragma unroll
            for (int i = 0; i < KEYS * CH / 32; ++i) {
                const int r = i * (32 / CH) + lane / CH;
                const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                const bool ok = src != kNoRow;
                const uint64_t off = static_cast<uint64_t>(ok ? src : 0u) * L::ROWB;
                const uint32_t d = r * L::ROWB + swz_chunk<CH>(r, lane % CH) * 16;
                attn::cp_async16(dk + d, k_lane + off, ok);
                attn::cp_async16(dv + d, v_lane + off, ok);
            }
        }
        attn::cp_commit();
    };
    // The first tiles of a piece, and its queries into Q buffer i, one warp per row.
    auto begin = [&](const Piece& p, int i) {
        key_next = p.key0 + warp * KEYS + (lane & (KEYS - 1));
        pg_next = c.page_of(key_next);
        id_next = key_next < p.hi ? page_entry(c, p.b, pg_next) : -1;
#pragma unroll
        for (int e = 0; e < ST - 1; ++e) fetch(p, e, e < p.n);
        float* qscale = reinterpret_cast<float*>(smem + S::QS_OFF) + i * R;
        for (int r = warp; r < R; r += kSplitWarps) {
            constexpr int PER = HD / 32;  // elements per lane: 2, 4 or 8
            uint32_t w[PER / 2];
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) w[e] = 0;
            if (r < p.rows) {
                const int tok = p.first + (p.row0 + r) / a.p.G, head = p.h * a.p.G + (p.row0 + r) % a.p.G;
                const uint8_t* src = a.q.p + (tok * a.q.ts + head * a.q.hs + lane * PER) * 2;
                if constexpr (PER == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                } else if constexpr (PER == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    w[0] = v.x, w[1] = v.y;
                } else {
                    w[0] = *reinterpret_cast<const uint32_t*>(src);
                }
            }
            if constexpr (ES == 2) {
                if (lane == 0) qscale[r] = 1.f;
            } else {  // power-of-two scale into fp16's range, bf16 or fp16 in
                float2 x[PER / 2];
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < PER / 2; ++e) {
                    x[e] = a.q_bf16 ? Half2<true>::unpack(w[e]) : Half2<false>::unpack(w[e]);
                    m = fmaxf(m, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                // the largest element goes to [2^14, 2^15), so that elements down to 2^-28 of it are normal numbers
                // (the products' sum stays in fp32: 2^15 * 448 * 256 < 2^33)
                int ex = 0;
                if (m > 0.f && m < INFINITY) frexpf(m, &ex);
                ex = max(ex, -112) - 15;  // (2^-ex is a number of fp32)
                const float down = ldexpf(1.f, -ex);
#pragma unroll
                for (int e = 0; e < PER / 2; ++e) w[e] = Half2<false>::pack(x[e].x * down, x[e].y * down);
                if (lane == 0) qscale[r] = ldexpf(1.f, ex);
            }
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) {
                int el = lane * PER + 2 * e;  // element pair el, el + 1
                if constexpr (ES == 1) {
                    // memory element 4t + 2j + i of a 16-block sits at k = 8j + 2t + i
                    const int blk = el & ~15, x = el & 15;
                    el = blk + ((x >> 1) & 1) * 8 + (x >> 2) * 2;
                }
                const int ch = el >> 3;
                *reinterpret_cast<uint32_t*>(smem + S::Q_OFF + i * S::Q_BYTES + r * (HD * 2) +
                                             swz_chunk<QCH>(r, ch) * 16 + (el & 7) * 2) = w[e];
            }
        }
    };

    if (warp == 0) {
        Walk walk;
        walk.start(c, a.p, lane, blockIdx.x, a.n_ctas);
        reinterpret_cast<Walk*>(smem + S::WALK_OFF)[lane] = walk;
        walk_on(0);
    }
    __syncthreads();
    Piece s = *slot_of(0);
    if (!s.end) begin(s, 0);
    for (int cur = 0; !s.end; cur ^= 1) {
        if (warp == 0) walk_on(cur ^ 1);
        const int h = s.h, row0 = s.row0, rows = s.rows;
        const int key_first = s.key0 + warp * KEYS;
        const int n_tiles = s.n;
        const uint32_t sq = sbase + S::Q_OFF + cur * S::Q_BYTES;
        const float* qscale = reinterpret_cast<const float*>(smem + S::QS_OFF) + cur * R;

        // visible range and score factor of this thread's rows (columns 2 t4, 2 t4 + 1 of each tile)
        int vlo[NT][2], vhi[NT][2];
        int all_lo = 0, all_hi = s.hi;  // keys every row of the tile sees
        {
            int lo_l, hi_f, dummy;
            visible(s.pos0 + row0 / a.p.G, s.len, a.p.causal, a.p.window, dummy, hi_f);
            visible(s.pos0 + (row0 + rows - 1) / a.p.G, s.len, a.p.causal, a.p.window, lo_l, dummy);
            all_lo = lo_l;
            all_hi = hi_f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = min(nt * 8 + 2 * t4 + j, rows - 1);
                visible(s.pos0 + (row0 + r) / a.p.G, s.len, a.p.causal, a.p.window, vlo[nt][j], vhi[nt][j]);
            }
        __syncthreads();  // queries and the next piece are there, the join's memory is free
        const float kscale = ES == 1 ? __ldg(c.k_scale + h) : 1.f;
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // (the scale first with the query's own, whose product is of the order of one)
                const float f = a.scale * (ES == 1 ? qscale[nt * 8 + 2 * t4 + j] : 1.f) * kscale;
                fac[nt][j] = f * kLog2e;
            }
        const float inv_cap = a.cap > 0.f ? kLn2 / a.cap : 0.f;  // of a log2-domain score

        // one tile of rows: its queries' operands stay in registers
        uint32_t qf[NT == 1 ? HD / 32 : 1][4];
        if constexpr (NT == 1) {
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk)
                attn::ldsm_x4(sq + (lane & 7) * (HD * 2) + swz_chunk<QCH>(lane & 7, 4 * kk + (lane >> 3)) * 16, qf[kk][0],
                              qf[kk][1], qf[kk][2], qf[kk][3]);
        }

        float o[HD / 16][NT][4];
        float m_run[NT][2], l_run[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m_run[nt][0] = m_run[nt][1] = -INFINITY;
            l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < HD / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
        }

        for (int i = 0; i < n_tiles; ++i) {
            attn::cp_wait<ST - 2>();
            __syncwarp();
            const int stage = i % ST;
            const uint32_t mask = s_mask[stage];
            const int key0 = key_first + i * L::BLOCK_KEYS;
            if (mask != 0) {  // (warp-uniform)
                const uint32_t tk = ring + stage * (2 * L::TILE), tv = tk + L::TILE;
                // (two accumulators each: products on one wait for each other)
                float sc[MT][NT][4], sd[MT][NT][4];
#pragma unroll
                for (int km = 0; km < MT; ++km)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[km][nt][e] = sd[km][nt][e] = 0.f;
                // S^T = K Q^T, 32 elements of hd per step
#pragma unroll
                for (int kk = 0; kk < HD / 32; ++kk) {
                    uint32_t b[NT][4];  // k 0-7, 8-15, 16-23, 24-31 of query rows nt * 8 ..
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (NT == 1) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[nt][e] = qf[kk][e];
                            continue;
                        }
                        const int qr = nt * 8 + (lane & 7);
                        attn::ldsm_x4(sq + qr * (HD * 2) + swz_chunk<QCH>(qr, 4 * kk + (lane >> 3)) * 16, b[nt][0],
                                      b[nt][1], b[nt][2], b[nt][3]);
                    }
#pragma unroll
                    for (int km = 0; km < MT; ++km) {
                        uint32_t ka[2][4];
                        const int r = km * 16 + (lane & 15);
                        if constexpr (ES == 2) {
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                attn::ldsm_x4(tk + r * L::ROWB + swz_chunk<CH>(r, 4 * kk + 2 * u + (lane >> 4)) * 16,
                                              ka[u][0], ka[u][1], ka[u][2], ka[u][3]);
                        } else {
                            uint32_t x[4];  // keys 0-7 / 8-15 of the first 16 bytes, then of the second
                            attn::ldsm_x4(tk + r * L::ROWB + swz_chunk<CH>(r, 2 * kk + (lane >> 4)) * 16, x[0], x[1],
                                          x[2], x[3]);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const uint32_t v = x[2 * u + half];
                                    ka[u][half] = e4m3x2_f16x2(static_cast<uint16_t>(v));
                                    ka[u][2 + half] = e4m3x2_f16x2(static_cast<uint16_t>(v >> 16));
                                }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816<BF>(sc[km][nt], ka[0], b[nt][0], b[nt][1]);
                            mma_16816<BF>(sd[km][nt], ka[1], b[nt][2], b[nt][3]);
                        }
                    }
                }
#pragma unroll
                for (int km = 0; km < MT; ++km)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[km][nt][e] += sd[km][nt][e];
                // log2-domain scores, masks, running maximum
                if (a.cap > 0.f) {
                    bool small = true;
#pragma unroll
                    for (int km = 0; km < MT; ++km)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                small &= fabsf(sc[km][nt][e] * fac[nt][e & 1] * inv_cap) <= kTanhSmall;
                    if (__all_sync(0xffffffffu, small)) {
#pragma unroll
                        for (int km = 0; km < MT; ++km)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float x = sc[km][nt][e] * fac[nt][e & 1];
                                    sc[km][nt][e] = capped_small(x, x * inv_cap);
                                }
                    } else {
#pragma unroll
                        for (int km = 0; km < MT; ++km)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    sc[km][nt][e] =
                                        capped_any(sc[km][nt][e] * fac[nt][e & 1] * inv_cap, kLog2e * a.cap);
                    }
                } else {
#pragma unroll
                    for (int km = 0; km < MT; ++km)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sc[km][nt][e] *= fac[nt][e & 1];
                }
                if (!(mask == kAllKeys && key0 >= all_lo && key0 + KEYS <= all_hi)) {
#pragma unroll
                    for (int km = 0; km < MT; ++km)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int kr = km * 16 + g + 8 * (e >> 1), key = key0 + kr;
                                if (!((mask >> kr) & 1u) || key < vlo[nt][e & 1] || key >= vhi[nt][e & 1])
                                    sc[km][nt][e] = -INFINITY;
                            }
                }
                bool move = false;
                float top[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float mx = fmaxf(sc[0][nt][j], sc[0][nt][2 + j]);
#pragma unroll
                        for (int km = 1; km < MT; ++km) mx = fmaxf(mx, fmaxf(sc[km][nt][j], sc[km][nt][2 + j]));
#pragma unroll
                        for (int w = 4; w <= 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                        top[nt][j] = mx;
                        move |= mx > m_run[nt][j] + kRescale || (m_run[nt][j] == -INFINITY && mx > -INFINITY);
                    }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float corr[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float mn = fmaxf(m_run[nt][j], top[nt][j]);
                            corr[j] = m_run[nt][j] == -INFINITY ? 0.f : ex2(m_run[nt][j] - mn);
                            m_run[nt][j] = mn;
                            l_run[nt][j] *= corr[j];
                        }
#pragma unroll
                        for (int mt = 0; mt < HD / 16; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[mt][nt][e] *= corr[e & 1];
                    }
                }
                uint32_t ph[MT][NT][2], pl[MT][NT][2];
                const bool low = ES == 2 || !a.q_bf16;
#pragma unroll
                for (int km = 0; km < MT; ++km)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float mu = m_run[nt][e & 1] == -INFINITY ? 0.f : m_run[nt][e & 1] - LIFT;
                            p[e] = ex2(sc[km][nt][e] - mu);
                            l_run[nt][e & 1] += p[e];
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t hi = H2::pack(p[2 * half], p[2 * half + 1]);
                            const float2 hf = H2::unpack(hi);
                            ph[km][nt][half] = movmatrix_t(hi);
                            if (low) pl[km][nt][half] = movmatrix_t(H2::pack(p[2 * half] - hf.x, p[2 * half + 1] - hf.y));
                        }
                    }
                // O^T += V^T P^T, four (two) rows of tiles at a time, all their hi parts before the lo parts
                const int vc = (lane >> 3) & 1;
                constexpr int GM = HD == 256 || NT > 1 ? 2 : 4;
#pragma unroll
                for (int km = 0; km < MT; ++km) {
                    const int vr = km * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                    for (int m0 = 0; m0 < HD / 16; m0 += GM) {
                        uint32_t va[GM][4];
                        if constexpr (ES == 2) {
#pragma unroll
                            for (int i = 0; i < GM; ++i)
                                attn::ldsm_x4_t(tv + vr * L::ROWB + swz_chunk<CH>(vr, 2 * (m0 + i) + vc) * 16, va[i][0],
                                                va[i][1], va[i][2], va[i][3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < GM; i += 2) {
                                uint32_t x[4];  // two 16-byte columns x keys 0-7, then keys 8-15
                                attn::ldsm_x4_t(tv + vr * L::ROWB + swz_chunk<CH>(vr, m0 + i + vc) * 16, x[0], x[1],
                                                x[2], x[3]);
#pragma unroll
                                for (int u = 0; u < 2; ++u)
#pragma unroll
                                    for (int half = 0; half < 2; ++half) {
                                        // bytes 2g, 2g + 1 of key 2t, then of key 2t + 1: rows g and g + 8
                                        const uint32_t v = __byte_perm(x[2 * half + u], 0, 0x3120);
                                        va[i + u][2 * half] = e4m3x2_f16x2(static_cast<uint16_t>(v));
                                        va[i + u][2 * half + 1] = e4m3x2_f16x2(static_cast<uint16_t>(v >> 16));
                                    }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < GM; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816<BF>(o[m0 + i][nt], va[i], ph[km][nt][0], ph[km][nt][1]);
                        if (low) {
#pragma unroll
                            for (int i = 0; i < GM; ++i)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_16816<BF>(o[m0 + i][nt], va[i], pl[km][nt][0], pl[km][nt][1]);
                        }
                    }
                }
            }
            __syncwarp();  // every lane has read stage `stage` and its mask
            fetch(s, (i + ST - 1) % ST, i + ST - 1 < n_tiles);
        }
        attn::cp_wait<0>();
        const Piece following = *slot_of(cur ^ 1);
        if (S::EARLY && !following.end) begin(following, cur ^ 1);

        // join the four warps: m and l, then O scaled to the common m: two warps' in memory, on which the other
        // two add
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int w = 4; w <= 16; w <<= 1) l_run[nt][j] += __shfl_xor_sync(0xffffffffu, l_run[nt][j], w);
                if (g == 0) {
                    s_m[warp * R + nt * 8 + 2 * t4 + j] = m_run[nt][j];
                    s_l[warp * R + nt * 8 + 2 * t4 + j] = l_run[nt][j];
                }
            }
        __syncthreads();
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            if ((warp >> 1) != pass) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = nt * 8 + 2 * t4 + j;
                        const float f = m_run[nt][j] == -INFINITY
                                            ? 0.f
                                            : exp2f(m_run[nt][j] - fmaxf(fmaxf(s_m[r], s_m[R + r]),
                                                                         fmaxf(s_m[2 * R + r], s_m[3 * R + r])));
#pragma unroll
                        for (int mt = 0; mt < HD / 16; ++mt)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int col = ES == 2 ? mt * 16 + g + 8 * half : mt * 16 + 2 * g + half;
                                float& to = join[((warp & 1) * R + r) * S::OP + col];
                                const float v = o[mt][nt][2 * half + j] * f;
                                to = pass == 0 ? v : to + v;
                            }
                    }
            }
            __syncthreads();
        }
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s.starts ? 1 : 0);
        const bool out_bf = ES == 2 ? BF : a.q_bf16 != 0;
        const float vscale = ES == 1 ? __ldg(c.v_scale + h) : 1.f;
        for (int i = threadIdx.x; i < rows * (HD / 4); i += kSplitWarps * 32) {
            const int r = i / (HD / 4), col = (i % (HD / 4)) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const float m = fmaxf(fmaxf(s_m[r], s_m[R + r]), fmaxf(s_m[2 * R + r], s_m[3 * R + r]));
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(join + (w * R + r) * S::OP + col);
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
#pragma unroll
            for (int w = 0; w < kSplitWarps; ++w) {
                // (a warp without a maximum has l = 0, or NaN from NaN scores)
                l += s_l[w * R + r] * (s_m[w * R + r] == -INFINITY ? 1.f : exp2f(s_m[w * R + r] - m));
            }
            if (s.whole) {
                store4(a, s, out_bf, vscale, r, col, v, m - LIFT, l);
            } else {
                __stcg(reinterpret_cast<float4*>(part_o(a, HD, slot, r) + col), v);
                if (col == 0) __stcg(reinterpret_cast<float2*>(part_ml(a, HD, slot, r)), make_float2(m - LIFT, l));
            }
        }
        if (!s.whole) {
            // (the barrier orders all threads' stores before thread 0's release, and its acquire before their loads)
            const unsigned last = s.t_last - s.t_first;
            __syncthreads();
            if (threadIdx.x == 0) *s_flag = inc_acq_rel(a.counters + s.t_first, last) == last;
            __syncthreads();
            if (*s_flag) {  // every piece of this unit is in memory; the counter is back at zero
                join_pieces<HD>(a, s, 0, out_bf, vscale, 0, rows, threadIdx.x, kSplitWarps * 32);
            }
        }
        if (!S::EARLY && !following.end) {
            __syncthreads();  // the join's memory is the ring's
            begin(following, cur ^ 1);
        }
        s = following;
    }
}

}  // namespace paged
}  // namespace dgen
