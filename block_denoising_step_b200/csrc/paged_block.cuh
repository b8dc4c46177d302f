// Attention of many query rows per KV head over the paged cache (a canvas over
// its prompt, a chunk of a prompt) on the 5th-generation tensor cores.
//
// The same formula and masks as paged_split.cuh.  The rows of a tile are the
// tokens times the G query heads of one KV head (row = token * G + head), up to
// 128, so K and V are read once for the whole group.  One CTA per SM walks the
// units of paged_work.cuh in blocks of 128 keys:
//
//   warp 0           producer: Q by one TMA box per 64 columns ([tokens][G] rows),
//                    K and V in stages of 128 keys x SC columns (32 KB), one TMA box
//                    per page part (BR rows, a power of two that divides the page
//                    size) and 64 columns, each lane issuing its own box;
//   warp 1           MMA issuer: S = Q K^T (128 x 128 fp32) into one of two TMEM
//                    buffers, O += P V with P from tensor memory (the low 64 columns
//                    of its S buffer) and V MN-major from shared memory;
//   4 or 8 warps     softmax: thread = query row.  One warpgroup takes every
//                    tile at hd 256, where O fills half the tensor memory and the
//                    products take longer than the exponentials; at hd <= 128 two
//                    warpgroups take alternate tiles with an O, m and l each, joined
//                    at the unit's end.
//
// Order of the products: S0, S1, P0 V0, S2, P1 V1, S3, ...: the softmax of one
// tile runs beside the products of its neighbours.  Tiles of 128 keys, because
// S = Q K^T with N = 64 would read 6 KB of operands per 32 cycles, more than shared
// memory delivers; with N = 128 it is 8 KB per 64.
// P is rounded once to the operand type (bf16 / fp16): hi + lo parts as in the
// split kernel would add half as many products again.  Its error is that of one
// rounding per weight, averaged over the keys, below the output's own rounding.
//
// Keys behind the sequence's end and absent pages are not loaded; scores there
// are replaced by -inf, and the V rows are zeroed before use (shared memory may
// hold anything).  Every wait is bounded; on a timeout the kernel records an
// error, drains its own copies and MMAs, frees its tensor memory and exits.
#pragma once

#include "paged_work.cuh"

namespace dgen {
namespace paged {

enum : int { ERR_BLOCK_PRODUCER = 20, ERR_BLOCK_MMA = 21, ERR_BLOCK_SOFTMAX = 22, ERR_BLOCK_DRAIN = 23 };

constexpr int kBlkKeys = 128;
constexpr int kBlkRows = 128;

template <int HD>
struct BlockLayout {
    static constexpr int SC = HD < 128 ? HD : 128;    // columns of a stage
    static constexpr int NS = HD / SC;                // stages per K or V tile
    static constexpr int NG = HD == 256 ? 1 : 2;      // softmax warpgroups
    static constexpr int THREADS = 64 + NG * 128;
    static constexpr int Q_BYTES = kBlkRows * HD * 2; // HD / 64 boxes of [128 rows x 128 B]
    static constexpr int STAGE = kBlkKeys * SC * 2;   // SC / 64 boxes of [128 rows x 128 B]
    static constexpr int STAGES = HD == 256 ? 5 : (HD == 128 ? 5 : 8);
    static constexpr int KV_OFF = Q_BYTES;
    static constexpr int ML_OFF = KV_OFF + STAGES * STAGE;           // float2 ml[NG][128]
    static constexpr int BAR_OFF = ML_OFF + NG * kBlkRows * 8;
    // q_full, q_empty, kv_full[ST], kv_empty[ST], s_full[2], p_full[2], pv_done[2], o_free, drain
    static constexpr int N_BARS = 2 + 2 * STAGES + 6 + 2;
    static constexpr int SLOT_OFF = BAR_OFF + N_BARS * 8;            // TMEM base, join flag
    static constexpr int SMEM_BYTES = SLOT_OFF + 16 + 1024;          // + slack for 1024-byte alignment
    static constexpr int T_S = NG * HD;                              // first S column
    static_assert(T_S + 2 * kBlkKeys <= 512, "tensor memory");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// D (TMEM) (+)= A (TMEM, K-major, two 16-bit values per column) x B (shared-memory descriptor)
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// bits [lo, hi) of a 32-bit word whose bit 0 is position `base`
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int base) {
    const int a = min(max(lo - base, 0), 32), b = min(max(hi - base, 0), 32);
    const uint32_t up = b >= 32 ? 0xFFFFFFFFu : (1u << b) - 1u, dn = a >= 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
    return up & ~dn;
}

// Page parts of a tile of 128 keys: lane i < nbox holds the cache row of part i
// (kNoRow: absent or behind hi).  The table entry is loaded one tile ahead.
struct Parts {
    int key, id;
    __device__ __forceinline__ void ahead(const CacheView& c, int b, int key_, int hi, int nbox, int lane) {
        key = key_;
        id = lane < nbox && key < hi ? page_entry(c, b, key / c.page) : -1;
    }
    __device__ __forceinline__ uint32_t row(const CacheView& c, int h) const {
        return id >= 0 ? row_in_page(c, id, h, key % c.page) : kNoRow;
    }
};

template <int HD, bool BF>
__global__ void __launch_bounds__(BlockLayout<HD>::THREADS, 1)
    paged_block_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const AttendArgs a, int log2_br, int* __restrict__ err) {
    using L = BlockLayout<HD>;
    using H2 = Half2<BF>;
    constexpr int NG = L::NG, ST = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem), sQ = sbase, sKV = sbase + L::KV_OFF;
    float2* s_ml = reinterpret_cast<float2*>(smem + L::ML_OFF);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t *q_full = bars, *q_empty = bars + 1, *kv_full = bars + 2, *kv_empty = kv_full + ST;
    uint64_t *s_full = kv_empty + ST, *p_full = s_full + 2, *pv_done = p_full + 2, *o_free = pv_done + 2,
             *drain = o_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    int* s_flag = reinterpret_cast<int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(o_free, 4 * NG);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_enter();
    const uint32_t tmem = *tmem_slot, t_s = tmem + L::T_S;
    const CacheView& c = a.c;
    const int br = 1 << log2_br, nbox = kBlkKeys >> log2_br;

    Walk walk;
    walk.start(c, a.p, lane, a.min_blocks);
    SeqInfo s;
    int unit, b0, b1;
    long long u0;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
        }
        int st = 0, unit_no = 0;
        uint32_t ph = 0, pending = 0, fill_ph = 0;
        bool ok = true;
        int q_phase = -1;  // parity of the last Q copy issued
        auto fetch = [&](const CUtensorMap* m, uint32_t row) {  // one K or V tile
            const uint32_t have = __ballot_sync(0xffffffffu, row != kNoRow);
#pragma unroll
            for (int n = 0; n < L::NS; ++n) {
                if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[st], ph ^ 1u, err, ERR_BLOCK_PRODUCER))) {
                    ok = false;
                    return;
                }
                if (lane == 0) mbar_expect_tx(&kv_full[st], __popc(have) * br * 128 * (L::SC / 64));
                __syncwarp();
                if (row != kNoRow) {
                    const uint32_t dst = sKV + st * L::STAGE + lane * br * 128;
#pragma unroll
                    for (int x = 0; x < L::SC / 64; ++x)
                        tma_load_2d(dst + x * (kBlkKeys * 128), m, n * L::SC + x * 64, static_cast<int>(row),
                                    smem_u32(&kv_full[st]));
                }
                pending |= 1u << st;
                fill_ph = (fill_ph & ~(1u << st)) | (ph << st);
                if (++st == ST) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        };
        while (ok && walk.next(c, a.p, lane, s, unit, b0, b1, u0)) {
            const int h = unit / s.tiles, rt = unit % s.tiles, n = b1 - b0;
            const int key0 = s.lo + b0 * kBlkKeys + lane * br;
            if (unit_no > 0 &&
                !__all_sync(0xffffffffu, mbar_wait(q_empty, (unit_no - 1) & 1, err, ERR_BLOCK_PRODUCER))) {
                ok = false;
                break;
            }
            if (lane == 0) {
                const int tok = s.first + rt * (a.p.R / a.p.G);
                mbar_expect_tx(q_full, a.p.R * HD * 2);
#pragma unroll
                for (int x = 0; x < HD / 64; ++x)
                    tma_load_3d(sQ + x * (kBlkRows * 128), &tmQ, x * 64, h * a.p.G, tok, smem_u32(q_full));
            }
            q_phase = unit_no & 1;
            Parts pk, pv;
            pk.ahead(c, s.b, key0, s.hi, nbox, lane);
            pv = pk;
            // K0, K1, V0, K2, V1, ...
            for (int j = 0; ok && j < n + 2; ++j) {
                if (j < n) {
                    const uint32_t row = pk.row(c, h);
                    if (j + 1 < n) pk.ahead(c, s.b, key0 + (j + 1) * kBlkKeys, s.hi, nbox, lane);
                    fetch(&tmK, row);
                }
                if (ok && j >= 1 && j - 1 < n) {
                    const uint32_t row = pv.row(c, h);
                    if (j < n) pv.ahead(c, s.b, key0 + j * kBlkKeys, s.hi, nbox, lane);
                    fetch(&tmV, row);
                }
            }
            ++unit_no;
        }
        // our own copies land before the CTA goes away, consumed or not
        if (q_phase >= 0) mbar_wait(q_full, q_phase, err, ERR_BLOCK_DRAIN);
        for (int i = 0; i < ST; ++i)
            if ((pending >> i) & 1u) mbar_wait(&kv_full[i], (fill_ph >> i) & 1u, err, ERR_BLOCK_DRAIN);
    } else if (warp == 1) {
        constexpr uint32_t type = BF ? (1u << 7) | (1u << 10) : 0u;  // operand types bf16 / f16
        constexpr uint32_t base = (1u << 4) | type | (static_cast<uint32_t>(kBlkRows >> 4) << 24);
        constexpr uint32_t idesc_s = base | (static_cast<uint32_t>(kBlkKeys >> 3) << 17);
        constexpr uint32_t idesc_pv = base | (1u << 16) | (static_cast<uint32_t>(L::SC >> 3) << 17);
        int st = 0, unit_no = 0, jj = 0;  // jj: tile counter of the CTA
        uint32_t ph = 0;
        bool ok = true;
        auto take = [&](int& stage) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&kv_full[st], ph, err, ERR_BLOCK_MMA))) return false;
            tc_fence_after();
            stage = st;
            if (++st == ST) {
                st = 0;
                ph ^= 1u;
            }
            return true;
        };
        while (ok && walk.next(c, a.p, lane, s, unit, b0, b1, u0)) {
            const int h = unit / s.tiles, n = b1 - b0;
            const int key0 = s.lo + b0 * kBlkKeys;
            Parts pv;
            pv.ahead(c, s.b, key0 + lane * br, s.hi, nbox, lane);
            if (!__all_sync(0xffffffffu, mbar_wait(q_full, unit_no & 1, err, ERR_BLOCK_MMA))) break;
            tc_fence_after();
            auto issue_s = [&](int j) -> bool {  // S of the unit's tile j
                const int buf = (jj + j) & 1;
#pragma unroll
                for (int x = 0; x < L::NS; ++x) {
                    int stage;
                    if (!take(stage)) return false;
                    if (lane == 0) {
                        const uint32_t sk = sKV + stage * L::STAGE;
#pragma unroll
                        for (int kk = 0; kk < L::SC / 16; ++kk) {
                            const uint64_t ad =
                                sdesc_sw128(sQ + (x * (L::SC / 64) + (kk >> 2)) * (kBlkRows * 128)) + 2 * (kk & 3);
                            const uint64_t bd = sdesc_sw128(sk + (kk >> 2) * (kBlkKeys * 128)) + 2 * (kk & 3);
                            mma_bf16_ss(t_s + buf * kBlkKeys, ad, bd, idesc_s, x > 0 || kk > 0 ? 1u : 0u);
                        }
                        mma_commit(smem_u32(&kv_empty[stage]));
                    }
                }
                if (lane == 0) {
                    mma_commit(smem_u32(&s_full[buf]));
                    if (j == n - 1) mma_commit(smem_u32(q_empty));
                }
                __syncwarp();
                return true;
            };
            ok = issue_s(0) && (n < 2 || issue_s(1));
            for (int j = 0; ok && j < n; ++j) {
                const int t = jj + j, buf = t & 1, og = NG == 2 ? buf : 0;
                const uint32_t row = pv.row(c, h);
                if (j + 1 < n) pv.ahead(c, s.b, key0 + (j + 1) * kBlkKeys + lane * br, s.hi, nbox, lane);
                const uint32_t have = __ballot_sync(0xffffffffu, row != kNoRow);
                const int live = s.hi - (key0 + j * kBlkKeys);  // rows of the tile before the end
                if (!__all_sync(0xffffffffu, mbar_wait(&p_full[buf], (t >> 1) & 1, err, ERR_BLOCK_MMA))) {
                    ok = false;
                    break;
                }
                if (j == 0 && unit_no > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(o_free, (unit_no - 1) & 1, err, ERR_BLOCK_MMA))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t tp = t_s + buf * kBlkKeys, t_o = tmem + og * HD;
                const bool first = j < NG;  // nothing in this O yet
#pragma unroll
                for (int x = 0; x < L::NS; ++x) {
                    int stage;
                    if (!take(stage)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sv = sKV + stage * L::STAGE;
                    if (live < kBlkKeys || have != (nbox == 32 ? 0xFFFFFFFFu : (1u << nbox) - 1u)) {
                        for (int r = lane; r < kBlkKeys; r += 32)
                            if (r >= live || !((have >> (r >> log2_br)) & 1u))
#pragma unroll
                                for (int e = 0; e < L::SC / 8; ++e)
                                    *reinterpret_cast<uint4*>(smem + L::KV_OFF + stage * L::STAGE +
                                                              (e >> 3) * (kBlkKeys * 128) + r * 128 + (e & 7) * 16) =
                                        make_uint4(0, 0, 0, 0);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                    if (lane == 0) {
#pragma unroll
                        for (int kk = 0; kk < kBlkKeys / 16; ++kk) {
                            const uint64_t vd = sdesc_sw128_mn(sv + kk * 2048, kBlkKeys * 128);
                            mma_ts(t_o + x * L::SC, tp + kk * 8, vd, idesc_pv, !first || kk > 0 ? 1u : 0u);
                        }
                        mma_commit(smem_u32(&kv_empty[stage]));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) mma_commit(smem_u32(&pv_done[buf]));
                __syncwarp();
                if (j + 2 < n) ok = issue_s(j + 2);
            }
            jj += n;
            ++unit_no;
        }
        if (lane == 0) {
            mma_commit(smem_u32(drain));  // arrives when every MMA issued above has completed
            mbar_wait(drain, 0, err, ERR_BLOCK_DRAIN);
        }
        __syncwarp();
    } else {
        const int grp = NG == 2 ? (warp - 2) >> 2 : 0;
        const int quarter = warp & 3;  // TMEM lanes this warp may access
        const int row = quarter * 32 + lane;
        const int tid = threadIdx.x - 64;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t t_o = tmem + (NG == 2 ? grp * HD : 0) + lane_off;
        const float fac = a.cap > 0.f ? a.scale * (2.f * kLog2e / a.cap) : a.scale * kLog2e;
        const uint32_t all_parts = (1u << nbox) - 1u;
        int jj = 0;
        bool ok = true;  // false after a wait ran out: the warp then only keeps the named barriers company
        while (walk.next(c, a.p, lane, s, unit, b0, b1, u0)) {
            const int h = unit / s.tiles, rt = unit % s.tiles, n = b1 - b0;
            const int row0 = rt * a.p.R, rows = min(a.p.R, s.n * a.p.G - row0);
            const int key0 = s.lo + b0 * kBlkKeys;
            int vlo, vhi;
            visible(s.pos0 + (row0 + min(row, rows - 1)) / a.p.G, s.len, a.p.causal, a.p.window, vlo, vhi);
            // keys every row of this warp sees (ranges only move up with the row)
            const int all_lo = __shfl_sync(0xffffffffu, vlo, 31), all_hi = __shfl_sync(0xffffffffu, vhi, 0);
            float m_run = -INFINITY, l_run = 0.f;
            // this warpgroup's tiles: those whose CTA-wide number has its parity
            int j = NG == 2 ? ((jj & 1) == grp ? 0 : 1) : 0;
            Parts pk;
            pk.ahead(c, s.b, key0 + j * kBlkKeys + lane * br, s.hi, nbox, lane);
            for (; ok && j < n; j += NG) {
                const int t = jj + j, buf = t & 1, k0 = key0 + j * kBlkKeys;
                const uint32_t have = __ballot_sync(0xffffffffu, pk.row(c, h) != kNoRow);
                if (j + NG < n) pk.ahead(c, s.b, k0 + NG * kBlkKeys + lane * br, s.hi, nbox, lane);
                const uint32_t tb = t_s + buf * kBlkKeys + lane_off;
                if (!__all_sync(0xffffffffu, mbar_wait(&s_full[buf], (t >> 1) & 1, err, ERR_BLOCK_SOFTMAX))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float x[kBlkKeys];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(tb + 32 * q, reinterpret_cast<uint32_t(&)[32]>(x[32 * q]));
                tmem_ld_wait();
                if (a.cap > 0.f) {
#pragma unroll
                    for (int e = 0; e < kBlkKeys; ++e) x[e] = capped_log2(x[e] * fac, a.cap);
                } else {
#pragma unroll
                    for (int e = 0; e < kBlkKeys; ++e) x[e] *= fac;
                }
                if (have != all_parts || k0 < all_lo || k0 + kBlkKeys > all_hi) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t bits = range_bits(vlo, vhi, k0 + 32 * q);
                        if (have != all_parts) {
                            uint32_t parts = 0;
                            for (int e = 0; e < 32; ++e) parts |= ((have >> ((32 * q + e) >> log2_br)) & 1u) << e;
                            bits &= parts;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) x[32 * q + e] = -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[e] = x[e];
#pragma unroll
                for (int e = 8; e < kBlkKeys; ++e) mx[e & 7] = fmaxf(mx[e & 7], x[e]);
                const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                       fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                const bool move = mt > m_run + kRescale || (m_run == -INFINITY && mt > -INFINITY);
                float corr = 1.f;
                if (move) {
                    corr = m_run == -INFINITY ? 0.f : ex2(m_run - mt);
                    l_run *= corr;
                    m_run = mt;
                }
                const float mu = m_run == -INFINITY ? 0.f : m_run;
                if (__any_sync(0xffffffffu, move && j >= NG)) {  // rescale O rows, after the P V before this one
                    const int tp = t - NG;
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(&pv_done[tp & 1], (tp >> 1) & 1, err, ERR_BLOCK_SOFTMAX))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int col = 0; col < HD; col += 32) {
                        uint32_t r[32];
                        tmem_ld32(t_o + col, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * corr);
                        tmem_st32(t_o + col, r);
                    }
                    tmem_st_wait();
                }
                float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float p0 = ex2(x[64 * half + 2 * e] - mu), p1 = ex2(x[64 * half + 2 * e + 1] - mu);
                        ls[e & 3] += p0 + p1;
                        p[e] = H2::pack(p0, p1);
                    }
                    tmem_st32(tb + 32 * half, p);
                }
                l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[buf]);
            }
            // the unit's last products
            for (int e = 1; ok && e <= 2 && e <= n; ++e) {
                const int tp = jj + n - e;
                ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[tp & 1], (tp >> 1) & 1, err, ERR_BLOCK_SOFTMAX));
            }
            tc_fence_after();
            jj += n;
            float f0 = 1.f, f1 = 0.f, m = m_run, l = l_run;
            bool has0 = true, has1 = false;
            if constexpr (NG == 2) {
                s_ml[grp * kBlkRows + row] = make_float2(m_run, l_run);
                bar_sync(1, NG * 128);
                const float2 A = s_ml[row], B = s_ml[kBlkRows + row];
                const int j_first = (jj - n) & 1;  // the group of the unit's first tile
                has0 = n > 1 || j_first == 0;
                has1 = n > 1 || j_first == 1;
                m = fmaxf(A.x, B.x);
                f0 = A.x == -INFINITY ? 1.f : ex2(A.x - m);
                f1 = B.x == -INFINITY ? 1.f : ex2(B.x - m);
                l = A.y * f0 + B.y * f1;
            }
            const bool whole = b0 == 0 && b1 == s.blocks, live = ok && row < rows;
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (b0 == 0 ? 1 : 0);
            const Tile tile{s.first, row0, rows, h};
            const int c_begin = NG == 2 ? grp * (HD / 2) : 0, c_end = c_begin + HD / NG;
            const uint32_t to = tmem + lane_off;
#pragma unroll 1
            for (int col = c_begin; col < c_end; col += 32) {
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.f;
                uint32_t r[32];
                if (has0) {
                    tmem_ld32(to + col, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * f0;
                }
                if (NG == 2 && has1) {
                    tmem_ld32(to + HD + col, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] += __uint_as_float(r[e]) * f1;
                }
                if (!live) continue;
                if (whole) {
                    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
                    const int tok = tile.first + (row0 + row) / a.p.G, head = h * a.p.G + (row0 + row) % a.p.G;
                    uint4* dst = reinterpret_cast<uint4*>(a.out.p + (tok * a.out.ts + head * a.out.hs + col) * 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[e] = make_uint4(H2::pack(v[8 * e] * inv, v[8 * e + 1] * inv),
                                            H2::pack(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                            H2::pack(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                            H2::pack(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                    if (a.lse != nullptr && col == 0)
                        a.lse[static_cast<size_t>(tok) * a.Hq + head] =
                            l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
                } else {
                    float4* dst = reinterpret_cast<float4*>(part_o(a, HD, slot, row) + col);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        __stcg(dst + e, make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
                    if (col == 0) __stcg(reinterpret_cast<float2*>(part_ml(a, HD, slot, row)), make_float2(m, l));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            if (!whole) {
                const int c_first = static_cast<int>(u0 / walk.per);
                const int c_last = static_cast<int>((u0 + s.blocks - 1) / walk.per);
                __threadfence();
                bar_sync(1, NG * 128);
                if (tid == 0)
                    *s_flag = ok && atomicInc(a.counters + c_first, c_last - c_first) ==
                              static_cast<unsigned>(c_last - c_first);
                bar_sync(1, NG * 128);
                if (*s_flag) {  // every piece of this unit is in memory; the counter is back at zero
                    __threadfence();
                    join_pieces<HD>(a, tile, BF, 1.f, c_first, c_last, tid, NG * 128);
                }
            }
            if (NG == 2 || !whole) bar_sync(1, NG * 128);  // s_ml and s_flag are free again
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace paged
}  // namespace dgen
