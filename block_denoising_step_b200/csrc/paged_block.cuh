// Attention of many query rows per KV head over the paged cache (a canvas over
// its prompt, a chunk of a prompt) on the 5th-generation tensor cores.
//
// The same formula and masks as paged_split.cuh.  The rows of a tile are the
// tokens times the G query heads of one KV head (row = token * G + head), up to
// 128, so K and V are read once for the whole group.  One CTA per SM walks the
// units of paged_work.cuh in blocks of 128 keys:
//
//   warp 2           scheduler: walks the units and hands each piece to the other
//                    warps through shared memory, two in flight;
//   warps 0, 3       producers: Q by one TMA box per 64 columns ([tokens][G] rows),
//                    K (warp 0) and V (warp 3) in stages of 128 keys x SC columns (32 KB), one TMA box
//                    per page part (BR rows, a power of two that divides the page
//                    size) and 64 columns;
//   warp 1           MMA issuer: S = Q K^T (128 x 128 fp32) into one of NB TMEM
//                    buffers, O += P V with P from tensor memory (the upper 64 columns
//                    of its S buffer) and V MN-major from shared memory;
//   8 warps          softmax: thread = query row.  Two warpgroups take alternate
//                    tiles; the running maximum goes from one to the other through
//                    shared memory as soon as a tile's is known, each keeps its own
//                    sum, joined at the unit's end.
//
// Order of the products, with NB score buffers: S0 .. S(NB-1), P0 V0, S(NB), P1 V1,
// S(NB+1), ...: two tiles' softmax run beside the products of their neighbours.
// hd <= 128 has room for a third buffer, so that a warpgroup finds its next scores
// ready when it has finished a tile (with two, and an O of its own for each
// warpgroup, it waited for P V and the next S: 2,700 cycles per tile at hd 128).  Tiles of 128 keys, because
// S = Q K^T with N = 64 would read 6 KB of operands per 32 cycles, more than shared
// memory delivers; with N = 128 it is 8 KB per 64.
// P is rounded once to the operand type (bf16 / fp16): hi + lo parts as in the
// split kernel would add half as many products again.  Its error is that of one
// rounding per weight: averaged over the keys where many count, as large as the
// output's own rounding where few do.
//
// Measured on a B200 (device time of a replayed graph): eight canvases of 256 tokens over
// 4,352 keys, 16 heads on 8 of 256, 128 to 131 us on several boxes (1,117 to 1,139 TFLOP/s;
// tensor cores); one over 2,304 keys 24.5 us (five blocks per CTA: start-up and join outweigh
// them); six ragged causal chunks of up to 1,024 tokens over 5,000 keys, 32 heads on 8 of 128,
// capped scores, 278 to 315 us (the capped scores' fp32 work; 470 with scores past the cap).
//
// Pages behind the sequence's end and absent ones are not loaded; the last page part is, as
// a whole.  Scores of keys that do not count are replaced by -inf, and their V rows by zeros
// (shared memory may hold anything).  Every wait is bounded; on a timeout the kernel records an
// error, drains its own copies and MMAs, frees its tensor memory and exits.
#pragma once

#include "paged_work.cuh"

namespace dgen {
namespace paged {

enum : int { ERR_BLOCK_PRODUCER = 20, ERR_BLOCK_MMA = 21, ERR_BLOCK_SOFTMAX = 22, ERR_BLOCK_DRAIN = 23, ERR_BLOCK_PIECE = 24 };

// Caps on the scores: none; usual ones, whose tanh is a polynomial of a tile's raw scores with the powers of scale /
// cap in its coefficients; any other, whose powers leave fp32's range: the form is chosen and computed per score.
enum class Cap { none, usual, any };
inline Cap cap_form(float scale, float cap) {
    if (cap <= 0.f) return Cap::none;
    const double fac = static_cast<double>(scale) * kLog2e, w2 = fac * kLn2 / cap * (fac * kLn2 / cap);
    const double last = fac * w2 * w2 * w2 * w2;  // of the last coefficient, which is 0.0153 of it
    return last >= 0x1p-119 && last <= 0x1p100 ? Cap::usual : Cap::any;
}

constexpr int kBlkKeys = 128;
constexpr int kBlkRows = 128;

template <int HD>
struct BlockLayout {
    static constexpr int SC = HD < 128 ? HD : 128;    // columns of a stage
    static constexpr int NS = HD / SC;                // stages per K or V tile
    static constexpr int NB = HD == 256 ? 2 : 3;      // score buffers in tensor memory
    static constexpr int THREADS = 384;               // four role warps, two warpgroups of softmax
    static constexpr int Q_BYTES = kBlkRows * HD * 2; // HD / 64 boxes of [128 rows x 128 B]
    static constexpr int STAGE = kBlkKeys * SC * 2;   // K: SC / 64 boxes of [128 rows x 128 B]
    // V: at hd 256 64 keys x 256 columns, so that one product covers all of them (N = 256: 128 cycles, half the
    // instructions for the issuing thread, and time for it to signal and wait in), else as K
    static constexpr int VR = HD == 256 ? 64 : kBlkKeys;
    static constexpr int VB = STAGE / (VR * 128);     // boxes of [VR rows x 128 B]
    static constexpr int STAGES = HD == 64 ? 8 : 5;
    static constexpr int KV_OFF = Q_BYTES;
    static constexpr int M_OFF = KV_OFF + STAGES * STAGE;  // float m[2][128]: the running maximum, by tile parity
    static constexpr int PIECE_OFF = M_OFF + 2 * kBlkRows * 4;
    static constexpr int BAR_OFF = PIECE_OFF + 2 * 64;
    // q_full, q_empty, kv_full[ST], kv_empty[ST], s_full[NB], p_full[NB], pv_done[NB], m_pub[2], l_full, l_read,
    // o_free, drain, tail, piece_full[2], piece_empty[2]
    static constexpr int N_BARS = 2 + 2 * STAGES + 3 * NB + 2 + 5 + 4;
    static constexpr int SLOT_OFF = BAR_OFF + N_BARS * 8;            // TMEM base
    static constexpr int SMEM_BYTES = SLOT_OFF + 16 + 1024;          // + slack for 1024-byte alignment
    static_assert(HD + NB * kBlkKeys <= 512, "tensor memory");
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
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}
// 32 lanes x 16 consecutive fp32 columns from registers
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 scores of each of this warp's rows: the load is started, and waited for, apart
// (the wait names the registers, so that nothing reads them before it)
__device__ __forceinline__ void scores_start(uint32_t taddr, float (&x)[32]) {
    tmem_ld32(taddr, reinterpret_cast<uint32_t(&)[32]>(x));
}
__device__ __forceinline__ void scores_wait(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]),
                   "+f"(x[22]), "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]),
                   "+f"(x[29])
                 :
                 : "memory");
    asm volatile("" : "+f"(x[30]), "+f"(x[31]));
}
// two fp32 values in one register pair: packed arithmetic halves the instructions
// of the softmax, which shares its issue slots with the exponentials
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// bits [lo, hi) of a 32-bit word whose bit 0 is position `base`
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int base) {
    const int a = min(max(lo - base, 0), 32), b = min(max(hi - base, 0), 32);
    const uint32_t up = b >= 32 ? 0xFFFFFFFFu : (1u << b) - 1u, dn = a >= 32 ? 0xFFFFFFFFu : (1u << a) - 1u;
    return up & ~dn;
}

// Sets 32 scores of the tile's columns c0 .. (keys k0 ..) to `none` outside [lo, hi) and
// in absent page parts.
__device__ __forceinline__ void mask_scores(float (&x)[32], int lo, int hi, int k0, int c0, uint32_t have, int log2_br,
                                            float none) {
    uint32_t parts = 0;
    if (log2_br >= 5) {
        parts = (have >> (c0 >> log2_br)) & 1u ? 0xFFFFFFFFu : 0u;
    } else {
        const uint32_t one = (1u << (1 << log2_br)) - 1u;
        for (int e = 0; e < 32; e += 1 << log2_br) parts |= (have >> ((c0 + e) >> log2_br)) & 1u ? one << e : 0u;
    }
    const uint32_t bits = range_bits(lo, hi, k0) & parts;
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!((bits >> e) & 1u)) x[e] = none;
}

// Partial results of this kernel: [slot][hd / 4][128 rows] float4, so that a warp
// (32 rows) writes and reads whole lines, then [slot][128] (m, l).
__device__ __forceinline__ float4* block_part(const AttendArgs& a, int hd, size_t slot, int col, int row) {
    return reinterpret_cast<float4*>(a.parts) + (slot * (hd / 4) + col / 4) * kBlkRows + row;
}
__device__ __forceinline__ float2* block_part_ml(const AttendArgs& a, int hd, size_t slot, int row) {
    return reinterpret_cast<float2*>(a.parts + 2 * static_cast<size_t>(a.n_ctas) * kBlkRows * hd) + slot * kBlkRows + row;
}

// Page parts of a tile of 128 keys: lane i < nbox holds the cache row of part i
// (kNoRow: absent or behind hi).  The table entry is loaded one tile ahead.
struct Parts {
    int key, id;
    __device__ __forceinline__ void ahead(const CacheView& c, int b, int key_, int hi, int nbox, int lane) {
        key = key_;
        id = lane < nbox && key < hi ? page_entry(c, b, c.page_of(key)) : -1;
    }
    __device__ __forceinline__ uint32_t row(const CacheView& c, int h) const {
        return id >= 0 ? row_in_page(c, id, h, key - c.page_of(key) * c.page) : kNoRow;
    }
};

template <int HD, bool BF, Cap CAP>
__global__ void __launch_bounds__(BlockLayout<HD>::THREADS, 1)
    paged_block_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const AttendArgs a, int log2_br, int* __restrict__ err) {
    using L = BlockLayout<HD>;
    using H2 = Half2<BF>;
    constexpr int NB = L::NB, ST = L::STAGES;
    constexpr float LIFT = BF ? 0.f : kHalfLift;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem), sQ = sbase, sKV = sbase + L::KV_OFF;
    float* s_m = reinterpret_cast<float*>(smem + L::M_OFF);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t *q_full = bars, *q_empty = bars + 1, *kv_full = bars + 2, *kv_empty = kv_full + ST;
    uint64_t *s_full = kv_empty + ST, *p_full = s_full + NB, *pv_done = p_full + NB, *m_pub = pv_done + NB;
    uint64_t *l_full = m_pub + 2, *l_read = l_full + 1, *o_free = l_read + 1, *drain = o_free + 1, *tail = drain + 1;
    uint64_t *piece_full = tail + 1, *piece_empty = piece_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    static_assert(sizeof(Piece) <= 64, "piece slot");
    volatile Piece* s_piece = reinterpret_cast<volatile Piece*>(smem + L::PIECE_OFF);  // 64 bytes apart

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(o_free, 8);
        mbar_init(drain, 1);
        mbar_init(tail, 1);
        mbar_init(l_full, 8);
        mbar_init(l_read, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m_pub[i], 4);
            mbar_init(&piece_full[i], 1);
            mbar_init(&piece_empty[i], 3 + 8);  // producers, MMA issuer, softmax warps
        }
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
    // all 512 columns are this CTA's, so its first column is column 0 (a constant base keeps the issue short)
    constexpr uint32_t t_s = HD;
    const CacheView& c = a.c;
    const int br = 1 << log2_br, nbox = kBlkKeys >> log2_br;

    Piece s;
    int piece_no = 0;
    // The next piece of the scheduler's walk into s; false at its end or when the wait ran out.
    auto next_piece = [&]() -> bool {
        const int i = piece_no & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&piece_full[i], (piece_no >> 1) & 1, err, ERR_BLOCK_PIECE))) return false;
        const volatile int* from = reinterpret_cast<const volatile int*>(reinterpret_cast<const volatile uint8_t*>(s_piece) + i * 64);
        int* to = reinterpret_cast<int*>(&s);
#pragma unroll
        for (int e = 0; e < static_cast<int>(sizeof(Piece) / 4); ++e) to[e] = from[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_empty[i]);
        ++piece_no;
        return s.end == 0;
    };

    if (warp == 2) {
        Walk walk;
        walk.start(c, a.p, lane, blockIdx.x, a.n_ctas);
        // What the join kernel has to know of the unit that starts here and goes on behind: none until it is met, so
        // that a walk that a wait ends early leaves no record of an earlier call.
        if (lane == 0) a.joins[blockIdx.x].end = 1;
        for (int i = 0;; ++i) {
            Piece q{};
            const bool have = walk.next(c, a.p, lane, q);
            q.end = !have;
            if (lane == 0 && have && q.starts && !q.whole && q.rows > 0) a.joins[blockIdx.x] = q;
            if (!__all_sync(0xffffffffu,
                            mbar_wait(&piece_empty[i & 1], ((i >> 1) & 1) ^ 1, err, ERR_BLOCK_PIECE)))
                break;
            if (lane == 0) {
                volatile int* to = reinterpret_cast<volatile int*>(reinterpret_cast<volatile uint8_t*>(s_piece) + (i & 1) * 64);
                const int* from = reinterpret_cast<const int*>(&q);
#pragma unroll
                for (int e = 0; e < static_cast<int>(sizeof(Piece) / 4); ++e) to[e] = from[e];
                mbar_arrive(&piece_full[i & 1]);
            }
            __syncwarp();
            if (!have) break;
        }
    } else if (warp == 0 || warp == 3) {
        const bool is_v = warp == 3;
        const CUtensorMap* tm = is_v ? &tmV : &tmK;
        if (lane == 0) {
            if (!is_v) prefetch_tmap(&tmQ);
            prefetch_tmap(tm);
        }
        int unit_no = 0, base = 0;  // base: stages of the ring used by the CTA's earlier pieces
        uint32_t pending = 0, fill_ph = 0, tail_ph = 0;
        const bool leader = elect_one();
        bool ok = true;
        bool tail_open = false;  // copies that report to `tail` are on their way
        int q_phase = -1;  // parity of the last Q copy issued
        // This warp's tile of 128 keys from key k0 on into the ring from its stage number `at` on; `row` is
        // this lane's page part.  V rows that must not count (behind hi, absent pages) are cleared here.
        auto fetch = [&](int at, uint32_t row, int k0) {
            const int live = min(s.hi - k0, kBlkKeys);
            const uint32_t have = __ballot_sync(0xffffffffu, row != kNoRow);
            const uint32_t absent = ~have & ((1u << nbox) - 1u);
            // rows to clear: the copies then report to a barrier of their own, and kv_full follows the clearing
            const bool clear = is_v && (live < kBlkKeys || absent != 0);
            const int stage_rows = is_v ? L::VR : kBlkKeys, boxes = is_v ? L::VB : L::SC / 64;
#pragma unroll
            for (int n = 0; n < L::NS; ++n) {
                const int st = (at + n) % ST;
                const uint32_t ph = ((at + n) / ST) & 1;
                // V at hd 256: stage n holds the keys 64 n .., else (and K): the columns SC n .. of all keys
                const bool by_keys = is_v && L::VR < kBlkKeys;
                const int r0 = by_keys ? n * L::VR : 0, x0 = by_keys ? 0 : n * L::SC;
                const uint32_t mine = by_keys ? ((1u << (L::VR >> log2_br)) - 1u) << (r0 >> log2_br) : 0xFFFFFFFFu;
                if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[st], ph ^ 1u, err, ERR_BLOCK_PRODUCER))) {
                    ok = false;
                    return;
                }
                uint64_t* done = clear ? tail : &kv_full[st];
                if (leader) mbar_expect_tx(done, __popc(have & mine) * br * 128 * boxes);
                __syncwarp();
                // (issued by one thread: copies of several lanes go out one by one at twice the cost)
                for (uint32_t left = have & mine; left != 0; left &= left - 1) {
                    const int part = __ffs(left) - 1;
                    const int r = static_cast<int>(__shfl_sync(0xffffffffu, row, part));
                    const uint32_t dst = sKV + st * L::STAGE + ((part << log2_br) - r0) * 128;
                    if (leader)
                        for (int x = 0; x < boxes; ++x)
                            tma_load_2d(dst + x * (stage_rows * 128), tm, x0 + x * 64, r, smem_u32(done));
                }
                if (clear) {
                    pending &= ~(1u << st);  // (what was there before has been consumed)
                    tail_open = true;
                    if (!__all_sync(0xffffffffu, mbar_wait(tail, tail_ph, err, ERR_BLOCK_PRODUCER))) {
                        ok = false;
                        return;
                    }
                    tail_open = false;
                    tail_ph ^= 1u;
                    constexpr int CH = L::VB * 8;  // 16-byte chunks of a stage row (which is cleared whole: no swizzle)
                    for (int i = lane; i < L::VR * CH; i += 32) {
                        const int r = i / CH, ch = i % CH;
                        if (r0 + r >= live || ((absent >> ((r0 + r) >> log2_br)) & 1u))
                            *reinterpret_cast<uint4*>(smem + L::KV_OFF + st * L::STAGE + (ch >> 3) * (L::VR * 128) +
                                                      r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (leader) mbar_arrive(&kv_full[st]);
                } else {
                    pending |= 1u << st;
                    fill_ph = (fill_ph & ~(1u << st)) | (ph << st);
                }
            }
        };
        while (ok && next_piece()) {
            const int h = s.h, n = s.n;
            if (n == 0) continue;
            const int key0 = s.key0 + lane * br;
            if (!is_v) {
                if (unit_no > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(q_empty, (unit_no - 1) & 1, err, ERR_BLOCK_PRODUCER))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int tok = s.first + s.row0 / a.p.G;
                    mbar_expect_tx(q_full, a.p.R * HD * 2);
#pragma unroll
                    for (int x = 0; x < HD / 64; ++x)
                        tma_load_3d(sQ + x * (kBlkRows * 128), &tmQ, x * 64, h * a.p.G, tok, smem_u32(q_full));
                }
                q_phase = unit_no & 1;
            }
            Parts parts;
            parts.ahead(c, s.b, key0, s.hi, nbox, lane);
            for (int j = 0; ok && j < n; ++j) {
                // ring order K0, .., K(NB-1), V0, K(NB), V1, ..., V(n-2), V(n-1)
                const int at = is_v ? j + min(n, j + NB) : (j < NB ? j : 2 * j - NB + 1);
                const uint32_t row = parts.row(c, h);
                if (j + 1 < n) parts.ahead(c, s.b, key0 + (j + 1) * kBlkKeys, s.hi, nbox, lane);
                fetch(base + at * L::NS, row, s.key0 + j * kBlkKeys);
            }
            // (the ring's length times two: the phase is what counts)
            base = (base + 2 * n * L::NS) % (2 * ST);
            ++unit_no;
        }
        if (!ok) {
            // let our own copies land before the CTA goes away (a stage that the other producer has filled since
            // was consumed before: its wait only runs out).  Without a failure the MMA issuer has waited for
            // every copy; if it alone gave up, it did so two seconds after the last of them.
            if (q_phase >= 0) mbar_wait(q_full, q_phase, err, ERR_BLOCK_DRAIN);
            if (tail_open) mbar_wait(tail, tail_ph, err, ERR_BLOCK_DRAIN);
            for (int i = 0; i < ST; ++i)
                if ((pending >> i) & 1u) mbar_wait(&kv_full[i], (fill_ph >> i) & 1u, err, ERR_BLOCK_DRAIN);
        }
    } else if (warp == 1) {
        // One elected thread issues everything.  A product of 128 x 128 x 16 takes 64 cycles, little more than
        // its issue: what else this thread does, the tensor cores wait for.
        if (elect_one()) {
            constexpr uint32_t type = BF ? (1u << 7) | (1u << 10) : 0u;  // operand types bf16 / f16
            constexpr uint32_t base = (1u << 4) | type | (static_cast<uint32_t>(kBlkRows >> 4) << 24);
            constexpr uint32_t idesc_s = base | (static_cast<uint32_t>(kBlkKeys >> 3) << 17);
            constexpr uint32_t idesc_pv = base | (1u << 16) | (static_cast<uint32_t>(HD >> 3) << 17);  // N = hd
            int st = 0, unit_no = 0;
            int buf = 0, sbuf = 0;      // score buffers of the next P V and the next S
            uint32_t p_ph = 0;          // phase of p_full[buf]
            uint32_t ph = 0;
            bool ok = true;
            auto issue_s = [&]() -> bool {  // the next K tile's scores
#pragma unroll
                for (int x = 0; x < L::NS; ++x) {
                    if (!mbar_wait(&kv_full[st], ph, err, ERR_BLOCK_MMA)) return false;
                    tc_fence_after();
                    const uint64_t ad0 = sdesc_sw128(sQ + x * (L::SC / 64) * (kBlkRows * 128));
                    const uint64_t bd0 = sdesc_sw128(sKV + st * L::STAGE);
#pragma unroll
                    for (int kk = 0; kk < L::SC / 16; ++kk) {
                        const int off = (kk >> 2) * (kBlkRows * 128 / 16) + 2 * (kk & 3);  // 16-byte units
                        mma_bf16_ss(t_s + sbuf * kBlkKeys, ad0 + off, bd0 + off, idesc_s, x > 0 || kk > 0 ? 1u : 0u);
                    }
                    mma_commit(smem_u32(&kv_empty[st]));
                    if (++st == ST) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                mma_commit(smem_u32(&s_full[sbuf]));
                if (++sbuf == NB) sbuf = 0;
                return true;
            };
            for (int i = 0; ok; ++i) {
                const volatile Piece* q = reinterpret_cast<const volatile Piece*>(
                    reinterpret_cast<const volatile uint8_t*>(s_piece) + (i & 1) * 64);
                if (!mbar_wait(&piece_full[i & 1], (i >> 1) & 1, err, ERR_BLOCK_PIECE)) break;
                const int n = q->n, end = q->end;
                mbar_arrive(&piece_empty[i & 1]);
                if (end) break;
                if (n == 0) continue;
                if (!mbar_wait(q_full, unit_no & 1, err, ERR_BLOCK_MMA)) break;
                for (int j = 0; ok && j < n && j < NB; ++j) ok = issue_s();
                if (n <= NB) mma_commit(smem_u32(q_empty));
                for (int j = 0; ok && j < n; ++j) {
                    if (!mbar_wait(&p_full[buf], p_ph, err, ERR_BLOCK_MMA) ||
                        (j == 0 && unit_no > 0 && !mbar_wait(o_free, (unit_no - 1) & 1, err, ERR_BLOCK_MMA))) {
                        ok = false;
                        break;
                    }
                    const uint32_t tp = t_s + buf * kBlkKeys + 64;
                    const uint32_t more = j > 0 ? 1u : 0u;  // (nothing in O yet)
#pragma unroll
                    for (int x = 0; x < L::NS; ++x) {
                        if (!mbar_wait(&kv_full[st], ph, err, ERR_BLOCK_MMA)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t vd0 = sdesc_sw128_mn(sKV + st * L::STAGE, L::VR * 128);
#pragma unroll
                        for (int kk = 0; kk < L::VR / 16; ++kk)
                            mma_ts(0, tp + x * (L::VR / 2) + kk * 8, vd0 + kk * (2048 / 16), idesc_pv,
                                   x > 0 || kk > 0 ? 1u : more);
                        mma_commit(smem_u32(&kv_empty[st]));
                        if (++st == ST) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    mma_commit(smem_u32(&pv_done[buf]));
                    if (++buf == NB) {
                        buf = 0;
                        p_ph ^= 1u;
                    }
                    if (j + NB < n) {
                        ok = issue_s();  // over the scores and weights of the tile just multiplied
                        if (j + NB + 1 == n) mma_commit(smem_u32(q_empty));
                    }
                }
                ++unit_no;
            }
            mma_commit(smem_u32(drain));  // arrives when every MMA issued above has completed
            mbar_wait(drain, 0, err, ERR_BLOCK_DRAIN);
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int grp = (warp - 4) >> 2;  // takes the tiles of its parity
        const int quarter = warp & 3;     // TMEM lanes this warp may access
        const int row = quarter * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const float fac = a.scale * kLog2e, inv_cap = a.cap > 0.f ? kLn2 / a.cap : 0.f;
        const uint32_t all_parts = (1u << nbox) - 1u;
        // tanh's coefficients for raw scores: fac c_i w^(2i + 2), w = fac inv_cap
        float tc[4];
        {
            const float w = fac * inv_cap, w2 = w * w;
            float f = fac * w2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                tc[i] = kTanhCoef[i] * f;
                f *= w2;
            }
        }
        int jj = 0, unit_no = 0;  // jj: tile counter of the CTA
        bool ok = true;
        while (ok && next_piece()) {
            const int h = s.h, n = s.n, row0 = s.row0, rows = s.rows, key0 = s.key0;
            if (rows <= 0) continue;
            int vlo, vhi;
            visible(s.pos0 + (row0 + min(row, rows - 1)) / a.p.G, s.len, a.p.causal, a.p.window, vlo, vhi);
            // keys every row of this warp sees (ranges only move up with the row)
            const int all_lo = __shfl_sync(0xffffffffu, vlo, 31), all_hi = __shfl_sync(0xffffffffu, vhi, 0);
            // is a page of these keys absent?  (looked up while the first scores are on their way)
            bool absent = false;
            if (n > 0) {
                const int p1 = c.page_of(min(key0 + n * kBlkKeys, s.hi) - 1);
#pragma unroll 4
                for (int e = c.page_of(key0) + lane; e <= p1; e += 32)
                    absent |= static_cast<uint32_t>(page_entry(c, s.b, e)) >= static_cast<uint32_t>(c.n_pages);
                absent = __any_sync(0xffffffffu, absent);
            }
            float m_run = -INFINITY, l_run = 0.f;  // the maximum this warp's l is relative to
            // the slots of m are free once every warp has read the sums of the unit before
            if (n > 0 && unit_no > 0 &&
                !__all_sync(0xffffffffu, mbar_wait(l_read, (unit_no - 1) & 1, err, ERR_BLOCK_SOFTMAX)))
                break;
            for (int j = (jj ^ grp) & 1; ok && j < n; j += 2) {
                const int t = jj + j, buf = t % NB, k0 = key0 + j * kBlkKeys;
                uint32_t have = all_parts;
                if (absent) {  // which page parts are there
                    const int key = k0 + lane * br;
                    have = __ballot_sync(0xffffffffu, lane < nbox && key < s.hi &&
                                                          static_cast<uint32_t>(page_entry(c, s.b, c.page_of(key))) <
                                                              static_cast<uint32_t>(c.n_pages));
                }
                const uint32_t tb = t_s + buf * kBlkKeys + lane_off;
                if (!__all_sync(0xffffffffu, mbar_wait(&s_full[buf], (t / NB) & 1, err, ERR_BLOCK_SOFTMAX))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // maximum of the raw scores (scale > 0 and the cap keep their order), 32 columns at a time, the
                // next 32 on their way meanwhile
                const bool cut = have != all_parts || k0 < all_lo || k0 + kBlkKeys > all_hi;
                float xa[32], xb[32];
                float mx[4], mn = INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = -INFINITY;
                auto look = [&](float(&x)[32], int c0) {
                    // (with a cap NaN, which maximum and minimum both pass over: what is masked chooses nothing)
                    if (cut) mask_scores(x, vlo, vhi, k0 + c0, c0, have, log2_br, CAP != Cap::none ? NAN : -INFINITY);
                    if constexpr (CAP == Cap::usual) {
                        float lo[4] = {mn, INFINITY, INFINITY, INFINITY};
#pragma unroll
                        for (int e = 0; e < 16; ++e) lo[e & 3] = min3(lo[e & 3], x[2 * e], x[2 * e + 1]);
                        mn = fminf(fminf(lo[0], lo[1]), fminf(lo[2], lo[3]));
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) mx[e & 3] = max3(mx[e & 3], x[2 * e], x[2 * e + 1]);
                };
                scores_start(tb, xa);
#pragma unroll 1
                for (int c0 = 0; c0 < kBlkKeys; c0 += 64) {
                    scores_wait(xa);
                    scores_start(tb + c0 + 32, xb);
                    look(xa, c0);
                    scores_wait(xb);
                    scores_start(tb + 64, xa);  // (the second time for the weights)
                    look(xb, c0 + 32);
                }
                const float raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                bool small = false;
                float mt = raw * fac;
                if constexpr (CAP != Cap::none) {
                    const float u = mt * inv_cap;
                    // (rows behind the tile's last hold whatever was there: they have no say in which form is taken)
                    if constexpr (CAP == Cap::usual)
                        small = __all_sync(0xffffffffu, row >= rows || raw == -INFINITY ||
                                                            (fabsf(u) <= kTanhSmall &&
                                                             fabsf(mn * fac * inv_cap) <= kTanhSmall));
                    if (raw > -INFINITY)
                        mt = (CAP == Cap::usual ? small : fabsf(u) <= kTanhSmall) ? capped_small(mt, u)
                                                                                 : capped_any(u, kLog2e * a.cap);
                }
                // the maximum after the tile before this one, from the other warpgroup
                float m_prev = -INFINITY;
                if (j > 0) {
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(&m_pub[(t - 1) & 1], ((t - 1) >> 1) & 1, err, ERR_BLOCK_SOFTMAX))) {
                        ok = false;
                        break;
                    }
                    m_prev = s_m[((t - 1) & 1) * kBlkRows + row];
                }
                const bool move = mt > m_prev + kRescale || (m_prev == -INFINITY && mt > -INFINITY);
                const float m_new = move ? mt : m_prev;
                s_m[(t & 1) * kBlkRows + row] = m_new;
                __syncwarp();
                if (lane == 0) mbar_arrive(&m_pub[t & 1]);
                if (m_new != m_run) {
                    l_run *= m_run == -INFINITY ? 0.f : ex2(m_run - m_new);
                    m_run = m_new;
                }
                const float mu = m_run == -INFINITY ? 0.f : m_run - LIFT;
                if (__any_sync(0xffffffffu, move && j > 0)) {  // rescale O rows, after the P V before this one
                    const float corr = move ? (m_prev == -INFINITY ? 0.f : ex2(m_prev - m_new)) : 1.f;
                    if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(t - 1) % NB], ((t - 1) / NB) & 1, err,
                                                           ERR_BLOCK_SOFTMAX))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int col = 0; col < HD; col += 32) {
                        uint32_t r[32];
                        tmem_ld32(col + lane_off, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * corr);
                        tmem_st32(col + lane_off, r);
                    }
                    tmem_st_wait();
                }
                f32x2 ls[2] = {0ull, 0ull};
                const f32x2 fac2 = pair(fac, fac), nmu2 = pair(-mu, -mu);
                // P of 32 columns c0 .. over columns 64 + c0 / 2 .. of S_j, whose scores have been read by then
                auto weigh = [&](float(&x)[32], int c0) {
                    uint32_t p[16];
                    if constexpr (CAP == Cap::none) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = unpair(fma2(pair(x[2 * e], x[2 * e + 1]), fac2, nmu2));
                            const float p0 = ex2(y.x), p1 = ex2(y.y);
                            ls[e & 1] = add2(ls[e & 1], pair(p0, p1));
                            p[e] = H2::pack(p0, p1);
                        }
                    } else if (small) {  // capped_small in pairs, its powers of 1 / cap in the coefficients
                        // (a masked -inf stays -inf: v z is, and q, whose leading coefficient is positive, is +inf)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const f32x2 v = pair(x[2 * e], x[2 * e + 1]), z = mul2(v, v);
                            f32x2 q = fma2(z, pair(tc[3], tc[3]), pair(tc[2], tc[2]));
                            q = fma2(z, q, pair(tc[1], tc[1]));
                            q = fma2(z, q, pair(tc[0], tc[0]));
                            const float2 y = unpair(fma2(mul2(v, z), q, fma2(v, fac2, nmu2)));
                            const float p0 = ex2(y.x), p1 = ex2(y.y);
                            ls[e & 1] = add2(ls[e & 1], pair(p0, p1));
                            p[e] = H2::pack(p0, p1);
                        }
                    } else {
                        const float cap2 = kLog2e * a.cap;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float pe[2];
#pragma unroll
                            for (int w = 0; w < 2; ++w) {
                                const float y = x[2 * e + w] * fac, u = y * inv_cap;
                                const float f = CAP == Cap::any && fabsf(u) <= kTanhSmall ? capped_small(y, u) : capped_any(u, cap2);
                                pe[w] = y == -INFINITY ? 0.f : ex2(f - mu);
                            }
                            ls[e & 1] = add2(ls[e & 1], pair(pe[0], pe[1]));
                            p[e] = H2::pack(pe[0], pe[1]);
                        }
                    }
                    tmem_st16(tb + 64 + c0 / 2, p);
                };
                // columns 96 .. (left from above), 64 .., 32 .., 0 ..
                if (CAP != Cap::none && cut) mask_scores(xb, vlo, vhi, k0 + 96, 96, have, log2_br, -INFINITY);
#pragma unroll 1
                for (int c0 = 64; c0 >= 0; c0 -= 64) {
                    weigh(xb, c0 + 32);
                    scores_wait(xa);
                    if (c0 > 0) scores_start(tb + 32, xb);
                    if (cut) mask_scores(xa, vlo, vhi, k0 + c0, c0, have, log2_br, -INFINITY);
                    weigh(xa, c0);
                    if (c0 > 0) {
                        scores_wait(xb);
                        scores_start(tb, xa);
                        if (cut) mask_scores(xb, vlo, vhi, k0 + 32, 32, have, log2_br, -INFINITY);
                    }
                }
                const float2 lsum = unpair(add2(ls[0], ls[1]));
                l_run += lsum.x + lsum.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[buf]);
            }
            if (!ok) break;
            // The unit's maximum is the last tile's; both warpgroups' sums relative to it.  They change hands in
            // the slots of m, which the two threads of a row alone use and have read by then.
            float m = -INFINITY, l = 0.f;
            if (n > 0) {
                const int last = jj + n - 1, own = (last & 1) == grp;
                m = m_run;
                if (!own) {
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(&m_pub[last & 1], (last >> 1) & 1, err, ERR_BLOCK_SOFTMAX)))
                        break;
                    m = s_m[(last & 1) * kBlkRows + row];
                    l_run *= m_run == -INFINITY ? 1.f : ex2(m_run - m);
                }
                s_m[((last + own) & 1) * kBlkRows + row] = l_run;
                __syncwarp();
                if (lane == 0) mbar_arrive(l_full);
                if (!__all_sync(0xffffffffu, mbar_wait(l_full, unit_no & 1, err, ERR_BLOCK_SOFTMAX))) break;
                l = l_run + s_m[((last + 1 - own) & 1) * kBlkRows + row];
                __syncwarp();
                if (lane == 0) mbar_arrive(l_read);
                if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[last % NB], (last / NB) & 1, err, ERR_BLOCK_SOFTMAX)))
                    break;
                tc_fence_after();
                m -= LIFT;
                jj += n;
                ++unit_no;
            }
            const bool whole = s.whole, live = row < rows;
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s.starts ? 1 : 0);
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const int tok = s.first + (row0 + row) / a.p.G, head = h * a.p.G + (row0 + row) % a.p.G;
            // half of the columns each; a piece that saw no key leaves (-inf, 0) alone
            const int c_end = n == 0 && !whole ? grp * (HD / 2) + 1 : (grp + 1) * (HD / 2);
#pragma unroll 1
            for (int col = grp * (HD / 2); col < c_end; col += 32) {
                float v[32];
                if (n > 0) {
                    tmem_ld32(col + lane_off, reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.f;
                }
                if (!live) continue;
                if (whole) {
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
                    float4* dst = block_part(a, HD, slot, col, row);
#pragma unroll
                    for (int e = 0; n > 0 && e < 8; ++e)
                        __stcg(dst + e * kBlkRows, make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
                    if (col == 0) __stcg(block_part_ml(a, HD, slot, row), make_float2(m, l));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && n > 0) mbar_arrive(o_free);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, 512);
    }
}

// Joins the units that paged_block_kernel's CTAs cut: block (c, y) adds 16 columns
// of CTA c's row tile of the unit that starts in its team and goes on behind it, if
// there is one (a.joins, written by the scheduler).  A launch of its own, because a
// row tile's pieces are up to 128 KB each: the CTA that finishes last would read
// them alone (one canvas of 256 tokens over 2,304 keys at hd 256: 132 us so, 45 with this
// launch and scores read twice instead of kept; 24 now).  Nothing is joined while the
// workspace holds an error: pieces may be missing.
constexpr int kJoinCols = 16;
template <int HD, bool BF>
__global__ void __launch_bounds__(256) paged_block_join_kernel(const AttendArgs a, const int* __restrict__ err) {
    using H2 = Half2<BF>;
    pdl_enter();
    const int cta = blockIdx.x, member = cta & (a.p.TS - 1);
    const Piece s = a.joins[cta];
    const int row = threadIdx.x & (kBlkRows - 1), col = blockIdx.y * kJoinCols + (threadIdx.x >> 7) * 8;
    if (s.end || row >= s.rows || __ldcg(err) != 0) return;
    float m = -INFINITY, l = 0.f, v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
    for (int k = s.t_first; k <= s.t_last; ++k) {  // in piece order
        const size_t slot = 2 * static_cast<size_t>(k * a.p.TS + member) + (k == s.t_first ? 1 : 0);
        const float2 ml = __ldcg(block_part_ml(a, HD, slot, row));
        const float4 x0 = __ldcg(block_part(a, HD, slot, col, row)), x1 = __ldcg(block_part(a, HD, slot, col + 4, row));
        const float mn = fmaxf(m, ml.x);
        const float fo = m == -INFINITY ? 1.f : ex2(m - mn), fn = ml.x == -INFINITY ? 1.f : ex2(ml.x - mn);
        const bool none = ml.x == -INFINITY && ml.y == 0.f;  // no key seen: nothing was written
        const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * fo + (none ? 0.f : x[e] * fn);
        l = l * fo + ml.y * fn;
        m = mn;
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int tok = s.first + (s.row0 + row) / a.p.G, head = s.h * a.p.G + (s.row0 + row) % a.p.G;
    *reinterpret_cast<uint4*>(a.out.p + (tok * a.out.ts + head * a.out.hs + col) * 2) =
        make_uint4(H2::pack(v[0] * inv, v[1] * inv), H2::pack(v[2] * inv, v[3] * inv),
                   H2::pack(v[4] * inv, v[5] * inv), H2::pack(v[6] * inv, v[7] * inv));
    if (a.lse != nullptr && col == 0)
        a.lse[static_cast<size_t>(tok) * a.Hq + head] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace paged
}  // namespace dgen
