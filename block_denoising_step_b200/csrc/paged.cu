// Host side of the paged KV cache's C entry points (include/dgen.h): argument
// checks, the choice of kernel, launches.  No handle: the calls launch on the
// current device and keep nothing but per-device constants.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <utility>

#include "dgen.h"
#include "launch.cuh"
#include "paged_append.cuh"
#include "paged_block.cuh"
#include "paged_split.cuh"

using namespace dgen;

namespace {

constexpr int kMaxGrid = 1023;           // CTAs of an attention launch at most (its counters)
constexpr size_t kCounterBytes = (kMaxGrid + 1) * sizeof(unsigned int);  // and the device-side error word
constexpr size_t kHeadBytes = kCounterBytes + kMaxGrid * 64;             // and the block kernel's join list
static_assert(sizeof(paged::Piece) <= 64, "join list");
constexpr int kMaxLine = INT32_MAX - kMaxGrid;  // blocks of all units: rounded up to the grid they count in 32 bits
constexpr int kMaxDevices = 64;
constexpr int kMaxHeads = 65536;         // query or KV heads: a token's rows and items count in 32 bits
constexpr int kMaxSms = 148;             // SMs that an attention launch uses at most (its workspace)
constexpr int kMaxSplitCtas = 4;         // CTAs per SM of the split kernel at most

int sm_count(int dev) {
    static std::atomic<int> known[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }  // (or null)

// 16-byte access to every row: base and strides (of dimensions above one)
bool good_rows(const dgen_token_rows* r, int tokens, int heads) {
    return r && aligned16(r->dev) && (tokens == 1 || r->token_stride % 8 == 0) &&
           (heads == 1 || r->head_stride % 8 == 0);
}

// Rows that are written: as above, and no two of them share an element (the longer of the two strides passes over all
// rows of the shorter one, and that over a row)
bool good_rows_out(const dgen_token_rows* r, int tokens, int heads, int hd) {
    if (!good_rows(r, tokens, heads)) return false;
    int64_t ts = tokens > 1 ? std::abs(r->token_stride) : INT64_MAX, hs = heads > 1 ? std::abs(r->head_stride) : INT64_MAX;
    int inner = ts < hs ? tokens : heads;
    if (ts < hs) std::swap(ts, hs);  // hs: the shorter
    return hs >= hd && (ts == INT64_MAX || (ts - hd) / hs >= inner - 1);
}

paged::RowsView view(const dgen_token_rows* r) {
    return {static_cast<uint8_t*>(r->dev), r->token_stride, r->head_stride};
}

int check_cache(const dgen_paged_cache* c, int n_tokens, const int32_t* cu) {
    if (!c || !aligned16(c->k_dev) || !aligned16(c->v_dev) || !c->page_table_dev || !c->kv_len_dev) return DGEN_EINVAL;
    if (c->type != DGEN_TYPE_BF16 && c->type != DGEN_TYPE_F16 && c->type != DGEN_TYPE_E4M3) return DGEN_EINVAL;
    if ((c->type == DGEN_TYPE_E4M3) != (c->k_scale_dev != nullptr) || !c->k_scale_dev != !c->v_scale_dev)
        return DGEN_EINVAL;
    if (!aligned4(c->page_table_dev) || !aligned4(c->kv_len_dev) || !aligned4(c->k_scale_dev) ||
        !aligned4(c->v_scale_dev) || !aligned4(cu))
        return DGEN_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DGEN_EINVAL;
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads || c->page_size < 1 || c->batch < 1 || c->table_pages < 1 ||
        c->table_stride < c->table_pages)
        return DGEN_EINVAL;
    const int64_t rows = static_cast<int64_t>(c->n_pages) * c->n_kv_heads;  // rows of the cache count in 32 bits
    if (rows > INT32_MAX || rows * c->page_size >= static_cast<int64_t>(UINT32_MAX)) return DGEN_EINVAL;
    if (static_cast<int64_t>(c->table_pages) * c->page_size > (int64_t{1} << 30)) return DGEN_EINVAL;
    if (n_tokens < 0 || (!cu && n_tokens % c->batch)) return DGEN_EINVAL;
    return DGEN_OK;
}

paged::CacheView view(const dgen_paged_cache* c, int n_tokens, const int32_t* cu) {
    paged::CacheView v{};
    v.k = static_cast<uint8_t*>(c->k_dev);
    v.v = static_cast<uint8_t*>(c->v_dev);
    v.k_scale = c->k_scale_dev;
    v.v_scale = c->v_scale_dev;
    v.table = c->page_table_dev;
    v.kv_len = c->kv_len_dev;
    v.cu = cu;
    v.n_pages = c->n_pages;
    v.Hkv = c->n_kv_heads;
    v.page = c->page_size;
    v.B = c->batch;
    v.table_stride = c->table_stride;
    v.table_pages = c->table_pages;
    v.n_tokens = n_tokens;
    v.n_uniform = n_tokens / c->batch;
    // k = 30 + ceil(log2 page), mul = ceil(2^k / page): mul page - 2^k < page, so pos (mul page - 2^k) < 2^k and
    // the quotient is exact for every pos < 2^30
    int bits = 0;
    while ((int64_t{1} << bits) < c->page_size) ++bits;
    v.page_shift = 30 + bits;
    v.page_mul = static_cast<uint32_t>(((uint64_t{1} << v.page_shift) + c->page_size - 1) / c->page_size);
    return v;
}

template <int HD, bool BF, bool E4M3>
int launch_append(cudaStream_t st, const paged::AppendArgs& a, int per_block) {
    const int blocks = a.c.n_tokens / per_block + (a.c.n_tokens % per_block != 0);
    return launch_ex(st, paged::paged_append_kernel<HD, BF, E4M3>, dim3(blocks), dim3(paged::kAppendThreads), 0, a,
                     per_block) == cudaSuccess
               ? DGEN_OK
               : DGEN_ECUDA;
}

template <int HD>
int append_hd(cudaStream_t st, const paged::AppendArgs& a, int per_block, bool bf, bool e4m3) {
    if (bf) return e4m3 ? launch_append<HD, true, true>(st, a, per_block) : launch_append<HD, true, false>(st, a, per_block);
    return e4m3 ? launch_append<HD, false, true>(st, a, per_block) : launch_append<HD, false, false>(st, a, per_block);
}

struct Workspace {
    unsigned int* counters;
    int* err;
    paged::Piece* joins;
    float* parts;
    size_t floats;
};

template <int HD, int ES, bool BF, int NT>
int launch_split(cudaStream_t st, int dev, int sms, paged::AttendArgs a, const Workspace& ws, int64_t rows_most) {
    using S = paged::SplitSmem<HD, ES, NT>;
    // whole tokens per row tile, where a token's rows fit one (the walk counts a tile's keys by its tokens)
    const bool tokens_fit = a.p.G <= S::R;
    a.p.R = tokens_fit ? S::R / a.p.G * a.p.G : S::R;
    a.p.KB = paged::SplitLayout<HD, ES, NT>::BLOCK_KEYS;
    a.p.log2_kb = a.p.KB == 64 ? 6 : 7;
    static_assert(paged::SplitLayout<HD, ES, NT>::BLOCK_KEYS == 64 || paged::SplitLayout<HD, ES, NT>::BLOCK_KEYS == 128,
                  "log2_kb");
    a.p.align = rows_most <= a.p.R || !tokens_fit ? 1 : a.p.KB;
    a.p.TS = 1;
    a.p.tokens = std::max(1, a.p.R / a.p.G);
    a.p.unit_cost = 3;
    auto kern = paged::paged_split_kernel<HD, ES, BF, NT>;
    set_smem_attr_once(kern, S::BYTES, dev);
    static std::atomic<int> per_sm{0};  // resident CTAs per SM: a property of the kernel
    if (per_sm.load(std::memory_order_relaxed) == 0) {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, paged::kSplitWarps * 32, S::BYTES) != cudaSuccess)
            return DGEN_ECUDA;
        per_sm.store(std::clamp(n, 1, kMaxSplitCtas), std::memory_order_relaxed);
    }
    int64_t grid = std::min(kMaxGrid, sms * per_sm.load(std::memory_order_relaxed));
    // no more CTAs than blocks of the longest possible line
    const int64_t rows = static_cast<int64_t>(a.c.n_tokens) * a.p.G;
    const int64_t tiles = std::min<int64_t>(rows, rows / a.p.R + a.c.B) * a.c.Hkv;
    const int64_t blocks = (static_cast<int64_t>(a.c.table_pages) * a.c.page + a.p.KB - 1) / a.p.KB;
    if (tiles * (blocks + 3) >= kMaxLine) return DGEN_EINVAL;  // (rows <= 2^31, blocks <= 2^24: no overflow)
    grid = std::max<int64_t>(1, std::min(grid, tiles * blocks));
    if (2 * static_cast<size_t>(grid) * S::R * (HD + 2) > ws.floats) return DGEN_ESCRATCH;
    a.counters = ws.counters;
    a.parts = ws.parts;
    a.n_ctas = static_cast<int>(grid);
    return launch_ex(st, kern, dim3(static_cast<unsigned>(grid)), dim3(paged::kSplitWarps * 32), S::BYTES, a) == cudaSuccess
               ? DGEN_OK
               : DGEN_ECUDA;
}

// Row tiles of 8, 16 or (hd <= 128: the accumulators of 32 rows of 256 would not
// fit the registers) 32 query rows, by the rows a sequence of this launch has on average.
template <int HD, int ES, bool BF>
int split_rows(cudaStream_t st, int dev, int sms, const paged::AttendArgs& a, const Workspace& ws, int64_t most) {
    const int64_t rows = std::min<int64_t>((static_cast<int64_t>(a.c.n_tokens) + a.c.B - 1) / a.c.B * a.p.G, a.p.rows_max);
    if (rows <= 8) return launch_split<HD, ES, BF, 1>(st, dev, sms, a, ws, most);
    if constexpr (HD <= 128)
        if (rows > 16) return launch_split<HD, ES, BF, 4>(st, dev, sms, a, ws, most);
    return launch_split<HD, ES, BF, 2>(st, dev, sms, a, ws, most);
}

template <int HD>
int split_hd(cudaStream_t st, int dev, int sms, const paged::AttendArgs& a, const Workspace& ws, int cache_type,
             int64_t most) {
    if (cache_type == DGEN_TYPE_E4M3) return split_rows<HD, 1, false>(st, dev, sms, a, ws, most);
    if (cache_type == DGEN_TYPE_BF16) return split_rows<HD, 2, true>(st, dev, sms, a, ws, most);
    return split_rows<HD, 2, false>(st, dev, sms, a, ws, most);
}

// Rows per KV head of one sequence above which the tcgen05 kernel takes it, although its tiles hold 128: it
// reads the keys once for all of them (and rounds each weight once, where the split kernel keeps about 16 bits).
// Split kernel / tcgen05 kernel in us, 8 KV heads, lengths of 4,352 keys in 16 sequences (and one of 301):
// hd 128, 8 rows 51 / 50 (9.8 / 11.1), 16 rows 57 / 51 (13.9 / 11.1), 24 rows 100 / 52; hd 256, 8 rows 99 / 91
// (12.9 / 15.5), 16 rows 111 / 94 (19.7 / 15.5), 24 rows 195 / 94; hd 64, whose short rows the split kernel
// streams with more warps, 16 rows 37 / 43 (10.7 / 14.0), 24 rows 53 / 42 (14.0 / 14.1).  No count serves every
// length at hd 64: 64 sequences of 16 rows over 8,192 keys take 101 / 149, one of 12 rows over 40,000 45 / 33.
constexpr int block_min_rows(int hd) { return hd >= 128 ? 8 : 16; }

// Whether the tcgen05 kernel can take this call's long sequences: 16-bit cache, a
// group that fits a row tile, pages that TMA boxes of 8 rows or more divide, and
// rows and coordinates within a tensor map's reach.
bool block_fits(const dgen_paged_cache* c, const paged::AttendArgs& a) {
    const int64_t rows = static_cast<int64_t>(c->n_pages) * c->n_kv_heads * c->page_size;
    return c->type != DGEN_TYPE_E4M3 && a.p.G <= paged::kBlkRows && c->page_size % 8 == 0 && rows <= INT32_MAX &&
           (a.c.n_tokens == 1 || a.q.ts > 0) && (a.Hq == 1 || a.q.hs > 0);
}

bool encode_16bit(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
    const cuuint32_t es[3] = {1, 1, 1};
    // (bits are copied, not computed with: one 16-bit type serves both)
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF>
int launch_block(cudaStream_t st, int dev, int sms, paged::AttendArgs a, const Workspace& ws) {
    using L = paged::BlockLayout<HD>;
    if (!load_encode()) return DGEN_ECUDA;
    const int tokens = paged::kBlkRows / a.p.G;  // per row tile
    a.p.R = tokens * a.p.G;
    a.p.KB = a.p.align = paged::kBlkKeys;
    a.p.log2_kb = 7;
    int log2_br = 3;
    while ((1 << log2_br) < L::VR && a.c.page % (2 << log2_br) == 0) ++log2_br;  // box rows: at most a V stage's
    CUtensorMap tq, tk, tv;
    {
        const cuuint64_t ts = a.c.n_tokens > 1 ? a.q.ts * 2 : static_cast<cuuint64_t>(a.Hq) * HD * 2;
        const cuuint64_t hs = a.Hq > 1 ? a.q.hs * 2 : HD * 2;
        const cuuint64_t dims[3] = {HD, static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.c.n_tokens)};
        const cuuint64_t strides[2] = {hs, ts};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.p.G), static_cast<cuuint32_t>(tokens)};
        const cuuint64_t kdims[2] = {HD, static_cast<cuuint64_t>(a.c.n_pages) * a.c.Hkv * a.c.page};
        const cuuint64_t kstrides[1] = {HD * 2};
        const cuuint32_t kbox[2] = {64, 1u << log2_br};
        if (!encode_16bit(&tq, a.q.p, 3, dims, strides, box) || !encode_16bit(&tk, a.c.k, 2, kdims, kstrides, kbox) ||
            !encode_16bit(&tv, a.c.v, 2, kdims, kstrides, kbox))
            return DGEN_EINVAL;
    }
    // teams of 4 or 2 row tiles where the average sequence's tiles fill them to 7/8 (eight canvases of 256 tokens
    // over 4,352 keys: 132 us in fours, 145 in twos or alone; even chunks of 1,024 tokens 699, 719, 731); of 2 at most
    // for a ragged batch, whose last teams have idle members (ragged chunks 289 us in twos, 307 in fours, 293 alone)
    const int64_t rows = static_cast<int64_t>(a.c.n_tokens) * a.p.G;
    const int64_t avg = std::max<int64_t>(1, (rows / a.c.B + a.p.R - 1) / a.p.R);
    a.p.TS = 1;
    for (int ts : {4, 2})
        if (a.p.TS == 1 && (ts == 2 || !a.c.cu) && 8 * avg >= 7 * ((avg + ts - 1) / ts * ts)) a.p.TS = ts;
    a.p.tokens = tokens * a.p.TS;
    a.p.unit_cost = 4;
    const int64_t units = std::min<int64_t>(rows, rows / (a.p.R * a.p.TS) + a.c.B) * a.c.Hkv;
    const int64_t blocks = (static_cast<int64_t>(a.c.table_pages) * a.c.page + 2 * paged::kBlkKeys - 2) / paged::kBlkKeys;
    if (units * (blocks + 4) >= kMaxLine) return DGEN_EINVAL;
    const int64_t teams = std::max<int64_t>(1, std::min<int64_t>(std::min(sms, kMaxGrid) / a.p.TS, units * blocks));
    const int64_t grid = teams * a.p.TS;
    if (2 * static_cast<size_t>(grid) * paged::kBlkRows * (HD + 2) > ws.floats) return DGEN_ESCRATCH;
    const paged::Cap cap = paged::cap_form(a.scale, a.cap);
    auto kern = cap == paged::Cap::none    ? paged::paged_block_kernel<HD, BF, paged::Cap::none>
                : cap == paged::Cap::usual ? paged::paged_block_kernel<HD, BF, paged::Cap::usual>
                                           : paged::paged_block_kernel<HD, BF, paged::Cap::any>;
    a.joins = ws.joins;
    set_smem_attr_once(kern, L::SMEM_BYTES, dev);
    a.parts = ws.parts;
    a.n_ctas = static_cast<int>(grid);
    if (launch_ex(st, kern, dim3(a.n_ctas), dim3(L::THREADS), L::SMEM_BYTES, tq, tk, tv, a, log2_br, ws.err) !=
        cudaSuccess)
        return DGEN_ECUDA;
    if (teams == 1) return DGEN_OK;
    return launch_ex(st, paged::paged_block_join_kernel<HD, BF>, dim3(a.n_ctas, HD / paged::kJoinCols), dim3(256), 0, a,
                     static_cast<const int*>(ws.err)) == cudaSuccess
               ? DGEN_OK
               : DGEN_ECUDA;
}

// Sequences with more than block_min_rows query rows per KV head go to the tcgen05
// kernel, the others to the split kernel; a ragged batch may hold both kinds, and
// each launch passes over the other's.
template <int HD>
int attend_hd(cudaStream_t st, int dev, int sms, const dgen_paged_cache* c, paged::AttendArgs a, const Workspace& ws) {
    // the most rows one sequence has if none is without a new token (where some are, the split kernel also
    // takes longer ones): a decode batch given with cu_new costs no second launch
    const int64_t most = (a.c.cu ? std::max(a.c.n_tokens - a.c.B + 1, 1) : a.c.n_uniform) * static_cast<int64_t>(a.p.G);
    constexpr int min_rows = block_min_rows(HD);
    const bool block = block_fits(c, a) && most > min_rows;
    if (block) {
        paged::AttendArgs b = a;
        b.p.rows_min = min_rows + 1;
        const int rc = c->type == DGEN_TYPE_BF16 ? launch_block<HD, true>(st, dev, sms, b, ws)
                                                 : launch_block<HD, false>(st, dev, sms, b, ws);
        // (a single token's rows alone can pass the limit: then no sequence is left)
        if (rc != DGEN_OK || !a.c.cu || a.p.G > min_rows) return rc;
        a.p.rows_max = min_rows;
    }
    return split_hd<HD>(st, dev, sms, a, ws, c->type, std::min<int64_t>(most, a.p.rows_max));
}

int append(const dgen_paged_cache* cache, int32_t n_tokens, const int32_t* cu, int32_t type, const dgen_token_rows* k,
           const dgen_token_rows* v, int32_t n_q_heads, const dgen_token_rows* q, const dgen_token_rows* q_out,
           float rope_base, void* stream) {
    const int rc = check_cache(cache, n_tokens, cu);
    if (rc != DGEN_OK) return rc;
    if (type != DGEN_TYPE_BF16 && type != DGEN_TYPE_F16) return DGEN_EINVAL;
    if (cache->type != DGEN_TYPE_E4M3 && cache->type != type) return DGEN_EINVAL;
    if (n_q_heads < 0 || n_q_heads > kMaxHeads || !(rope_base >= 0.f) || std::isinf(rope_base)) return DGEN_EINVAL;
    if (n_tokens == 0) return DGEN_OK;
    if (!good_rows(k, n_tokens, cache->n_kv_heads) || !good_rows(v, n_tokens, cache->n_kv_heads)) return DGEN_EINVAL;
    if ((n_q_heads > 0) != (q != nullptr) || !q != !q_out) return DGEN_EINVAL;
    if (q && (!good_rows(q, n_tokens, n_q_heads) || !good_rows_out(q_out, n_tokens, n_q_heads, cache->head_dim)))
        return DGEN_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DGEN_ECUDA;
    const int sms = sm_count(dev);
    if (sms < 1) return DGEN_ECUDA;
    paged::AppendArgs a{};
    a.c = view(cache, n_tokens, cu);
    a.k = view(k);
    a.v = view(v);
    a.Hq = n_q_heads;
    if (q) {
        a.q = view(q);
        a.q_out = view(q_out);
    }
    a.rotate = rope_base > 0.f;
    a.log2_base = a.rotate ? std::log2(static_cast<double>(rope_base)) : 0.0;
    // Tokens per block: up to four items a thread (2,048 tokens of 32 rows of 256 took 16 us at two a block, 19 at
    // six) and three blocks an SM (1,000 tokens of 40 rows of 64: 4.6 us at three a block, 6.0 at one, 6.6 at
    // six); more for very many tokens, whose blocks' lookups then cost less.
    const int items = (n_q_heads + 2 * cache->n_kv_heads) * (cache->head_dim / 16);
    const int per_block = std::clamp(std::max(std::min(4 * paged::kAppendThreads / items, n_tokens / (3 * sms)),
                                              n_tokens / (16 * sms)), 1, paged::kAppendTokens);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf = type == DGEN_TYPE_BF16, e4 = cache->type == DGEN_TYPE_E4M3;
    if (cache->head_dim == 64) return append_hd<64>(st, a, per_block, bf, e4);
    if (cache->head_dim == 128) return append_hd<128>(st, a, per_block, bf, e4);
    return append_hd<256>(st, a, per_block, bf, e4);
}

int attend(const dgen_paged_cache* cache, int32_t n_tokens, const int32_t* cu, int32_t type, int32_t n_q_heads,
           const dgen_token_rows* q, const dgen_token_rows* out, float scale, int32_t causal, int32_t window, float cap,
           float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    const int rc = check_cache(cache, n_tokens, cu);
    if (rc != DGEN_OK) return rc;
    if (type != DGEN_TYPE_BF16 && type != DGEN_TYPE_F16) return DGEN_EINVAL;
    if (cache->type != DGEN_TYPE_E4M3 && cache->type != type) return DGEN_EINVAL;
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return DGEN_EINVAL;
    if (static_cast<int64_t>(n_tokens) * n_q_heads > INT32_MAX) return DGEN_EINVAL;
    if (!std::isfinite(scale * paged::kLog2e) || !(scale > 0.f) || !(cap >= 0.f) || std::isinf(cap) || window < 0 || (causal != 0 && causal != 1))
        return DGEN_EINVAL;
    if (n_tokens == 0) return DGEN_OK;
    if (!good_rows(q, n_tokens, n_q_heads) || !good_rows_out(out, n_tokens, n_q_heads, cache->head_dim)) return DGEN_EINVAL;
    if (!aligned16(workspace) || !aligned4(lse)) return DGEN_EINVAL;
    if (workspace_bytes < static_cast<int64_t>(kHeadBytes)) return DGEN_ESCRATCH;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DGEN_ECUDA;
    const int sms = std::min(sm_count(dev), kMaxSms);
    if (sms < 1) return DGEN_ECUDA;
    paged::AttendArgs a{};
    a.c = view(cache, n_tokens, cu);
    a.q = view(q);
    a.out = view(out);
    a.p.G = n_q_heads / cache->n_kv_heads;
    a.p.causal = causal;
    a.p.window = window;
    a.p.rows_min = 1;
    a.p.rows_max = INT32_MAX;
    a.lse = lse;
    a.Hq = n_q_heads;
    a.scale = scale;
    // Within 2^-100 .. 2^126 the kernels' factors stay in fp32's range; a cap beyond acts as the nearer limit does:
    // scores below 2^-100 weigh alike, and those that 2^126 bends are so far apart that one key takes all.
    a.cap = cap > 0.f ? std::clamp(cap, 0x1p-100f, 0x1p126f) : 0.f;
    a.q_bf16 = type == DGEN_TYPE_BF16;
    Workspace ws{static_cast<unsigned int*>(workspace), static_cast<int*>(workspace) + kMaxGrid,
                 reinterpret_cast<paged::Piece*>(static_cast<uint8_t*>(workspace) + kCounterBytes),
                 reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeadBytes),
                 (static_cast<size_t>(workspace_bytes) - kHeadBytes) / sizeof(float)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->head_dim == 64) return attend_hd<64>(st, dev, sms, cache, a, ws);
    if (cache->head_dim == 128) return attend_hd<128>(st, dev, sms, cache, a, ws);
    return attend_hd<256>(st, dev, sms, cache, a, ws);
}

}  // namespace

extern "C" {

int dgen_paged_append(const dgen_paged_cache* cache, int32_t n_tokens, const int32_t* cu_new_dev_or_null, int32_t type,
                      const dgen_token_rows* k, const dgen_token_rows* v, int32_t n_q_heads,
                      const dgen_token_rows* q_or_null, const dgen_token_rows* q_out_or_null, float rope_base,
                      void* stream) {
    try {
        return append(cache, n_tokens, cu_new_dev_or_null, type, k, v, n_q_heads, q_or_null, q_out_or_null, rope_base,
                      stream);
    } catch (...) {
        return DGEN_ENOMEM;
    }
}

int dgen_paged_attention(const dgen_paged_cache* cache, int32_t n_tokens, const int32_t* cu_new_dev_or_null,
                         int32_t type, int32_t n_q_heads, const dgen_token_rows* q, const dgen_token_rows* out,
                         float scale, int32_t causal, int32_t window, float cap, float* lse_dev_or_null,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    try {
        return attend(cache, n_tokens, cu_new_dev_or_null, type, n_q_heads, q, out, scale, causal, window, cap,
                      lse_dev_or_null, workspace, workspace_bytes, stream);
    } catch (...) {
        return DGEN_ENOMEM;
    }
}

int64_t dgen_paged_workspace_bytes(void) {
    // two partial results per CTA of the largest launch (128 rows x (256 + 2) floats each)
    return static_cast<int64_t>(kHeadBytes) + int64_t{2} * kMaxSms * paged::kBlkRows * 258 * 4;
}

int dgen_paged_synchronize(void* workspace, void* stream) {
    if (!aligned16(workspace)) return DGEN_EINVAL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* word = static_cast<int*>(workspace) + kMaxGrid;
    int err = 0;
    if (cudaMemcpyAsync(&err, word, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return DGEN_ECUDA;
    if (err == 0) return DGEN_OK;
    // the call that gave up may have left its counters in between and its join list unfinished
    if (cudaMemsetAsync(workspace, 0, kHeadBytes, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return DGEN_ECUDA;
    return DGEN_EDEVICE;
}

}  // extern "C"
