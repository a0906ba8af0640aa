// kt_attn_split.cu -- attention over a paged cache for few query rows: every
// warp streams its own keys and values and keeps its own softmax state.
//
// An item is (sequence, cache head, 16 query rows; of an 8-bit cache 8 for calls of
// up to 8 rows): row r of a sequence is its new token r / group under query head
// r % group of the cache head's group, so the heads that share a cache head share
// its loads.  A warp takes blocks of 16
// keys (32 for heads of up to 64: the same bytes), through a ring of TMA loads
// of its own: no barrier among warps until the item's end.  S = Q K^T and P V
// are mma.sync products of 16 rows: the operator is bound by reading the cache
// (16 flops a byte for 8 heads a cache head), which they keep up with, and their
// latency is a warp's, where a tensor-memory tile's would be a CTA's.  P goes into
// the product with V in two parts of the element type, P rounded to it and the
// remainder rounded to it (16 bits of P in bf16, 22 in fp16): the tensor cores wait
// for the cache anyway, so that the second product costs 0 to 1.5 % of a large
// cache's time and 3 % of a short one's (one part, the other way: 207 against 209
// us, 10.1 against 10.3), and the error is that of fp32 and the result's rounding.
//
// Few items are cut into pieces that each have a CTA of their own; many lie on a
// line that is cut into equal runs, so that one long sequence and many short ones
// keep the GPU equally busy.  A cut item leaves partial sums (maximum, sum,
// unnormalised output) in the workspace, and the CTA that finishes last joins
// them in order, so the result does not depend on which one that was.
//
// Measured on GB300, machines differing: 64 single tokens after up to 8191, bf16,
// 64 / 8 heads of 128 (1.31 GB of cache), 208 to 216 us, 6.1 to 6.3 TB/s (90 to 93 %
// of the measured copy rate); 4 after up to 131071, fp16, heads of 64 (0.59 GB), 109
// to 119 us, 4.9 to 5.4 TB/s, of which about 10 us are the launch, the plan and the
// join.  One token after 500 keys: 10.3 us, of which 0.5 launch, 1.7 plan, 1.7 first
// look-ups and loads, 2 the keys, 3.5 the pieces' join (timed when it took 10.0);
// after 60 (no join) 6.1 us.  L2 promotion past a head's row (256 bytes for rows of
// 128) read 1.39 times the cache.
// Over 8-bit caches: 64 single tokens after up to 16383, bf16, 64 / 8 heads of 128
// (1.45 GB), 222 to 232 us on different machines, 6.3 to 6.6 TB/s (93 to 97 %); 4
// after up to 131071, fp16, heads of 64 (0.29 GB), 68 us, 4.3 TB/s; one after 700
// keys, 10.9 us.  The heads of 64 are bound by latency: issue slots 51 %, ALU 47 %,
// DRAM 53 %, tensor pipe 19 %, no unit full; a warp waits 1.4 cycles an instruction
// for its own last one, 0.6 for loads, 0.4 for a busy unit.
#include <algorithm>
#include <type_traits>

#include "kt_attn_dev.cuh"

namespace kt {

constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = kSplitWarps * 32;
constexpr int kSplitKeys = 16;                          // keys of one load (pages hold a multiple of it)
constexpr int kSplitMinUnits = 2;                       // least units of a piece
constexpr int kSplitItemUnits = 3;                      // what an item costs besides its units, in units
constexpr int kSplitJoinUnits = 4;                      // what cutting an item costs its last CTA, in units

template <int DP, bool KV8, int ROWS>
struct SplitCfg {
    static constexpr int kRows = ROWS;                               // query rows of an item: 16, or 8 (KV8)
    static constexpr int kSub = (DP == 128 ? 1 : 2) * (KV8 ? 2 : 1);   // loads of K and of V that make a warp's block
    static constexpr int kBlockKeys = kSub * kSplitKeys;
    static constexpr int kUnit = kSplitWarps * kBlockKeys;           // keys of one unit
    static constexpr int kRowBytes = DP * (KV8 ? 1 : 2);             // of a key in a block
    static constexpr int kBlockBytes = kBlockKeys * kRowBytes;       // one of K, V
    // KV8 heads of 64 wait for the chain of a block's instructions, which more warps hide (4 x 131k keys: 67 us with
    // three CTAs an SM, 71 with two), of 128 for the loads (64 single tokens: 222 us with two CTAs, 234 with three,
    // whose rings are smaller)
    static constexpr int kCtasPerSm = ROWS == 8 && DP == 64 ? 3 : 2;
    static constexpr int kStages = kCtasPerSm == 3 ? 2 : 3;          // 24 KB a warp, or 16
    static constexpr int kRing = kStages * 2 * kBlockBytes;          // per warp
    static constexpr int kMaxCtas = kSplitWarps * kRing / (kRows * 8);   // what a join of all of them has room for
    static constexpr int kSmem = kSplitWarps * kRing + 1024;
    static constexpr int kMergeRow = DP + 8;                         // floats of a row: rows start 8 banks apart
    static constexpr int kMergeBytes = kSplitWarps * kRows * kMergeRow * 4;
    static constexpr int kParts = kRows * DP / 4 / kSplitThreads;   // float4 per thread of an item's rows
};

struct SplitParams {
    AttnShape sh;
    const void* q;
    void* out;
    long long q_token, q_head, o_token, o_head;
    float4* part_o;      // [CTAs][2][16][DP / 4]
    float2* part_ml;     // [CTAs][2][16]
    unsigned* counters;  // [CTAs]
};

// Keys that the rows of row tile rt see: [lo, hi); units of the item (at least one, so that its rows are written).
struct SplitItem {
    int lo, hi, unit0, units;
};
template <typename Cfg>
__device__ __forceinline__ SplitItem split_item(const AttnShape& s, const SeqInfo& q, int rt) {
    constexpr int unit = Cfg::kUnit;
    SplitItem it;
    const int t0 = rt * Cfg::kRows / s.group;
    const int t1 = min((rt * Cfg::kRows + Cfg::kRows - 1) / s.group, q.q_len - 1);
    it.hi = max(0, min(q.first_pos + t1 + 1, q.keys));
    it.lo = window_start(q.first_pos + t0, s.window);
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.unit0 = it.lo / unit;
    it.units = max(1, (it.hi + unit - 1) / unit - it.unit0);
    return it;
}
template <typename Cfg>
__device__ __forceinline__ int split_row_tiles(const AttnShape& s, const SeqInfo& q) {
    return (q.q_len * s.group + Cfg::kRows - 1) / Cfg::kRows;
}

// The order of the CTAs.  A slot's heads lie side by side in memory, and a head's row of an 8-bit cache is 128 bytes at
// most: read at different times, such rows come at 5.5 TB/s (64 single tokens after up to 16383, 8 heads of 128:
// 264 us), where each head's slots follow one another at 6.7.  So there the runs are those of one head, and
// neighbouring CTAs take the same run of neighbouring heads (234), unless there are so many heads that CTAs would be
// left over.
struct SplitOrder {
    int runs;         // CTAs that share a line
    int heads;        // cache heads on a line
    int run, head;    // this CTA's
    int step, first;  // CTA of run r of the line: r * step + first
};
template <bool KV8>
__device__ __forceinline__ SplitOrder split_order(const AttnShape& s) {
    const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
    if (!KV8 || s.kv_heads * 8 > ctas) return SplitOrder{ctas, s.kv_heads, cta, 0, 1, 0};
    return SplitOrder{ctas / s.kv_heads, 1, cta / s.kv_heads, cta % s.kv_heads, s.kv_heads, cta % s.kv_heads};
}

// How the items are dealt to the CTAs of a line.  Few items: each is cut into pieces of at most `piece` units, a CTA
// takes one piece (piece > 0).  Many: they lie on a line, kSplitItemUnits before each one's units, that is cut into
// equal runs (piece == 0).  In both, [begin, begin + per) of `total` are this CTA's, in pieces or in units of the line.
struct SplitPlan {
    long long total, per, begin;
    long long in_seq;   // begin's place in sequence seq
    int piece, seq;
};
__device__ __forceinline__ int pieces_of(int units, int piece) { return (units + piece - 1) / piece; }
__device__ __forceinline__ int item_measure(const SplitItem& it, int piece) {
    return piece > 0 ? pieces_of(it.units, piece) : it.units + kSplitItemUnits;
}
template <typename Cfg>
__device__ __forceinline__ long long seq_measure(const AttnShape& s, int b, int piece, int heads) {
    const SeqInfo q = seq_info(s, b);
    const int tiles = split_row_tiles<Cfg>(s, q);
    long long n = 0;
    for (int rt = 0; rt < tiles; ++rt) n += item_measure(split_item<Cfg>(s, q, rt), piece);
    return n * heads;
}

// All threads of the CTA; `shared` is theirs.
template <typename Cfg>
__device__ __forceinline__ SplitPlan split_plan(const AttnShape& s, const SplitOrder& order, SplitPlan* shared) {
    __shared__ long long s_units[kSplitWarps], s_items[kSplitWarps];
    __shared__ int s_most[kSplitWarps];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    long long units = 0, items = 0;
    int most = 0;
    for (int b = tid; b < s.seqs; b += kSplitThreads) {
        const SeqInfo q = seq_info(s, b);
        const int tiles = split_row_tiles<Cfg>(s, q);
        for (int rt = 0; rt < tiles; ++rt) {
            const int n = split_item<Cfg>(s, q, rt).units;
            units += n;
            most = max(most, n);
        }
        items += tiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        units += __shfl_xor_sync(0xffffffffu, units, o);
        items += __shfl_xor_sync(0xffffffffu, items, o);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        s_units[warp] = units;
        s_items[warp] = items;
        s_most[warp] = most;
    }
    __syncthreads();
    units = items = 0;
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) {
        units += s_units[w];
        items += s_items[w];
        most = max(most, s_most[w]);
    }
    units *= order.heads;
    items *= order.heads;
    const long long ctas = order.runs;
    const long long line = units + items * kSplitItemUnits;
    const long long run = (line + ctas - 1) / ctas;
    int piece = 0;
    if (items <= ctas) {
        // sum of ceil(u / piece) <= units / piece + items <= CTAs
        const long long even = ctas > items ? (units + ctas - items - 1) / (ctas - items) : most;
        const long long least = even < most ? (even > kSplitMinUnits ? even : kSplitMinUnits) : most;
        if (least <= run + kSplitJoinUnits) piece = static_cast<int>(least);
    }
    SplitPlan plan;
    plan.piece = piece;
    plan.per = piece > 0 ? 1 : (run > kSplitItemUnits + kSplitMinUnits ? run : kSplitItemUnits + kSplitMinUnits);
    plan.begin = plan.per * order.run;
    // the sequence of this CTA's first piece or unit
    if (tid == 0) shared->seq = s.seqs;
    long long before = 0;
    for (int b0 = 0; b0 < s.seqs; b0 += kSplitThreads) {
        const long long n = b0 + tid < s.seqs ? seq_measure<Cfg>(s, b0 + tid, piece, order.heads) : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();
        if (lane == 31) s_units[warp] = incl;
        __syncthreads();
        long long prefix = before;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
            if (w < warp) prefix += s_units[w];
            before += s_units[w];
        }
        if (plan.begin >= prefix + incl - n && plan.begin < prefix + incl) {
            shared->seq = b0 + tid;
            shared->in_seq = plan.begin - (prefix + incl - n);
        }
        if (before > plan.begin) break;   // the same for every thread
    }
    __syncthreads();
    plan.total = piece > 0 ? before : line;   // (pieces: only whether begin lies below it counts)
    plan.seq = shared->seq;
    plan.in_seq = shared->in_seq;
    return plan;
}

// Address of 16-byte piece `piece` of key `row` in 16 keys of an 8-bit block at `base`, as TMA's swizzle leaves it.
template <int DP>
__device__ __forceinline__ uint32_t piece8(uint32_t base, int row, int piece) {
    return DP == 128 ? base + row * 128 + ((piece ^ (row & 7)) << 4)
                     : base + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

// KV8: the cache's elements are e4m3 codes with a power of two for 16 keys of a head.  The products are fp16 ones,
// which e4m3 has a conversion to (bf16 has none: bits moved by hand take 2.2 instructions an element, and 265 us for 64
// single tokens after up to 16383): codes go in without their powers, exact; bf16 queries times a power of two per row,
// exact down to 2^-31 of the row's largest element and off by at most 2^-39 of that below; softmax weights, their
// value's power included, relative to the largest of the row in the block's 32 or 64 keys, times 2^10: rounded to 11
// bits down to 2^-24 of that largest and off by at most 2^-35 of it below.  For fp16 results, which have as many bits,
// the weights go in in two parts (error 1.00 times that of rounding the result once; in one part up to 1.40, for 5 us
// less of 4 tokens after up to 131071 under heads of 64).
constexpr float kWeightLog2 = 10.0f;   // the largest weight of a block, log2; O stays multiplied by that to the end
constexpr float kLeastShareLog2 = -125.0f;   // (a unit above what ex2 flushes)
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// Codes 0 and 1 (in `lo`), 2 and 3 as pairs of fp16.
__device__ __forceinline__ void widen_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<unsigned short>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<unsigned short>(w >> 16)));
}

template <typename T, int DP, bool KV8, int ROWS>
__global__ void __launch_bounds__(kSplitThreads, SplitCfg<DP, KV8, ROWS>::kCtasPerSm)
    attn_split_kernel(const SplitParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Cfg = SplitCfg<DP, KV8, ROWS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kSplitWarps][Cfg::kStages];
    __shared__ int s_abort, s_last;
    __shared__ float2 s_ml[kSplitWarps][Cfg::kRows];
    __shared__ SplitPlan s_plan;
    __shared__ uint32_t s_scales[KV8 ? kSplitWarps : 1][Cfg::kStages][Cfg::kSub];   // of keys, of values << 8
    const AttnShape& sh = p.sh;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    uint8_t* ring_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = ring_base + warp * Cfg::kRing;
    float* merge = reinterpret_cast<float*>(ring_base);   // [warps][16][kMergeRow], once every warp has left its ring

    if (tid == 0) {
        s_abort = 0;
        for (int w = 0; w < kSplitWarps; ++w)
            for (int i = 0; i < Cfg::kStages; ++i) mbar_init(smem_u32(&s_full[w][i]), 1);
        fence_mbar_init();
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    griddep_wait();
    griddep_launch_dependents();
    const SplitOrder order = split_order<KV8>(sh);
    const SplitPlan plan = split_plan<Cfg>(sh, order, &s_plan);
    if (plan.seq >= sh.seqs) return;

    // ---- the item of this CTA's first piece or unit
    int b = plan.seq, rt = 0;
    SeqInfo sq = seq_info(sh, b);
    int row_tiles = split_row_tiles<Cfg>(sh, sq);
    SplitItem it = split_item<Cfg>(sh, sq, 0);
    long long at = plan.in_seq;
    while (at >= static_cast<long long>(item_measure(it, plan.piece)) * order.heads) {
        at -= static_cast<long long>(item_measure(it, plan.piece)) * order.heads;
        it = split_item<Cfg>(sh, sq, ++rt);
    }
    int hl, u0, u1;                // cache head of the line; the item's units in this run
    long long first = 0;           // line: the item's first unit
    const long long end = plan.begin + plan.per;
    {
        const int n = item_measure(it, plan.piece);
        hl = at >> 31 == 0 ? static_cast<int>(at) / n : static_cast<int>(at / n);
        const int in = static_cast<int>(at - static_cast<long long>(hl) * n);
        if (plan.piece > 0) {
            const int chunk = (it.units + n - 1) / n;   // the pieces of an item alike
            u0 = in * chunk;
            u1 = min(it.units, u0 + chunk);
        } else {
            first = plan.begin - in + kSplitItemUnits;
            u0 = max(in - kSplitItemUnits, 0);
            u1 = static_cast<int>(min(end - first, static_cast<long long>(it.units)));
        }
    }
    uint32_t loads = 0;            // blocks this warp has consumed so far
    bool gave_up = false;          // a wait ran out: the warp loads nothing more, but takes part in joins and counters
    const bool withhold = sh.withhold != 0 && blockIdx.x == 0 && warp == 0;
    const uint64_t policy = l2_policy_evict_first();   // 64 single tokens: 211 us, 215 without
    while (true) {
        if (u1 > u0) {
        const int32_t* pages = sh.block_table + b * sh.table_stride;
        const int h = order.head + hl;

        // ---- this warp's blocks: keys base + kUnit i, i in [i0, i1)
        const int base = (it.unit0 + u0) * Cfg::kUnit + warp * Cfg::kBlockKeys;
        int i0 = 0, i1 = u1 - u0;
        while (i0 < i1 && base + i0 * Cfg::kUnit + Cfg::kBlockKeys <= it.lo) ++i0;
        while (i1 > i0 && base + (i1 - 1) * Cfg::kUnit >= it.hi) --i1;
        if (gave_up) i1 = i0;
        int page_batch = -1, my_page = -1, my_slot = 0;
        uint32_t my_scales = 127u;   // nothing there: the values' power is the least
        auto issue = [&](int i) {   // whole warp; block i into its stage
            if (withhold && loads == 0 && i == i0) return;   // test hook
            // lanes look up the pages of the next 32 loads at a time
            const int batch = (i - i0) / (32 / Cfg::kSub);
            if (batch != page_batch) {
                page_batch = batch;
                const int mine = i0 + batch * (32 / Cfg::kSub) + lane / Cfg::kSub;
                const int key = base + mine * Cfg::kUnit + lane % Cfg::kSub * kSplitKeys;
                my_page = -1;
                my_slot = 0;
                my_scales = 127u;
                // (16 keys that no row sees, past them all or before the window: zeros from outside the cache)
                if (mine < i1 && key < it.hi && key + kSplitKeys > it.lo) {
                    my_page = checked_page(sh, pages, key);
                    my_slot = key % sh.page_size;
                    if (KV8 && my_page >= 0) {
                        const long long at = (static_cast<long long>(my_page) * (sh.page_size / KT_KV8_BLOCK) +
                                              my_slot / KT_KV8_BLOCK) * sh.kv_heads + h;
                        my_scales = sh.k_scales[at] | static_cast<uint32_t>(sh.v_scales[at]) << 8;
                    }
                }
            }
            const uint32_t st = (loads + static_cast<uint32_t>(i - i0)) % Cfg::kStages;
            const uint32_t bar = smem_u32(&s_full[warp][st]);
            const uint32_t k = smem_u32(ring + st * 2 * Cfg::kBlockBytes);
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * Cfg::kBlockBytes);
#pragma unroll
            for (int sub = 0; sub < Cfg::kSub; ++sub) {
                const int src = (i - i0) % (32 / Cfg::kSub) * Cfg::kSub + sub;
                const int page = __shfl_sync(0xffffffffu, my_page, src);
                const int slot = __shfl_sync(0xffffffffu, my_slot, src);
                if constexpr (KV8) {
                    const uint32_t scales = __shfl_sync(0xffffffffu, my_scales, src);
                    if (lane == 0) {
                        s_scales[warp][st][sub] = scales;
                        const uint32_t at_block = sub * kSplitKeys * DP;
                        tma_load_4d_once(k + at_block, &kmap, bar, 0, slot, h, page, policy);
                        tma_load_4d_once(k + Cfg::kBlockBytes + at_block, &vmap, bar, 0, slot, h, page, policy);
                    }
                } else if (lane == 0) {
#pragma unroll
                    for (int x = 0; x < DP; x += 64) {
                        const uint32_t at_block = (x * Cfg::kBlockKeys + sub * kSplitKeys * 64) * 2;
                        tma_load_4d_once(k + at_block, &kmap, bar, x, slot, h, page, policy);
                        tma_load_4d_once(k + Cfg::kBlockBytes + at_block, &vmap, bar, x, slot, h, page, policy);
                    }
                }
            }
        };
        const int n_blocks = i1 - i0;
        for (int i = 0; i < min(n_blocks, Cfg::kStages); ++i) issue(i0 + i);
        if (KV8) __syncwarp();   // the scales of those blocks

        auto block_ready = [&](int i) -> bool {   // whole warp
            const uint32_t seq_no = loads + static_cast<uint32_t>(i - i0);
            const uint32_t st = seq_no % Cfg::kStages;
            if (warp_wait(smem_u32(&s_full[warp][st]), (seq_no / Cfg::kStages) & 1u, &s_abort, sh.wait_limit_ns))
                return true;
            if (lane == 0 && !*reinterpret_cast<volatile int*>(&s_abort)) {
                s_abort = 1;
                set_error(sh.err, KT_DEVERR_TIMEOUT_LOAD);
            }
            // loads still in flight land before their memory has another use (each wait bounded)
            int never = 0;
            for (int k = i; k < min(i + Cfg::kStages, i1); ++k) {
                const uint32_t no = loads + static_cast<uint32_t>(k - i0);
                mbar_wait(smem_u32(&s_full[warp][no % Cfg::kStages]), (no / Cfg::kStages) & 1u, &never, kDrainLimitNs);
            }
            gave_up = true;
            return false;
        };
        const int g = lane >> 2, t4 = lane & 3;
        const int rows = min(Cfg::kRows, sq.q_len * sh.group - rt * Cfg::kRows);   // of the tile that hold tokens
        float* const mo = merge + warp * Cfg::kRows * Cfg::kMergeRow;
        if constexpr (!KV8) {
        // ---- queries: rows g and g + 8 of the tile in the MMA's A layout
        uint32_t qa[DP / 16][4];
        int last_key[2], first_key[2];   // what the row sees; rows of no token need no mask
        {
            const T* qp[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = rt * Cfg::kRows + g + 8 * e;
                const int tok = row / sh.group;
                const bool ok = tok < sq.q_len;
                last_key[e] = ok ? min(sq.first_pos + tok, sq.keys - 1) : 0x7fffffff;
                first_key[e] = ok ? window_start(sq.first_pos + tok, sh.window) : 0;
                qp[e] = ok ? static_cast<const T*>(p.q) + static_cast<long long>(sq.first_token + tok) * p.q_token +
                                 static_cast<long long>(h * sh.group + row - tok * sh.group) * p.q_head
                           : nullptr;
            }
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int d = ks * 16 + t4 * 2 + (f >> 1) * 8;
                    const T* src = qp[f & 1];
                    qa[ks][f] = src != nullptr && d < sh.head_dim ? *reinterpret_cast<const uint32_t*>(src + d) : 0u;
                }
        }

        float o[DP / 8][4];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int f = 0; f < 4; ++f) o[n][f] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        for (int i = i0; i < i1; ++i) {
            if (!block_ready(i)) break;
            const uint32_t st = (loads + static_cast<uint32_t>(i - i0)) % Cfg::kStages;
            const uint32_t kb = smem_u32(ring + st * 2 * Cfg::kBlockBytes);
            const uint32_t vb = kb + Cfg::kBlockBytes;
            const int key0 = base + i * Cfg::kUnit;

            // ---- S = Q K^T, 16 rows x kBlockKeys keys; two chains per product where there are few products
            constexpr int kCols = 2 * Cfg::kSub, kChains = Cfg::kSub == 1 ? 2 : 1;
            float sc[kChains][kCols][4];
#pragma unroll
            for (int c = 0; c < kChains * kCols * 4; ++c) sc[c / (kCols * 4)][c / 4 % kCols][c % 4] = 0.0f;
            const int krow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                for (int sub = 0; sub < Cfg::kSub; ++sub) {
                    uint32_t kf[4];
                    const int chunk = (ks & 3) * 2 + ((lane >> 3) & 1);
                    ldmatrix_x4(kf, kb + (ks >> 2) * (Cfg::kBlockKeys * 128) + sub * 2048 + krow * 128 +
                                        ((chunk ^ (krow & 7)) << 4));
                    mma_16816<T>(sc[ks % kChains][2 * sub], qa[ks], kf[0], kf[1]);
                    mma_16816<T>(sc[ks % kChains][2 * sub + 1], qa[ks], kf[2], kf[3]);
                }
            // ---- scale, mask, running maximum (base-2 exponents); x[e]: row g + 8 e, keys k0 + 8 c and the next
            float x[2][2 * kCols];
            const int k0 = key0 + t4 * 2;
            const bool masked = __any_sync(0xffffffffu, min(last_key[0], last_key[1]) < key0 + Cfg::kBlockKeys - 1 ||
                                                            max(first_key[0], first_key[1]) > key0);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float v = sc[0][c][2 * e + f];
                        if (kChains == 2) v += sc[kChains - 1][c][2 * e + f];
                        x[e][2 * c + f] = v * sh.scale_log2;
                    }
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 2 * kCols; ++c) {
                        const int key = k0 + (c >> 1) * 8 + (c & 1);
                        if (key > last_key[e] || key < first_key[e]) x[e][c] = -INFINITY;
                    }
                }
                float top = x[e][0];
#pragma unroll
                for (int c = 1; c < 2 * kCols; ++c) top = fmaxf(top, x[e][c]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[e], top);
                const float base_m = mn == -INFINITY ? 0.0f : mn;
                const float scale = ex2(m[e] - base_m);
                m[e] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < 2 * kCols; ++c) {
                    x[e][c] = ex2(x[e][c] - base_m);
                    sum += x[e][c];
                }
                l[e] = l[e] * scale + sum;
                if (__any_sync(0xffffffffu, scale != 1.0f)) {
#pragma unroll
                    for (int n = 0; n < DP / 8; ++n) {
                        o[n][2 * e] *= scale;
                        o[n][2 * e + 1] *= scale;
                    }
                }
            }
            // ---- O += P V; value rows past the keys are not multiplied (0 x NaN)
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
            const bool ragged = key0 + Cfg::kBlockKeys > it.hi || key0 < it.lo;
#pragma unroll
            for (int sub = 0; sub < Cfg::kSub; ++sub) {
                uint32_t pa[4], pb[4];   // the two parts of the weights
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const float lo = x[f & 1][4 * sub + (f >> 1) * 2], hi = x[f & 1][4 * sub + (f >> 1) * 2 + 1];
                    pa[f] = pack2<T>(lo, hi);
                    pb[f] = pack2<T>(lo - low_of<T>(pa[f]), hi - high_of<T>(pa[f]));
                }
#pragma unroll
                for (int n = 0; n < DP / 8; n += 2) {
                    uint32_t vf[4];
                    const int chunk = (n & 7) + (lane >> 4);
                    ldmatrix_x4_trans(vf, vb + (n >> 3) * (Cfg::kBlockKeys * 128) + sub * 2048 + vrow * 128 +
                                              ((chunk ^ (vrow & 7)) << 4));
                    if (ragged) {
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const int key = k0 + sub * kSplitKeys + (f & 1) * 8;
                            if (key >= it.hi || key < it.lo) vf[f] &= 0xffff0000u;
                            if (key + 1 >= it.hi || key + 1 < it.lo) vf[f] &= 0x0000ffffu;
                        }
                    }
                    mma_16816<T>(o[n], pa, vf[0], vf[1]);
                    mma_16816<T>(o[n + 1], pa, vf[2], vf[3]);
#pragma unroll
                    for (int f = 0; f < 4; ++f) vf[f] = finite_pair<T>(vf[f]);   // (a second part of 0 x infinity)
                    mma_16816<T>(o[n], pb, vf[0], vf[1]);
                    mma_16816<T>(o[n + 1], pb, vf[2], vf[3]);
                }
            }
            __syncwarp();
            if (i + Cfg::kStages < i1) issue(i + Cfg::kStages);
        }
        loads += static_cast<uint32_t>(n_blocks);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }

        __syncthreads();
        {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (8 * e >= rows) break;
#pragma unroll
                for (int n = 0; n < DP / 8; ++n)
                    *reinterpret_cast<float2*>(mo + (g + 8 * e) * Cfg::kMergeRow + n * 8 + t4 * 2) =
                        make_float2(o[n][2 * e], o[n][2 * e + 1]);
                if (t4 == 0) s_ml[warp][g + 8 * e] = make_float2(m[e], l[e]);
            }
        }
        } else {
        // ---- S^T = K Q^T and O^T += V^T P^T: keys and head elements are the products' 16 rows, query rows their
        // columns, eight to a tile (a single token's rows under 8 heads: half the products and registers of rows as
        // rows).  Lane (g, t) holds keys g and g + 8 and elements 2g and 2g + 1 of each 16 under the query rows 2t and
        // 2t + 1.
        constexpr int kTiles = ROWS / 8, kSub = Cfg::kSub;
        constexpr bool kHalf = std::is_same<T, __half>::value;
        constexpr int kParts = kHalf ? 2 : 1;       // of the weights
        uint32_t qb[kTiles][DP / 16][2];            // rows g of the tiles in the MMA's B layout, pairs of fp16
        float q_scale[kTiles][2];                   // of rows 2t and 2t + 1: what their scores are to be multiplied by
        int last_key[kTiles][2], first_key[kTiles][2];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const int row = rt * ROWS + n * 8 + g, tok = row / sh.group;
            const T* qp = static_cast<const T*>(p.q) + static_cast<long long>(sq.first_token + tok) * p.q_token +
                          static_cast<long long>(h * sh.group + row - tok * sh.group) * p.q_head;
            uint2 raw[DP / 16];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {
                const int d = c * 16 + t4 * 4;
                raw[c] = n * 8 + g < rows && d < sh.head_dim ? *reinterpret_cast<const uint2*>(qp + d)
                                                             : make_uint2(0, 0);
                top = max(top, max(max(magnitude(low_of<T>(raw[c].x)), magnitude(high_of<T>(raw[c].x))),
                                   max(magnitude(low_of<T>(raw[c].y)), magnitude(high_of<T>(raw[c].y)))));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // times 2^a the largest is 2^14 to 2^15 (a up to 126, for rows of next to nothing); the scores' factor back
            // is NaN for a row that is not finite
            const int a = kHalf ? 0 : max(min(141 - static_cast<int>(top >> 23), 126), -113);
            const float up = __uint_as_float(static_cast<uint32_t>(a + 127) << 23);
            const float back = !kHalf && top >= 0x7f800000u
                                   ? __uint_as_float(0x7fc00000u)
                                   : sh.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - a) << 23);
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) {   // elements 4t to 4t + 3 of the 16
                qb[n][c][0] = raw[c].x;
                qb[n][c][1] = raw[c].y;
                if (!kHalf) {
                    qb[n][c][0] = pack2<__half>(low_of<T>(raw[c].x) * up, high_of<T>(raw[c].x) * up);
                    qb[n][c][1] = pack2<__half>(low_of<T>(raw[c].y) * up, high_of<T>(raw[c].y) * up);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                q_scale[n][e] = __shfl_sync(0xffffffffu, back, (t4 * 2 + e) * 4);
                const int r = n * 8 + t4 * 2 + e, t = (rt * ROWS + r) / sh.group;
                last_key[n][e] = r < rows ? min(sq.first_pos + t, sq.keys - 1) : 0x7fffffff;
                first_key[n][e] = r < rows ? window_start(sq.first_pos + t, sh.window) : 0;
            }
        }
        float o[kTiles][DP / 16][4], m[kTiles][2], l[kTiles][2];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
#pragma unroll
            for (int c = 0; c < DP / 4; ++c) o[n][c / 4][c % 4] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
        for (int i = i0; i < i1; ++i) {
            if (!block_ready(i)) break;
            const uint32_t st = (loads + static_cast<uint32_t>(i - i0)) % Cfg::kStages;
            const uint32_t kb = smem_u32(ring + st * 2 * Cfg::kBlockBytes);
            const uint32_t vb = kb + Cfg::kBlockBytes;
            const int key0 = base + i * Cfg::kUnit;
            float sc[kTiles][kSub][4];   // of each 16 keys
#pragma unroll
            for (int c = 0; c < kTiles * kSub * 4; ++c) sc[c / (4 * kSub)][c / 4 % kSub][c % 4] = 0.0f;
            const int krow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ks += 2)
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
                    uint32_t kf[4];   // keys 0-7 of two times 16 elements, keys 8-15
                    ldmatrix_x4(kf, piece8<DP>(kb + sub * kSplitKeys * DP, krow, ks + ((lane >> 3) & 1)));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t a[4];
                        widen_e4m3(kf[k], a[0], a[2]);
                        widen_e4m3(kf[k + 2], a[1], a[3]);
#pragma unroll
                        for (int n = 0; n < kTiles; ++n)
                            mma_16816<__half>(sc[n][sub], a, qb[n][ks + k][0], qb[n][ks + k][1]);
                    }
                }
            // ---- scores (base-2 exponents), masks, maxima; weights in parts, turned to the B layout
            int first_all = first_key[0][0], last_all = last_key[0][0];
#pragma unroll
            for (int c = 1; c < 2 * kTiles; ++c) {
                first_all = max(first_all, first_key[c / 2][c % 2]);
                last_all = min(last_all, last_key[c / 2][c % 2]);
            }
            const bool masked = __any_sync(0xffffffffu, last_all < key0 + Cfg::kBlockKeys - 1 || first_all > key0);
            // Values of scale 255 are NaN to the rows that see a key of their 16, by those rows' sums of weights; in the
            // products they are zeros under the least power, so that no other row meets them.
            uint32_t scales[kSub];
            float v_exp[kSub];   // the values' exponents
            bool nan_values = false;
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
                scales[sub] = s_scales[warp][st][sub];
                const int byte = static_cast<int>(scales[sub] >> 8);
                nan_values = nan_values || byte == 255;
                v_exp[sub] = static_cast<float>((byte == 255 ? 0 : byte) - 127);
            }
            uint32_t pw[kTiles][kSub][kParts][2];   // [16 keys][part][keys 0-7, 8-15]
            float share[kTiles][2];   // what a row's sums over this block are to be multiplied by
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                float x[kSub][4];
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
                    const float k_scale = e8m0_power(scales[sub] & 255u);
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        x[sub][f] = sc[n][sub][f] * (q_scale[n][f & 1] * k_scale);
                        const int key = key0 + sub * kSplitKeys + g + (f >> 1) * 8;
                        if (masked && (key > last_key[n][f & 1] || key < first_key[n][f & 1])) x[sub][f] = -INFINITY;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top[kSub], mn = m[n][e];
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub) top[sub] = fmaxf(x[sub][e], x[sub][e + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2)
#pragma unroll
                        for (int sub = 0; sub < kSub; ++sub)
                            top[sub] = fmaxf(top[sub], __shfl_xor_sync(0xffffffffu, top[sub], d));
#pragma unroll
                    for (int sub = 0; sub < kSub; sub += 2) mn = max3(mn, top[sub], top[sub + 1]);
                    const float base_m = mn == -INFINITY ? 0.0f : mn;
                    const float scale = ex2(m[n][e] - base_m);
                    m[n][e] = mn;
                    // The largest weight times its value's power, relative to the maximum: the block's weights, powers
                    // included, are taken as multiples of it, so that they use fp16's range whatever the blocks' powers
                    // are.  What ex2 would flush (below 2^-126) stays with the weights, which have room for it: at the
                    // least power, 2^-117, a block's largest weight keeps its 11 bits down to 2^-32.  (Scores that are
                    // NaN, which fmaxf passes over, are in the row's sum of weights.)
                    float ref = kLeastShareLog2;
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub) ref = fmaxf(ref, top[sub] - base_m + v_exp[sub]);
                    share[n][e] = ex2(ref);
                    float sum = 0.0f;
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
                        for (int f = e; f < 4; f += 2) {
                            const float d = x[sub][f] - base_m;
                            sum += ex2(d);
                            x[sub][f] = ex2(d + (v_exp[sub] - ref + kWeightLog2));
                        }
                    if (nan_values) {
#pragma unroll
                        for (int sub = 0; sub < kSub; ++sub)
                            if (scales[sub] >> 8 == 255 && top[sub] != -INFINITY) sum = __uint_as_float(0x7fc00000u);
                    }
                    l[n][e] = l[n][e] * scale + sum;
                    if (__any_sync(0xffffffffu, scale != 1.0f)) {
#pragma unroll
                        for (int c = 0; c < DP / 16; ++c) {
                            o[n][c][e] *= scale;
                            o[n][c][e + 2] *= scale;
                        }
                    }
                }
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float lo = x[sub][2 * f], hi = x[sub][2 * f + 1];
                        const uint32_t w = pack2<__half>(lo, hi);
                        pw[n][sub][0][f] = transpose_8x8(w);
                        if (kParts == 2)
                            pw[n][sub][kParts - 1][f] =
                                transpose_8x8(pack2<__half>(lo - low_of<__half>(w), hi - high_of<__half>(w)));
                    }
            }
            // ---- O^T += V^T P^T; value rows that no token sees, or that are NaN, are not multiplied (0 x NaN)
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
            const bool ragged = nan_values || key0 + Cfg::kBlockKeys > it.hi || key0 < it.lo;
#pragma unroll
            for (int c = 0; c < DP / 16; c += 2) {
                uint32_t a[kSub][2][4];   // [16 keys][16 elements]
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) {
                    uint32_t vf[4];    // keys 0-7 and 8-15 of two times 16 elements
                    ldmatrix_x4_trans(vf, piece8<DP>(vb + sub * kSplitKeys * DP, vrow, c + (lane >> 4)));
                    if (ragged) {
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const int key = key0 + sub * kSplitKeys + t4 * 2 + (f & 1) * 8;
                            if (key >= it.hi || key < it.lo) vf[f] &= 0xffff0000u;
                            if (key + 1 >= it.hi || key + 1 < it.lo) vf[f] &= 0x0000ffffu;
                            if (scales[sub] >> 8 == 255) vf[f] = 0;
                        }
                    }
                    // keys 2t and 2t + 1 of element 2g, of element 2g + 1
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        widen_e4m3(__byte_perm(vf[2 * k], 0, 0x3120), a[sub][k][0], a[sub][k][1]);
                        widen_e4m3(__byte_perm(vf[2 * k + 1], 0, 0x3120), a[sub][k][2], a[sub][k][3]);
                    }
                }
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    float y[2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma_16816_first(y[k], a[0][k], pw[n][0][0][0], pw[n][0][0][1]);
#pragma unroll
                    for (int sub = 1; sub < kSub; ++sub)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_16816<__half>(y[k], a[sub][k], pw[n][sub][0][0], pw[n][sub][0][1]);
                    if (kParts == 2) {
#pragma unroll
                        for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                mma_16816<__half>(y[k], a[sub][k], pw[n][sub][kParts - 1][0],
                                                  pw[n][sub][kParts - 1][1]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int f = 0; f < 4; ++f) o[n][c + k][f] = fmaf(y[k][f], share[n][f & 1], o[n][c + k][f]);
                }
            }
            __syncwarp();
            if (i + Cfg::kStages < i1) issue(i + Cfg::kStages);
        }
        loads += static_cast<uint32_t>(n_blocks);
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], d);
        constexpr float kUnweight = 1.0f / 1024.0f;   // 2^-kWeightLog2
        __syncthreads();
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = n * 8 + t4 * 2 + e;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c)
                    *reinterpret_cast<float2*>(mo + row * Cfg::kMergeRow + c * 16 + g * 2) =
                        make_float2(o[n][c][e] * kUnweight, o[n][c][e + 2] * kUnweight);
                if (g == 0) s_ml[warp][row] = make_float2(m[n][e], l[n][e]);
            }
        }
        __syncthreads();
        // ---- join the warps: a thread takes the float4 tid, tid + 128, .. of the rows
        float4 acc[Cfg::kParts];
        float2 ml[Cfg::kParts];
        auto part_row = [&](int k) { return (tid + k * kSplitThreads) / (DP / 4); };
        const int d = (tid % (DP / 4)) * 4;   // kSplitThreads is a multiple of DP / 4
#pragma unroll
        for (int k = 0; k < Cfg::kParts; ++k) {
            const int row = part_row(k);
            if (row >= rows) break;
            float top = s_ml[0][row].x;
#pragma unroll
            for (int w = 1; w < kSplitWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kSplitWarps; ++w) {
                const float2 e = s_ml[w][row];
                const float f = ex2(e.x - ref);
                const float4 v =
                    *reinterpret_cast<const float4*>(merge + (w * Cfg::kRows + row) * Cfg::kMergeRow + d);
                sum += f * e.y;
                a.x += f * v.x;
                a.y += f * v.y;
                a.z += f * v.z;
                a.w += f * v.w;
            }
            acc[k] = a;
            ml[k] = make_float2(top, sum);
        }
        auto store = [&](int row, float4 a, float2 e) {
            const int r = rt * Cfg::kRows + row;
            const int tok = r / sh.group;
            const int head = h * sh.group + r - tok * sh.group;
            if (d >= sh.head_dim) return;
            float f = 1.0f;
            if (sh.sinks != nullptr) {
                const float sk = sh.sinks[head] * kLog2e;
                const float top = fmaxf(e.x, sk);
                const float ref = top == -INFINITY ? 0.0f : top;
                f = ex2(e.x - ref);
                e.y = e.y * f + ex2(sk - ref);
            }
            f = e.y == 0.0f ? 0.0f : f / e.y;
            T* dst = static_cast<T*>(p.out) + static_cast<long long>(sq.first_token + tok) * p.o_token +
                     static_cast<long long>(head) * p.o_head + d;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(a.x * f, a.y * f), pack2<T>(a.z * f, a.w * f));
        };

        if (u0 == 0 && u1 == it.units) {
#pragma unroll
            for (int k = 0; k < Cfg::kParts; ++k)
                if (part_row(k) < rows) store(part_row(k), acc[k], ml[k]);
        } else {
            // The item's pieces lie with the CTAs of runs c0 .. c0 + n - 1.  On the line, the first is its CTA's last
            // piece (slot 1), the others their CTAs' first (slot 0).
            int c0, n;
            if (plan.piece > 0) {
                n = pieces_of(it.units, plan.piece);
                c0 = order.run - u0 / ((it.units + n - 1) / n);
            } else {
                c0 = static_cast<int>(first / plan.per);
                n = static_cast<int>((first + it.units - 1) / plan.per) - c0 + 1;
            }
            const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0);
#pragma unroll
            for (int k = 0; k < Cfg::kParts; ++k) {
                const int row = part_row(k);
                if (row >= rows) break;
                p.part_o[(slot * Cfg::kRows + row) * (DP / 4) + d / 4] = acc[k];
                if (d == 0) p.part_ml[slot * Cfg::kRows + row] = ml[k];
            }
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                const unsigned seen = atomicAdd(&p.counters[c0 * order.step + order.first], 1u);
                s_last = seen == static_cast<unsigned>(n - 1);
                if (s_last) p.counters[c0 * order.step + order.first] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                // maxima and sums of all pieces into shared memory, then their outputs, several loads under way
                float2* all = reinterpret_cast<float2*>(ring_base);   // [pieces][16]; the merge is over
                auto slot_of = [&](int c) { return 2 * ((c0 + c) * order.step + order.first) + (c == 0 ? 1 : 0); };
                for (int i = tid; i < n * Cfg::kRows; i += kSplitThreads)
                    all[i] = __ldcg(&p.part_ml[slot_of(i / Cfg::kRows) * Cfg::kRows + i % Cfg::kRows]);
                __syncthreads();
                auto join = [&](auto live) {   // live: parts per thread that hold rows, so that 16 loads are under way
                    constexpr int kLive = decltype(live)::value;
                    float ref[kLive];
#pragma unroll
                    for (int k = 0; k < kLive; ++k) {
                        const int row = part_row(k);
                        float top = -INFINITY;
                        for (int c = 0; c < n; ++c) top = fmaxf(top, all[c * Cfg::kRows + row].x);
                        ref[k] = top == -INFINITY ? 0.0f : top;
                        ml[k] = make_float2(top, 0.0f);
                        acc[k] = make_float4(0, 0, 0, 0);
                    }
#pragma unroll (16 / kLive)
                    for (int c = 0; c < n; ++c) {
#pragma unroll
                        for (int k = 0; k < kLive; ++k) {
                            const int row = part_row(k);
                            const float2 e = all[c * Cfg::kRows + row];
                            const float4 v = row < rows
                                                 ? __ldcg(&p.part_o[(slot_of(c) * Cfg::kRows + row) * (DP / 4) + d / 4])
                                                 : make_float4(0, 0, 0, 0);
                            const float f = ex2(e.x - ref[k]);
                            ml[k].y += f * e.y;
                            acc[k].x += f * v.x;
                            acc[k].y += f * v.y;
                            acc[k].z += f * v.z;
                            acc[k].w += f * v.w;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kLive; ++k)
                        if (part_row(k) < rows) store(part_row(k), acc[k], ml[k]);
                };
                if (rows * (DP / 4) <= kSplitThreads) join(std::integral_constant<int, 1>());
                else if (Cfg::kParts > 2 && rows * (DP / 4) <= 2 * kSplitThreads)
                    join(std::integral_constant<int, 2>());
                else join(std::integral_constant<int, Cfg::kParts>());
            }
        }
        }   // of an item with units in the run

        // ---- the run's next item
        if (plan.piece > 0) break;
        first += it.units + kSplitItemUnits;
        if (first >= end) break;
        if (++hl == order.heads) {
            hl = 0;
            if (++rt == row_tiles) {
                rt = 0;
                do {
                    if (++b >= sh.seqs) return;
                    sq = seq_info(sh, b);
                    row_tiles = split_row_tiles<Cfg>(sh, sq);
                } while (row_tiles == 0);
            }
            it = split_item<Cfg>(sh, sq, rt);
        }
        u0 = 0;
        u1 = static_cast<int>(min(end - first, static_cast<long long>(it.units)));
        // generic reads and writes of the merge area come before the next item's loads into it
        fence_proxy_async_smem();
        __syncthreads();
    }
}

template <typename Cfg>
static int split_ctas() {
    return std::min(sm_count() * Cfg::kCtasPerSm, std::min(static_cast<int>(kAttnMaxCounters), Cfg::kMaxCtas));
}

size_t attn_split_workspace_bytes() {
    const size_t c =
        static_cast<size_t>(std::max(split_ctas<SplitCfg<128, false, 16>>(), split_ctas<SplitCfg<64, true, 8>>()));
    return c * 2 * 16 * (128 + 2) * sizeof(float);
}

template <typename T, int DP, bool KV8, int ROWS>
static kt_status launch_split_typed(const AttnArgs& a, cudaStream_t s) {
    using Cfg = SplitCfg<DP, KV8, ROWS>;
    CUtensorMap kmap, vmap;
    auto encode = [&](CUtensorMap* m, bool values) {
        const CUtensorMapSwizzle swizzle = DP == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
        return KV8 ? encode_kv8_map(m, a.kv, values, DP, kSplitKeys, swizzle)
                   : encode_kv_map(m, a.kv, values, kSplitKeys);
    };
    if (!encode(&kmap, false) || !encode(&vmap, true))
        return report(KT_ERR_CUDA, "tensor map encoding failed");
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<T, DP, KV8, ROWS>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e != cudaSuccess) return cuda_status(e);
        attr_set[dev] = true;
    }
    SplitParams p{};
    p.sh = attn_shape(a);
    p.q = a.q.ptr;
    p.out = a.out.ptr;
    p.q_token = a.q.token_stride;
    p.q_head = a.q.head_stride;
    p.o_token = a.out.token_stride;
    p.o_head = a.out.head_stride;
    const size_t c = static_cast<size_t>(split_ctas<Cfg>());
    p.counters = a.counters;
    p.part_o = reinterpret_cast<float4*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + c * 2 * Cfg::kRows * 32);
    count_launches(1);
    return cuda_status(launch_chained(attn_split_kernel<T, DP, KV8, ROWS>, dim3(static_cast<unsigned>(c)),
                                      dim3(kSplitThreads), Cfg::kSmem, s, static_cast<const SplitParams&>(p),
                                      static_cast<const CUtensorMap&>(kmap), static_cast<const CUtensorMap&>(vmap)));
}

template <typename T>
static kt_status launch_split_of(const AttnArgs& a, int rows, cudaStream_t s) {
    const bool wide = a.kv.head_dim > 64;
    if (a.k_scales == nullptr)
        return wide ? launch_split_typed<T, 128, false, 16>(a, s) : launch_split_typed<T, 64, false, 16>(a, s);
    if (rows <= 8) return wide ? launch_split_typed<T, 128, true, 8>(a, s) : launch_split_typed<T, 64, true, 8>(a, s);
    return wide ? launch_split_typed<T, 128, true, 16>(a, s) : launch_split_typed<T, 64, true, 16>(a, s);
}

kt_status launch_attn_split(const AttnArgs& a, int rows, cudaStream_t s) {
    return a.kv.dtype == KT_DTYPE_BF16 ? launch_split_of<__nv_bfloat16>(a, rows, s)
                                       : launch_split_of<__half>(a, rows, s);
}

}  // namespace kt
