// kt_attn_split.cu -- attention over a paged cache for few query rows: every
// warp streams its own keys and values and keeps its own softmax state.
//
// An item is (sequence, cache head, 16 query rows): row r of a sequence is its
// new token r / group under query head r % group of the cache head's group, so
// the heads that share a cache head share its loads.  A warp takes blocks of 16
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
#include <algorithm>
#include <type_traits>

#include "kt_attn_dev.cuh"

namespace kt {

constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = kSplitWarps * 32;
constexpr int kSplitKeys = 16;                          // keys of one load (pages hold a multiple of it)
constexpr int kSplitRows = 16;
constexpr int kSplitCtasPerSm = 2;
constexpr int kSplitMinUnits = 2;                       // least units of a piece
constexpr int kSplitItemUnits = 3;                      // what an item costs besides its units, in units
constexpr int kSplitJoinUnits = 4;                      // what cutting an item costs its last CTA, in units

template <int DP>
struct SplitCfg {
    static constexpr int kSub = DP == 128 ? 1 : 2;                   // loads of K and of V that make a warp's block
    static constexpr int kBlockKeys = kSub * kSplitKeys;
    static constexpr int kUnit = kSplitWarps * kBlockKeys;           // keys of one unit
    static constexpr int kBlockBytes = kBlockKeys * DP * 2;          // one of K, V
    static constexpr int kStages = 3;
    static constexpr int kRing = kStages * 2 * kBlockBytes;          // per warp
    static constexpr int kSmem = kSplitWarps * kRing + 1024;
    static constexpr int kMergeRow = DP + 8;                         // floats of a row: rows start 8 banks apart
    static constexpr int kMergeBytes = kSplitWarps * kSplitRows * kMergeRow * 4;
    static constexpr int kParts = kSplitRows * DP / 4 / kSplitThreads;   // float4 per thread of 16 rows
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

// Keys that the 16 rows of row tile rt see: [lo, hi); units of the item (at least one, so that its rows are written).
struct SplitItem {
    int lo, hi, unit0, units;
};
__device__ __forceinline__ SplitItem split_item(const AttnShape& s, const SeqInfo& q, int rt, int unit) {
    SplitItem it;
    const int t0 = rt * kSplitRows / s.group;
    const int t1 = min((rt * kSplitRows + kSplitRows - 1) / s.group, q.q_len - 1);
    it.hi = max(0, min(q.first_pos + t1 + 1, q.keys));
    it.lo = window_start(q.first_pos + t0, s.window);
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.unit0 = it.lo / unit;
    it.units = max(1, (it.hi + unit - 1) / unit - it.unit0);
    return it;
}
__device__ __forceinline__ int split_row_tiles(const AttnShape& s, const SeqInfo& q) {
    return (q.q_len * s.group + kSplitRows - 1) / kSplitRows;
}

// How the items are dealt to the CTAs.  Few items: each is cut into pieces of at most `piece` units, a CTA takes one
// piece (piece > 0).  Many: they lie on a line, kSplitItemUnits before each one's units, that is cut into equal runs
// (piece == 0).  In both, [begin, begin + per) of `total` are this CTA's, in pieces or in units of the line.
struct SplitPlan {
    long long total, per, begin;
    long long in_seq;   // begin's place in sequence seq
    int piece, seq;
};
__device__ __forceinline__ int pieces_of(int units, int piece) { return (units + piece - 1) / piece; }
__device__ __forceinline__ int item_measure(const SplitItem& it, int piece) {
    return piece > 0 ? pieces_of(it.units, piece) : it.units + kSplitItemUnits;
}
__device__ __forceinline__ long long seq_measure(const AttnShape& s, int b, int piece, int unit) {
    const SeqInfo q = seq_info(s, b);
    const int tiles = split_row_tiles(s, q);
    long long n = 0;
    for (int rt = 0; rt < tiles; ++rt) n += item_measure(split_item(s, q, rt, unit), piece);
    return n * s.kv_heads;
}

// All threads of the CTA; `shared` is theirs.
__device__ __forceinline__ SplitPlan split_plan(const AttnShape& s, int unit, SplitPlan* shared) {
    __shared__ long long s_units[kSplitWarps], s_items[kSplitWarps];
    __shared__ int s_most[kSplitWarps];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    long long units = 0, items = 0;
    int most = 0;
    for (int b = tid; b < s.seqs; b += kSplitThreads) {
        const SeqInfo q = seq_info(s, b);
        const int tiles = split_row_tiles(s, q);
        for (int rt = 0; rt < tiles; ++rt) {
            const int n = split_item(s, q, rt, unit).units;
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
    units *= s.kv_heads;
    items *= s.kv_heads;
    const long long ctas = gridDim.x;
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
    plan.begin = plan.per * blockIdx.x;
    // the sequence of this CTA's first piece or unit
    if (tid == 0) shared->seq = s.seqs;
    long long before = 0;
    for (int b0 = 0; b0 < s.seqs; b0 += kSplitThreads) {
        const long long n = b0 + tid < s.seqs ? seq_measure(s, b0 + tid, piece, unit) : 0;
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

template <typename T, int DP>
__global__ void __launch_bounds__(kSplitThreads, kSplitCtasPerSm)
    attn_split_kernel(const SplitParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Cfg = SplitCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kSplitWarps][Cfg::kStages];
    __shared__ int s_abort, s_last;
    __shared__ float2 s_ml[kSplitWarps][kSplitRows];
    __shared__ SplitPlan s_plan;
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
    const SplitPlan plan = split_plan(sh, Cfg::kUnit, &s_plan);
    if (plan.seq >= sh.seqs) return;

    // ---- the item of this CTA's first piece or unit
    int b = plan.seq, rt = 0;
    SeqInfo sq = seq_info(sh, b);
    int row_tiles = split_row_tiles(sh, sq);
    SplitItem it = split_item(sh, sq, 0, Cfg::kUnit);
    long long at = plan.in_seq;
    while (at >= static_cast<long long>(item_measure(it, plan.piece)) * sh.kv_heads) {
        at -= static_cast<long long>(item_measure(it, plan.piece)) * sh.kv_heads;
        it = split_item(sh, sq, ++rt, Cfg::kUnit);
    }
    int h, u0, u1;                 // cache head; the item's units in this run
    long long first = 0;           // line: the item's first unit
    const long long end = plan.begin + plan.per;
    {
        const int n = item_measure(it, plan.piece);
        h = at >> 31 == 0 ? static_cast<int>(at) / n : static_cast<int>(at / n);
        const int in = static_cast<int>(at - static_cast<long long>(h) * n);
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

        // ---- this warp's blocks: keys base + kUnit i, i in [i0, i1)
        const int base = (it.unit0 + u0) * Cfg::kUnit + warp * Cfg::kBlockKeys;
        int i0 = 0, i1 = u1 - u0;
        while (i0 < i1 && base + i0 * Cfg::kUnit + Cfg::kBlockKeys <= it.lo) ++i0;
        while (i1 > i0 && base + (i1 - 1) * Cfg::kUnit >= it.hi) --i1;
        if (gave_up) i1 = i0;
        int page_batch = -1, my_page = -1, my_slot = 0;
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
                // (16 keys that no row sees, past them all or before the window: zeros from outside the cache)
                if (mine < i1 && key < it.hi && key + kSplitKeys > it.lo) {
                    my_page = checked_page(sh, pages, key);
                    my_slot = key % sh.page_size;
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
                if (lane == 0) {
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

        // ---- queries: rows g and g + 8 of the tile in the MMA's A layout
        const int g = lane >> 2, t4 = lane & 3;
        uint32_t qa[DP / 16][4];
        int last_key[2], first_key[2];   // what the row sees; rows of no token need no mask
        {
            const T* qp[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = rt * kSplitRows + g + 8 * e;
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
            const uint32_t seq_no = loads + static_cast<uint32_t>(i - i0);
            const uint32_t st = seq_no % Cfg::kStages;
            if (!warp_wait(smem_u32(&s_full[warp][st]), (seq_no / Cfg::kStages) & 1u, &s_abort, sh.wait_limit_ns)) {
                if (lane == 0 && !*reinterpret_cast<volatile int*>(&s_abort)) {
                    s_abort = 1;
                    set_error(sh.err, KT_DEVERR_TIMEOUT_LOAD);
                }
                // loads still in flight land before their memory has another use (each wait bounded)
                int never = 0;
                for (int k = i; k < min(i + Cfg::kStages, i1); ++k) {
                    const uint32_t no = loads + static_cast<uint32_t>(k - i0);
                    mbar_wait(smem_u32(&s_full[warp][no % Cfg::kStages]), (no / Cfg::kStages) & 1u, &never,
                              kDrainLimitNs);
                }
                gave_up = true;
                break;
            }
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

        // ---- join the warps: a thread takes the float4 tid, tid + 128, .. of the tile's rows that hold tokens
        const int rows = min(kSplitRows, sq.q_len * sh.group - rt * kSplitRows);
        __syncthreads();
        {
            float* mo = merge + warp * kSplitRows * Cfg::kMergeRow;
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
        __syncthreads();
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
                    *reinterpret_cast<const float4*>(merge + (w * kSplitRows + row) * Cfg::kMergeRow + d);
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
            const int r = rt * kSplitRows + row;
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
            // The item's pieces lie with CTAs c0 .. c0 + n - 1.  On the line, the first is its CTA's last piece (slot
            // 1), the others their CTAs' first (slot 0).
            int c0, n;
            if (plan.piece > 0) {
                n = pieces_of(it.units, plan.piece);
                c0 = static_cast<int>(blockIdx.x) - u0 / ((it.units + n - 1) / n);
            } else {
                c0 = static_cast<int>(first / plan.per);
                n = static_cast<int>((first + it.units - 1) / plan.per) - c0 + 1;
            }
            const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0);
#pragma unroll
            for (int k = 0; k < Cfg::kParts; ++k) {
                const int row = part_row(k);
                if (row >= rows) break;
                p.part_o[(slot * kSplitRows + row) * (DP / 4) + d / 4] = acc[k];
                if (d == 0) p.part_ml[slot * kSplitRows + row] = ml[k];
            }
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                const unsigned seen = atomicAdd(&p.counters[c0], 1u);
                s_last = seen == static_cast<unsigned>(n - 1);
                if (s_last) p.counters[c0] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                // maxima and sums of all pieces into shared memory, then their outputs, several loads under way
                float2* all = reinterpret_cast<float2*>(ring_base + Cfg::kMergeBytes);   // [pieces][16]
                auto slot_of = [&](int c) { return 2 * (c0 + c) + (c == 0 ? 1 : 0); };
                for (int i = tid; i < n * kSplitRows; i += kSplitThreads)
                    all[i] = __ldcg(&p.part_ml[slot_of(i / kSplitRows) * kSplitRows + i % kSplitRows]);
                __syncthreads();
                auto join = [&](auto live) {   // live: parts per thread that hold rows, so that 16 loads are under way
                    constexpr int kLive = decltype(live)::value;
                    float ref[kLive];
#pragma unroll
                    for (int k = 0; k < kLive; ++k) {
                        const int row = part_row(k);
                        float top = -INFINITY;
                        for (int c = 0; c < n; ++c) top = fmaxf(top, all[c * kSplitRows + row].x);
                        ref[k] = top == -INFINITY ? 0.0f : top;
                        ml[k] = make_float2(top, 0.0f);
                        acc[k] = make_float4(0, 0, 0, 0);
                    }
#pragma unroll (16 / kLive)
                    for (int c = 0; c < n; ++c) {
#pragma unroll
                        for (int k = 0; k < kLive; ++k) {
                            const int row = part_row(k);
                            const float2 e = all[c * kSplitRows + row];
                            const float4 v = row < rows
                                                 ? __ldcg(&p.part_o[(slot_of(c) * kSplitRows + row) * (DP / 4) + d / 4])
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
        if (++h == sh.kv_heads) {
            h = 0;
            if (++rt == row_tiles) {
                rt = 0;
                do {
                    if (++b >= sh.seqs) return;
                    sq = seq_info(sh, b);
                    row_tiles = split_row_tiles(sh, sq);
                } while (row_tiles == 0);
            }
            it = split_item(sh, sq, rt, Cfg::kUnit);
        }
        u0 = 0;
        u1 = static_cast<int>(min(end - first, static_cast<long long>(it.units)));
        // generic reads and writes of the merge area come before the next item's loads into it
        fence_proxy_async_smem();
        __syncthreads();
    }
}

static int split_ctas() {
    return std::min(sm_count() * kSplitCtasPerSm, static_cast<int>(kAttnMaxCounters));
}

size_t attn_split_workspace_bytes() {
    const size_t c = static_cast<size_t>(split_ctas());
    return c * 2 * kSplitRows * (128 + 2) * sizeof(float);
}

template <typename T, int DP>
static kt_status launch_split_typed(const AttnArgs& a, cudaStream_t s) {
    using Cfg = SplitCfg<DP>;
    CUtensorMap kmap, vmap;
    if (!encode_kv_map(&kmap, a.kv, false, kSplitKeys) || !encode_kv_map(&vmap, a.kv, true, kSplitKeys))
        return report(KT_ERR_CUDA, "tensor map encoding failed");
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<T, DP>,
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
    const size_t c = static_cast<size_t>(split_ctas());
    p.counters = a.counters;
    p.part_o = reinterpret_cast<float4*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + c * 2 * kSplitRows * 32);
    count_launches(1);
    return cuda_status(launch_chained(attn_split_kernel<T, DP>, dim3(static_cast<unsigned>(c)), dim3(kSplitThreads),
                                      Cfg::kSmem, s, static_cast<const SplitParams&>(p),
                                      static_cast<const CUtensorMap&>(kmap), static_cast<const CUtensorMap&>(vmap)));
}

kt_status launch_attn_split(const AttnArgs& a, cudaStream_t s) {
    const bool wide = a.kv.head_dim > 64;
    if (a.kv.dtype == KT_DTYPE_BF16)
        return wide ? launch_split_typed<__nv_bfloat16, 128>(a, s) : launch_split_typed<__nv_bfloat16, 64>(a, s);
    return wide ? launch_split_typed<__half, 128>(a, s) : launch_split_typed<__half, 64>(a, s);
}

}  // namespace kt
