// kt_attn_tile.cu -- attention over a paged cache for chunks of new tokens, on
// the tcgen05 tensor cores.
//
// An item is (sequence, cache head, 2 x 128 query rows): a group of 128 rows
// holds 128 / group consecutive tokens under the cache head's query heads, so
// heads that share a cache head share its key and value tiles.  Per tile of 128
// keys and row group the CTA computes
//   S = Q K^T            (tensor cores, fp32 in tensor memory)
//   P = 2^(c S - c m)    (one thread per row; c = scale log2 e, m the row's reference)
//   O += P V             (tensor cores; P is read from tensor memory, where it replaces S)
// The two groups alternate: while one group's softmax runs, the tensor cores
// work on the other's products.  m is the running maximum as of its last change;
// it follows the true maximum only when that has grown by more than 2^8, so the
// rescaling of O (by the row's own thread) is rare, and the sums stay exact in
// fp32 (P up to 2^8 rounds with the same relative error, and fp16 holds it).
// P is rounded to the element type because the tensor cores multiply it with V
// in that type (once: a second product with what the rounding left would add half
// of their work again, and they are what heads of 128 wait for); the sum that
// divides O is of the unrounded weights.  Error against 64 bits: 1.1 to 1.4 times
// that of rounding the exact result once.
//
// Work is dealt to one CTA per SM: all items' key tiles (and two more each, what
// an item costs besides: 1 to 5 measured, 2 fastest) form one line that is cut
// into equal runs, so causal items of any length keep the SMs equally busy; a
// cut item leaves partial sums in the workspace and the CTA that finishes it
// last joins them in order, so the result does not depend on which that was.
//
// Warps: 0-3 softmax of group 0, 4-7 of group 1, 8 issues the MMAs, 9 to 11 the
// TMA loads of keys, values and queries.
//
// Bound: for heads of 128 the tensor cores (2630 of 3000 cycles of a tile pair),
// for smaller heads the softmax (128 exponentials a row and tile: 1370 cycles of
// issue and exponential unit for the two warps of a scheduler, measured alone).
// Measured on GB300 (bf16): an 8192-token prompt, 64 / 8 heads of 128, 670 us on
// the fastest machine (1640 TFLOP/s, 85 % of the measured burst matmul rate, 96 %
// of the sustained one), up to 790 us on others; heads of 64, 600 to 652 us, 842 to
// 916 TFLOP/s; 2048 tokens after 30001 on 16-slot pages (fp16, 32 / 8 heads of 128)
// 652 to 702 us, 1480 to 1600 TFLOP/s (757 us in seconds of calls, under the power
// cap at 1537 MHz).
//
// Tried and left out (8192-token prompt): P beside S so that the next S comes
// early (heads of 64: 636 against 614 us, both groups then contend for the
// exponential unit); the maximum of the second half under the first half's
// weights (738 against 677 us, registers spill); 224 registers for the softmax
// warps (694 against 674 us); the weights handed over at once (705 against 674).
#include <algorithm>
#include <type_traits>

#include "kt_attn_dev.cuh"

namespace kt {

constexpr int kTileKeys = 128;
constexpr int kTileThreads = 384;
constexpr int kItemUnits = 2;         // what an item costs besides its key tiles, in key tiles
constexpr int kTileMinUnits = kItemUnits + 2;   // least units of a CTA's run
constexpr int kPlanSeqs = 512;        // sequences planned at a time
constexpr float kLazyLog2 = 8.0f;     // growth of the maximum (log2) that is let stand

// Tensor memory: the CTA takes all 512 columns, so it starts at 0.  S of the groups, P in its first half, then O.
constexpr uint32_t kTmemS = 0, kTmemO = 256;

template <int DP>
struct TileCfg {
    static constexpr int kQBytes = 128 * DP * 2;         // one row group
    static constexpr int kStageBytes = kTileKeys * DP * 2;   // one tile of K or V
    static constexpr int kStages = DP == 128 ? 5 : 9;        // odd: K and V alternate in a stage
    static constexpr int kQBufs = DP == 128 ? 1 : 2;
    static constexpr int kQAll = kQBufs * 2 * kQBytes;
    static constexpr int kSmem = kQAll + kStages * kStageBytes + 1024;
};

struct TileGeometry {
    int tokens;      // of a row group: 128 / group
    int box_slots;   // slots of one load: the largest power of two that divides page_size, at most 128
};

struct TileParams {
    AttnShape sh;
    void* out;
    long long o_token, o_head;
    TileGeometry geo;
    float4* part_o;         // [CTAs][2 pieces][DP / 4][256 rows]
    float2* part_ml;        // [CTAs][2][256]
    unsigned* counters;     // [CTAs][2 groups]
};

struct TileItem {
    int lo, hi;        // keys that some row sees: [lo, hi)
    int base, tiles;   // first key of its first key tile, key tiles (at least one)
};
__device__ __forceinline__ TileItem tile_item(const AttnShape& s, const SeqInfo& q, const TileGeometry& g, int rt) {
    TileItem it;
    const int t0 = rt * 2 * g.tokens;
    const int t1 = min(t0 + 2 * g.tokens, q.q_len) - 1;
    it.hi = max(0, min(q.first_pos + t1 + 1, q.keys));
    it.lo = window_start(q.first_pos + t0, s.window);
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.base = it.lo & ~(g.box_slots - 1);
    it.tiles = max(1, (it.hi - it.base + kTileKeys - 1) / kTileKeys);
    return it;
}

// Units of item rt on the line: its key tiles, and the tiles' worth of time that any item takes besides.
__device__ __forceinline__ int item_units(const TileItem& it) { return it.tiles + kItemUnits; }

// A CTA's run of the line: [begin, begin + per) of `total` units, its first unit being unit in_seq of sequence seq.
struct RunPlan {
    long long total, per, begin, in_seq;
    int seq;
};

// Walks a CTA's run [begin, end) of units item by item; every role of the CTA walks it for itself.
struct TileWalk {
    int b, rt, row_tiles, h;
    int t0, t1;               // the item's key tiles in this run
    long long first, end;     // the item's first key tile on the line; end of the run
    SeqInfo sq;
    TileItem it;

    __device__ __forceinline__ bool load_seq(const AttnShape& s, const TileGeometry& g) {
        for (; b < s.seqs; ++b) {
            sq = seq_info(s, b);
            row_tiles = (sq.q_len + 2 * g.tokens - 1) / (2 * g.tokens);
            if (row_tiles > 0) return true;
        }
        return false;
    }
    __device__ __forceinline__ void cut(long long begin) {
        t0 = static_cast<int>(max(begin - first, 0ll));
        t1 = static_cast<int>(min(end - first, static_cast<long long>(it.tiles)));
    }
    // whole warp: finds the item of unit plan.in_seq of sequence plan.seq; false: no work
    __device__ __forceinline__ bool start(const AttnShape& s, const TileGeometry& g, const RunPlan& plan) {
        const int lane = static_cast<int>(threadIdx.x) & 31;
        end = min(plan.begin + plan.per, plan.total);
        if (plan.begin >= end) return false;
        b = plan.seq;
        rt = 0;
        load_seq(s, g);
        long long before = 0;
        for (int r0 = 0; r0 < row_tiles; r0 += 32) {
            const int r = r0 + lane;
            const long long n =
                r < row_tiles ? static_cast<long long>(item_units(tile_item(s, sq, g, r))) * s.kv_heads : 0;
            long long incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const unsigned found = __ballot_sync(0xffffffffu, before + incl > plan.in_seq);
            if (found != 0) {
                const int src = __ffs(static_cast<int>(found)) - 1;
                before += __shfl_sync(0xffffffffu, incl - n, src);
                rt = r0 + src;
                break;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        it = tile_item(s, sq, g, rt);
        const long long in = plan.in_seq - before;
        h = static_cast<int>(in / item_units(it));
        first = plan.begin - (in - static_cast<long long>(h) * item_units(it)) + kItemUnits;
        cut(plan.begin);
        return t1 > t0 || next(s, g);
    }
    __device__ __forceinline__ bool next(const AttnShape& s, const TileGeometry& g) {
        first += it.tiles + kItemUnits;   // a run that goes on has finished this item
        if (first >= end) return false;
        if (++h == s.kv_heads) {
            h = 0;
            if (++rt == row_tiles) {
                rt = 0;
                ++b;
                if (!load_seq(s, g)) return false;
            }
            it = tile_item(s, sq, g, rt);
        }
        t0 = 0;
        t1 = static_cast<int>(min(end - first, static_cast<long long>(it.tiles)));
        return true;
    }
    __device__ __forceinline__ int groups(int tpg) const { return sq.q_len - rt * 2 * tpg > tpg ? 2 : 1; }
};

// Deals all sequences' units in equal runs.  A warp sums a sequence: a long chunk has many items.
__device__ __forceinline__ RunPlan plan_tiles(const AttnShape& s, const TileGeometry& g, unsigned long long* costs,
                                              RunPlan* shared) {
    constexpr int kWarps = kTileThreads / 32;
    __shared__ long long s_sum[kWarps];
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    auto fill = [&](int b0) {   // costs of sequences [b0, b0 + kPlanSeqs): units / kv_heads
        for (int b = b0 + warp; b < min(s.seqs, b0 + kPlanSeqs); b += kWarps) {
            const SeqInfo q = seq_info(s, b);
            const int tiles = (q.q_len + 2 * g.tokens - 1) / (2 * g.tokens);
            unsigned long long n = 0;
            for (int r = lane; r < tiles; r += 32)
                n += static_cast<unsigned long long>(item_units(tile_item(s, q, g, r)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if (lane == 0) costs[b - b0] = n;
        }
        __syncthreads();
    };
    long long mine = 0;
    for (int b0 = 0; b0 < s.seqs; b0 += kPlanSeqs) {
        if (b0 > 0) __syncthreads();
        fill(b0);
        for (int i = tid; i < min(s.seqs - b0, kPlanSeqs); i += kTileThreads) mine += static_cast<long long>(costs[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_sum[w];
    total *= s.kv_heads;
    const long long even = (total + gridDim.x - 1) / gridDim.x;
    const long long per = even > kTileMinUnits ? even : kTileMinUnits;
    const long long begin = per * blockIdx.x;
    if (tid == 0) *shared = RunPlan{total, per, begin, 0, s.seqs};
    __syncthreads();
    // the sequence of unit `begin`: warp 0 scans the costs 32 at a time
    long long before = 0;
    for (int b0 = 0; b0 < s.seqs && begin < total; b0 += kPlanSeqs) {
        if (s.seqs > kPlanSeqs) {
            __syncthreads();
            fill(b0);
        }
        const int count = min(s.seqs - b0, kPlanSeqs);
        if (warp == 0) {
            for (int i0 = 0; i0 < count && before <= begin; i0 += 32) {
                const long long n =
                    i0 + lane < count ? static_cast<long long>(costs[i0 + lane]) * s.kv_heads : 0;
                long long incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += up;
                }
                const long long prefix = before + incl - n;
                if (begin >= prefix && begin < prefix + n) {
                    shared->seq = b0 + i0 + lane;
                    shared->in_seq = begin - prefix;
                }
                before += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
    }
    __syncthreads();
    return *shared;
}

// Shared-memory matrix descriptors (128-byte swizzle, 8-row groups 1024 bytes apart) from the low word of the start
// address.  K-major operands (queries, keys) advance 32 bytes per 16 elements inside the 128-byte row; the values are
// the MN-major B operand, with 64-element blocks of the head `leading` bytes apart, and advance 16 rows per 16 keys.
__device__ __forceinline__ uint32_t sdesc_low(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t sdesc(uint32_t low, uint32_t leading) {
    const uint32_t high = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride offset, descriptor version, swizzle
    return static_cast<uint64_t>(high) << 32 | (low | (leading >> 4) << 16);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P1;\n\telect.sync _|P1, 0xffffffff;\n\tselp.b32 %0, 1, 0, P1;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulate, M = 128, N = n, A and B both bf16 or both fp16.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    const uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "setp.ne.b32 P1, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, P1;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "setp.ne.b32 P1, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, P1;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_st_16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, "
                 "%8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                   "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tc_ld_16(uint32_t taddr, float (&x)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
                 "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]),
                   "=f"(x[8]), "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]),
                   "=f"(x[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld_16(float (&x)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}],"
        " [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tc_ld_f32(uint32_t taddr, float (&x)[32]) {
    tc_ld_32x32b_x32(taddr, reinterpret_cast<uint32_t(&)[32]>(x));
}

// Waits for the tensor-memory loads; x is among them, so nothing that uses it moves before the wait.
__device__ __forceinline__ void tc_wait_ld_of(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]),
                 "+f"(x[7]), "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]),
                 "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]),
                 "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]), "+f"(x[24]),
                 "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29]), "+f"(x[30]),
                 "+f"(x[31])
                 :
                 : "memory");
}

// Nothing that uses x moves before this point.
__device__ __forceinline__ void pin(float (&x)[32]) {
    asm volatile("" : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                      "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                      "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]),
                      "+f"(x[22]), "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]),
                      "+f"(x[29]), "+f"(x[30]), "+f"(x[31]));
}

// x[i] = -inf outside lo <= i <= hi
__device__ __forceinline__ void mask32(float (&x)[32], int lo, int hi) {
    const uint32_t below = hi >= 31 ? 0xffffffffu : hi < 0 ? 0u : (2u << hi) - 1u;
    const uint32_t seen = lo <= 0 ? below : lo > 31 ? 0u : below & (0xffffffffu << lo);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = (seen >> i) & 1u ? x[i] : -INFINITY;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max32(const float (&x)[32]) {
    float a = max3(x[0], x[1], x[2]), b = max3(x[3], x[4], x[5]);
#pragma unroll
    for (int i = 6; i < 30; i += 4) {
        a = max3(a, x[i], x[i + 1]);
        b = max3(b, x[i + 2], x[i + 3]);
    }
    return max3(max3(a, x[30], x[31]), b, b);
}

// 32 softmax weights 2^(c s + neg), packed in pairs; their sum is added to `sum` (two halves).
template <typename T>
__device__ __forceinline__ void weights32(const float (&x)[32], uint64_t c2, uint64_t neg2, uint32_t (&pk)[16],
                                          uint64_t& sum_a, uint64_t& sum_b) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float a0, a1, b0, b1;
        unpair(fma2(pair(x[i], x[i + 1]), c2, neg2), a0, a1);
        unpair(fma2(pair(x[i + 2], x[i + 3]), c2, neg2), b0, b1);
        a0 = ex2(a0);
        a1 = ex2(a1);
        b0 = ex2(b0);
        b1 = ex2(b1);
        sum_a = add2(sum_a, pair(a0, a1));
        sum_b = add2(sum_b, pair(b0, b1));
        pk[i / 2] = pack2<T>(a0, a1);
        pk[i / 2 + 1] = pack2<T>(b0, b1);
    }
}

// The item's tile whose last rows lie past the sequence's end inside a page, if it is in this run; else -1.
__device__ __forceinline__ int ragged_tile(const TileWalk& w, int box_slots) {
    const int j = w.sq.keys >= w.it.base ? (w.sq.keys - w.it.base) / kTileKeys : -1;
    return j >= w.t0 && j < w.t1 && (w.sq.keys & (box_slots - 1)) != 0 ? j : -1;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kTileThreads, 1)
    attn_tile_kernel(const TileParams p, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using Cfg = TileCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_kv_full[Cfg::kStages], s_kv_empty[Cfg::kStages];
    __shared__ __align__(8) uint64_t s_q_full[Cfg::kQBufs][2], s_q_empty[Cfg::kQBufs][2];
    __shared__ __align__(8) uint64_t s_s_full[2], s_p_full[2][2], s_o_full[2], s_sync[2], s_done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_last[2];
    __shared__ long long s_counted[2];   // first tile of the last item that a group has counted
    __shared__ RunPlan s_plan;
    const AttnShape& sh = p.sh;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    const int tpg = p.geo.tokens;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t q_smem = smem_u32(smem);
    uint8_t* kv_ptr = smem + Cfg::kQAll;
    const uint32_t kv_smem = smem_u32(kv_ptr);

    if (tid == 0) {
        s_abort = 0;
        s_counted[0] = s_counted[1] = -1;
        for (int i = 0; i < Cfg::kStages; ++i) {
            mbar_init(smem_u32(&s_kv_full[i]), 1);
            mbar_init(smem_u32(&s_kv_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int b = 0; b < Cfg::kQBufs; ++b) {
                mbar_init(smem_u32(&s_q_full[b][i]), 1);
                mbar_init(smem_u32(&s_q_empty[b][i]), 1);
            }
            mbar_init(smem_u32(&s_s_full[i]), 1);
            mbar_init(smem_u32(&s_p_full[i][0]), 4);   // the group's warps
            mbar_init(smem_u32(&s_p_full[i][1]), 4);
            mbar_init(smem_u32(&s_o_full[i]), 1);
            mbar_init(smem_u32(&s_sync[i]), 4);
        }
        mbar_init(smem_u32(&s_done), 1);
        fence_mbar_init();
        tma_prefetch_map(&qmap);
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    if (warp == 8) {
        tc_alloc(smem_u32(&s_tmem), 512);
        tc_relinquish();
    }
    if (tpg * sh.group < 128) {   // rows of no token: zeros for good (the loads do not touch them)
        for (int i = tid; i < Cfg::kQAll / 16; i += kTileThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    }
    griddep_wait();
    griddep_launch_dependents();
    const RunPlan plan = plan_tiles(sh, p.geo, reinterpret_cast<unsigned long long*>(kv_ptr), &s_plan);
    tc_fence_before();
    fence_proxy_async_smem();   // the plan's and the zeros' generic writes before the first loads
    __syncthreads();
    tc_fence_after();
    const int* abort_flag = &s_abort;
    const unsigned long long limit = sh.wait_limit_ns;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        TileWalk w;
        bool more_items = w.start(sh, p.geo, plan);
        if (warp == 9 || warp == 10) {
            // ------------------------------------------------ loads of keys by warp 9, of values by warp 10
            // (with 16-slot pages a tile takes 16 loads: one warp cannot issue both's at the tensor cores' pace)
            uint32_t load = warp == 10 ? 1 : 0;   // tiles lie in the ring as K0 V0 K1 V1 ...
            const int boxes = kTileKeys / p.geo.box_slots;
            const int box = lane % boxes;   // of 1, 2, 4 or 8 per 64 elements (page_size is a multiple of 16)
            const CUtensorMap* map = warp == 10 ? &vmap : &kmap;
            bool ok = true;
            for (; more_items && ok; more_items = w.next(sh, p.geo)) {
                const int32_t* pages = sh.block_table + w.b * sh.table_stride;
                for (int j = w.t0; j < w.t1; ++j) {
                    const uint32_t stage = load % Cfg::kStages, round = load / Cfg::kStages;
                    const uint32_t full = smem_u32(&s_kv_full[stage]);
                    // boxes that no row sees come from outside the cache, as zeros
                    const int key = w.it.base + j * kTileKeys + box * p.geo.box_slots;
                    int page = -1;
                    if (lane < boxes && key < w.it.hi && key + p.geo.box_slots > w.it.lo)
                        page = checked_page(sh, pages, key);
                    page = __shfl_sync(0xffffffffu, page, box);
                    if (round > 0) ok = warp_wait(smem_u32(&s_kv_empty[stage]), (round - 1) & 1u, abort_flag, limit);
                    if (!ok) break;
                    if (sh.withhold != 0 && blockIdx.x == 0 && load == 0) {   // test hook: the first keys
                        load += 2;
                        continue;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, Cfg::kStageBytes);
                    __syncwarp();
                    if (lane < boxes * (DP / 64)) {
                        const int x = lane / boxes;
                        tma_load_4d(kv_smem + stage * Cfg::kStageBytes + x * (kTileKeys * 128) +
                                        box * p.geo.box_slots * 128,
                                    map, full, x * 64, key % sh.page_size, w.h, page);
                    }
                    __syncwarp();
                    load += 2;
                }
            }
            if (!ok) {
                if (lane == 0 && !*reinterpret_cast<volatile int*>(&s_abort)) {
                    s_abort = 1;
                    set_error(sh.err, KT_DEVERR_TIMEOUT_LOAD);
                }
                // loads still in flight land before the CTA ends (each wait bounded)
                int never = 0;
                for (int i = 0; i < Cfg::kStages && load >= 2; ++i) {
                    load -= 2;
                    mbar_wait(smem_u32(&s_kv_full[load % Cfg::kStages]), (load / Cfg::kStages) & 1u, &never,
                              kDrainLimitNs);
                }
            }
        } else if (warp == 11) {
            // ------------------------------------------------ loads of queries
            uint32_t item_no[2] = {0, 0};   // of each group
            bool ok = true;
            for (; more_items && ok; more_items = w.next(sh, p.geo)) {
                const int groups = w.groups(tpg);
                for (int i = 0; i < groups; ++i) {
                    const uint32_t buf = item_no[i] % Cfg::kQBufs, round = item_no[i] / Cfg::kQBufs;
                    if (round > 0) ok = warp_wait(smem_u32(&s_q_empty[buf][i]), (round - 1) & 1u, abort_flag, limit);
                    if (!ok) break;
                    ++item_no[i];
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&s_q_full[buf][i]);
                        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(tpg * sh.group * DP * 2));
                        for (int x = 0; x < DP; x += 64)
                            tma_load_3d(q_smem + (buf * 2 + i) * Cfg::kQBytes + (x / 64) * (128 * 128), &qmap, bar, x,
                                        w.h * sh.group, w.sq.first_token + (w.rt * 2 + i) * tpg);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                if (lane == 0 && !*reinterpret_cast<volatile int*>(&s_abort)) {
                    s_abort = 1;
                    set_error(sh.err, KT_DEVERR_TIMEOUT_LOAD);
                }
                int never = 0;
                for (int i = 0; i < 2; ++i)
                    for (uint32_t k = 0; k < Cfg::kQBufs && k < item_no[i]; ++k) {
                        const uint32_t n = item_no[i] - 1 - k;
                        mbar_wait(smem_u32(&s_q_full[n % Cfg::kQBufs][i]), (n / Cfg::kQBufs) & 1u, &never,
                                  kDrainLimitNs);
                    }
            }
        } else if (warp == 8 && elect_one()) {
            // ------------------------------------------------ MMAs, issued by one thread
            // The run is one stream of tiles, S one tile ahead of O, across the items' ends as well.
            constexpr uint32_t kIdescQK = idesc_f16<T>(kTileKeys, false);
            const int steps = (sh.head_dim + 15) / 16;   // of 16 elements: past the head, zeros in S and unused in O
            const uint32_t idesc_pv = idesc_f16<T>(steps * 16, true);
            struct Tile {
                int groups;
                bool first, last;   // of its item's tiles in this run
            };
            int ahead = w.t0;                                       // S's next tile, in item w
            struct Ring {
                uint32_t stage, parity;
                __device__ __forceinline__ void step() {   // K and V alternate
                    stage += 2;
                    if (stage >= Cfg::kStages) {
                        stage -= Cfg::kStages;
                        parity ^= 1u;
                    }
                }
            };
            Ring k_ring{0, 0}, v_ring{1, 0};
            // parities of each group's next query item and weights; query buffer
            uint32_t q_parity0 = 0, q_parity1 = 0, q_buf0 = 0, q_buf1 = 0, p_parity0 = 0, p_parity1 = 0;
            auto wait = [&](uint64_t& bar, uint32_t par) { return mbar_wait(smem_u32(&bar), par, abort_flag, limit); };
            auto tile_ahead = [&](Tile& t) {   // false: no more
                if (ahead == w.t1) {
                    more_items = more_items && w.next(sh, p.geo);
                    ahead = w.t0;
                }
                if (!more_items) return false;
                t = Tile{w.groups(tpg), ahead == w.t0, ahead + 1 == w.t1};
                ++ahead;
                return true;
            };
            auto qk = [&](auto group, const Tile& t) -> bool {   // S_i = Q_i K^T
                constexpr int i = decltype(group)::value;
                uint32_t& q_parity = i == 0 ? q_parity0 : q_parity1;
                uint32_t& buf = i == 0 ? q_buf0 : q_buf1;
                if (t.first && !wait(s_q_full[buf][i], q_parity)) return false;
                if (i == 0 && !wait(s_kv_full[k_ring.stage], k_ring.parity)) return false;
                tc_fence_after();
                const uint32_t a = sdesc_low(q_smem + (buf * 2 + i) * Cfg::kQBytes);
                const uint32_t b = sdesc_low(kv_smem + k_ring.stage * Cfg::kStageBytes);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    if (ks >= steps) break;
                    const uint32_t off = ((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4;
                    tc_mma_ss(kTmemS + i * 128, sdesc(a + off, 16), sdesc(b + off, 16), kIdescQK, ks > 0 ? 1u : 0u);
                }
                tc_commit(smem_u32(&s_s_full[i]));
                if (t.last) {
                    tc_commit(smem_u32(&s_q_empty[buf][i]));
                    if (Cfg::kQBufs == 1 || (buf ^= 1u) == 0) q_parity ^= 1u;
                }
                if (i + 1 == t.groups) {
                    tc_commit(smem_u32(&s_kv_empty[k_ring.stage]));
                    k_ring.step();
                }
                return true;
            };
            auto pv = [&](auto group, const Tile& t) -> bool {   // O_i (+)= P_i V
                constexpr int i = decltype(group)::value;
                uint32_t& p_parity = i == 0 ? p_parity0 : p_parity1;
                if (i == 0 && !wait(s_kv_full[v_ring.stage], v_ring.parity)) return false;
                const uint32_t b = sdesc_low(kv_smem + v_ring.stage * Cfg::kStageBytes);
                if (!wait(s_p_full[i][0], p_parity)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < kTileKeys / 16; ++ks) {
                    if (ks == kTileKeys / 32) {
                        if (!wait(s_p_full[i][1], p_parity)) return false;
                        tc_fence_after();
                    }
                    tc_mma_ts(kTmemO + i * DP, kTmemS + i * 128 + ks * 8,
                              sdesc(b + ((ks * 16 * 128) >> 4), kTileKeys * 128), idesc_pv,
                              ks > 0 || !t.first ? 1u : 0u);
                }
                p_parity ^= 1u;
                if (t.last) tc_commit(smem_u32(&s_o_full[i]));
                if (i + 1 == t.groups) {
                    tc_commit(smem_u32(&s_kv_empty[v_ring.stage]));
                    v_ring.step();
                }
                return true;
            };
            auto run = [&]() -> bool {
                const std::integral_constant<int, 0> group0{};
                const std::integral_constant<int, 1> group1{};
                Tile now{0, false, false}, next;   // (no groups before the first)
                while (true) {
                    const bool any = tile_ahead(next);
                    if (now.groups > 0 && !pv(group0, now)) return false;
                    if (any && !qk(group0, next)) return false;   // P has been read in that order
                    if (now.groups > 1 && !pv(group1, now)) return false;
                    if (!any) return true;
                    if (next.groups > 1 && !qk(group1, next)) return false;
                    now = next;
                }
            };
            if (!run() && !*reinterpret_cast<volatile int*>(&s_abort)) {
                s_abort = 1;
                set_error(sh.err, KT_DEVERR_TIMEOUT_MMA);
            }
            // every MMA has ended before the tensor memory is freed
            tc_commit(smem_u32(&s_done));
            int never = 0;
            mbar_wait(smem_u32(&s_done), 0, &never);
        }
    } else {
        // ---------------------------------------------------- softmax of one row per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int grp = warp >> 2;
        const int row = tid & 127;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = kTmemS + lane_base + grp * 128;
        const uint32_t t_o = kTmemO + lane_base + grp * DP;
        const float c = sh.scale_log2;
        const int row_tok = row / sh.group, row_head = row - row_tok * sh.group;   // token and head in its group
        const long long row_off = row_tok * p.o_token + row_head * p.o_head;
        uint32_t sync_no = 0;
        auto group_sync = [&]() {   // the group's four warps; bounded, as every wait here
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_sync[grp]));
            return warp_wait(smem_u32(&s_sync[grp]), sync_no++ & 1u, abort_flag, limit);
        };
        uint32_t tile_no = 0, item_no = 0, loads = 0;   // loads: key and value tiles of the items so far
        bool ok = true;
        TileWalk w;
        bool more = w.start(sh, p.geo, plan);
        // The pieces of a cut item lie with the CTA of its first tile (that CTA's slot 1) and the following ones (slot
        // 0); whoever counts last, as this says, clears the count for the next call.
        auto first_piece = [&]() { return static_cast<int>(w.first / plan.per); };
        auto last_piece = [&]() { return static_cast<int>((w.first + w.it.tiles - 1) / plan.per); };
        auto count_piece = [&]() -> bool {
            const int c0 = first_piece();
            const bool last = atomicAdd(&p.counters[2 * c0 + grp], 1u) == static_cast<unsigned>(last_piece() - c0);
            if (last) p.counters[2 * c0 + grp] = 0;
            return last;
        };
        for (; more && ok; more = w.next(sh, p.geo)) {
            if (grp >= w.groups(tpg)) continue;
            const int tok0 = (w.rt * 2 + grp) * tpg, tok = tok0 + row_tok;
            const bool valid = row_tok < tpg && tok < w.sq.q_len;
            const int pos = w.sq.first_pos + tok;
            // keys [first, last] are seen, and what all or some rows of the warp see; rows of no token compute without
            // masks and are not stored
            const int last = valid ? min(pos, w.sq.keys - 1) : 0x7fffffff;
            const int first = valid ? window_start(pos, sh.window) : 0;
            const int last_all = __reduce_min_sync(0xffffffffu, last);
            const int first_all = __reduce_max_sync(0xffffffffu, first);
            const int last_any = __reduce_max_sync(0xffffffffu, valid ? last : -1);
            const int first_any = __reduce_min_sync(0xffffffffu, valid ? first : 0x7fffffff);
            const int rag = ragged_tile(w, p.geo.box_slots);
            float m = -INFINITY, l = 0.0f;
            for (int j = w.t0; j < w.t1; ++j) {
                const int key0 = w.it.base + j * kTileKeys;
                ok = warp_wait(smem_u32(&s_s_full[grp]), tile_no & 1u, abort_flag, limit);
                if (!ok) break;
                ++tile_no;
                tc_fence_after();
                const bool masked = last_all < key0 + kTileKeys - 1 || first_all > key0;
                const int hi = last - key0, lo = first - key0;
                // the reference follows the maximum only when that has outgrown it (also from -inf)
                auto follow = [&](float top) {
                    const bool grown = (top - m) * c > kLazyLog2;
                    if (!__any_sync(0xffffffffu, grown)) return;
                    const float f = grown ? ex2((m - top) * c) : 1.0f;
                    if (grown) m = top;
                    l *= f;
                    if (j > w.t0) {
#pragma unroll 1
                        for (int q = 0; q < DP / 16; ++q) {
                            float o[16];
                            tc_ld_16(t_o + q * 16, o);
                            tc_wait_ld_16(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= f;
                            tc_st_16(t_o + q * 16, reinterpret_cast<const uint32_t(&)[16]>(o));
                        }
                    }
                };
                auto hand_over = [&](int part) {   // keys 0 to 63, then the others: the product starts with the first
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_p_full[grp][part]));
                };
                if (grp == 0 && j == rag) {
                    // Values past the sequence's end are whatever the page holds, and 0 x NaN is NaN: zeros, before
                    // this group lets the tile be multiplied (group 1's product is issued after it).
                    const uint32_t load = loads + 2 * static_cast<uint32_t>(j - w.t0) + 1;   // K0 V0 K1 V1 ...
                    const uint32_t st = load % Cfg::kStages;
                    ok = warp_wait(smem_u32(&s_kv_full[st]), (load / Cfg::kStages) & 1u, abort_flag, limit);
                    if (!ok) break;
                    const int past = w.sq.keys - key0;
                    const int end = (past / p.geo.box_slots + 1) * p.geo.box_slots;   // the rest was loaded as zeros
                    for (int i = row; i < (end - past) * (DP / 8); i += 128) {
                        const int r = past + i / (DP / 8), x = i % (DP / 8);
                        *reinterpret_cast<uint4*>(kv_ptr + st * Cfg::kStageBytes + (x >> 3) * (kTileKeys * 128) +
                                                  r * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                uint64_t sum_a = 0, sum_b = 0;   // two zeros each
                const uint64_t c2 = pair(c, c);
                if (!masked) {
                    float x[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tc_ld_f32(t_s + q * 32, x[q]);
                    tc_wait_ld_of(x[0]);
#pragma unroll
                    for (int q = 1; q < 4; ++q) pin(x[q]);
                    follow(max3(max3(max32(x[0]), max32(x[1]), max32(x[2])), max32(x[3]), m));
                    const float neg = m == -INFINITY ? 0.0f : -m * c;
                    const uint64_t neg2 = pair(neg, neg);
                    uint32_t pa[16], pb[16];
                    weights32<T>(x[0], c2, neg2, pa, sum_a, sum_b);
                    tc_st_16(t_s, pa);
                    weights32<T>(x[1], c2, neg2, pb, sum_a, sum_b);
                    tc_st_16(t_s + 16, pb);
                    weights32<T>(x[2], c2, neg2, pa, sum_a, sum_b);
                    weights32<T>(x[3], c2, neg2, pb, sum_a, sum_b);
                    hand_over(0);   // the first half's stores have landed meanwhile: no wait among the weights
                    tc_st_16(t_s + 32, pa);
                    tc_st_16(t_s + 48, pb);
                    hand_over(1);
                } else {
                    // The same by quarters, each read twice: what no row of the warp sees is skipped.  One copy of the
                    // code for the four, for a window's or a short prompt's tiles are all of this kind and straight
                    // code for them would not stay in the instruction cache.  (P of quarter q lies in S's columns of
                    // quarter q / 2, which have been read by then.)
                    auto dead = [&](int q) { return last_any < key0 + q * 32 || first_any > key0 + q * 32 + 31; };
                    auto load = [&](int q, float(&x)[32]) {
                        tc_ld_f32(t_s + q * 32, x);
                        tc_wait_ld_of(x);
                        if (last_all < key0 + q * 32 + 31 || first_all > key0 + q * 32)
                            mask32(x, lo - q * 32, hi - q * 32);
                    };
                    float top = m;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        if (dead(q)) continue;
                        float x[32];
                        load(q, x);
                        top = fmaxf(top, max32(x));
                    }
                    follow(top);
                    const float neg = m == -INFINITY ? 0.0f : -m * c;
                    const uint64_t neg2 = pair(neg, neg);
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        uint32_t pk[16] = {};
                        if (!dead(q)) {
                            float x[32];
                            load(q, x);
                            weights32<T>(x, c2, neg2, pk, sum_a, sum_b);
                        }
                        tc_st_16(t_s + q * 16, pk);
                        if (q & 1) hand_over(q >> 1);
                    }
                }
                float s0, s1;
                unpair(add2(sum_a, sum_b), s0, s1);
                l += s0 + s1;
            }
            if (!ok) break;
            loads += 2 * static_cast<uint32_t>(w.t1 - w.t0);
            ok = warp_wait(smem_u32(&s_o_full[grp]), item_no & 1u, abort_flag, limit);
            if (!ok) break;
            ++item_no;
            tc_fence_after();

            // ---- the item's piece is complete: store it, or leave it for the join
            const bool whole = w.t0 == 0 && w.t1 == w.it.tiles;
            const int rows = min(tpg, w.sq.q_len - tok0) * sh.group;   // of the group, that hold tokens
            T* const out0 = static_cast<T*>(p.out) + static_cast<long long>(w.sq.first_token + tok0) * p.o_token +
                            static_cast<long long>(w.h * sh.group) * p.o_head;   // of the group's first row
            auto closing = [&](int head, float mt, float lt) {   // 1 / sum, the sink's share included
                float scale_o = 1.0f;
                if (sh.sinks != nullptr) {
                    const float sk = sh.sinks[w.h * sh.group + head] * kLog2e;
                    const float mc = mt == -INFINITY ? -INFINITY : mt * c;
                    const float t = fmaxf(mc, sk);
                    const float tb = t == -INFINITY ? 0.0f : t;
                    scale_o = ex2(mc - tb);
                    lt = lt * scale_o + ex2(sk - tb);
                }
                return lt == 0.0f ? 0.0f : scale_o / lt;
            };
            // A row's 64 bytes lie with one lane; four lanes exchange 16-byte pieces, so as to write a row at a time
            // (16 scattered bytes a lane took 7.5 k cycles an item for the output).
            T* four[4];   // the rows of the lane's four (null: not stored), given its own
            auto meet = [&](T* own) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    four[k] = reinterpret_cast<T*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(own), (lane & ~3) + k));
            };
            auto store_64 = [&](uint32_t(&v)[16], int d) {   // elements [d, d + 32) of the rows
                const bool odd = lane & 1, upper = lane & 2;
#pragma unroll
                for (int i = 0; i < 16; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[i + k] : v[i + 4 + k], 1);
                        if (odd) v[i + k] = got;
                        else v[i + 4 + k] = got;
                    }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? v[k] : v[8 + k], 2);
                    if (upper) v[k] = got;
                    else v[8 + k] = got;
                }
                const int at = d + (lane & 3) * 8;
#pragma unroll
                for (int k = 0; k < 4; ++k)   // row k of the four
                    if (four[k] != nullptr && at < sh.head_dim)
                        *reinterpret_cast<uint4*>(four[k] + at) =
                            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            };
            if (whole) {
                const float inv = closing(row_head, m, l);
                meet(row < rows ? out0 + row_off : nullptr);
#pragma unroll 1
                for (int q = 0; q < DP / 32; ++q) {
                    float o[32];
                    tc_ld_f32(t_o + q * 32, o);
                    tc_wait_ld_of(o);
                    uint32_t v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = pack2<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
                    store_64(v, q * 32);
                }
                tc_fence_before();
                continue;
            }
            const int c0 = first_piece();
            const size_t slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
            const int prow = grp * 128 + row;
#pragma unroll 1
            for (int q = 0; q < DP / 32; ++q) {
                float o[32];
                tc_ld_f32(t_o + q * 32, o);
                tc_wait_ld_of(o);
#pragma unroll
                for (int i = 0; i < 32 && row < rows; i += 4)
                    p.part_o[(slot * (DP / 4) + (q * 32 + i) / 4) * 256 + prow] =
                        make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
            tc_fence_before();
            if (row < rows) p.part_ml[slot * 256 + prow] = make_float2(m, l);
            if (!(ok = group_sync())) break;
            if (row == 0) {
                __threadfence();
                s_last[grp] = count_piece();
                s_counted[grp] = w.first;
                __threadfence();
            }
            if (!(ok = group_sync())) break;
            if (!s_last[grp]) continue;
            // The join's time is that of its loads: few rows are shared out among all threads of the group, a part of
            // the head each, and eight loads of each of four pieces are under way.
            const int span = rows > 64 ? 128 : rows > 32 ? 64 : 32;   // rows to a part
            const int width = DP * span / 128 > 32 ? DP * span / 128 : 32;
            const int jrow = row % span, d0 = row / span * width;
            const bool joins = jrow < rows && d0 < DP;
            const int jtok = joins ? jrow / sh.group : 0, jhead = joins ? jrow - jtok * sh.group : 0;
            meet(joins ? out0 + jtok * p.o_token + jhead * p.o_head : nullptr);
            auto slot_of = [&](int k) { return 2 * static_cast<size_t>(c0 + k) + (k == 0 ? 1 : 0); };
            const int pieces = last_piece() - c0 + 1, jp = grp * 128 + (joins ? jrow : 0);
            float mt = -INFINITY, lt = 0.0f;
#pragma unroll 8
            for (int k = 0; k < pieces; ++k) mt = fmaxf(mt, __ldcg(&p.part_ml[slot_of(k) * 256 + jp]).x);
            const float mref = mt == -INFINITY ? 0.0f : mt;
#pragma unroll 8
            for (int k = 0; k < pieces; ++k) {
                const float2 ml = __ldcg(&p.part_ml[slot_of(k) * 256 + jp]);
                lt += ml.y * ex2((ml.x - mref) * c);
            }
            const float inv = closing(jhead, mt, lt);
#pragma unroll 1
            for (int q = 0; q < width; q += 32) {
                float acc[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = 0.0f;
                if (joins) {
#pragma unroll 4
                    for (int k = 0; k < pieces; ++k) {
                        const float f = ex2((__ldcg(&p.part_ml[slot_of(k) * 256 + jp]).x - mref) * c);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 v = __ldcg(&p.part_o[(slot_of(k) * (DP / 4) + (d0 + q + i) / 4) * 256 + jp]);
                            acc[i] += f * v.x;
                            acc[i + 1] += f * v.y;
                            acc[i + 2] += f * v.z;
                            acc[i + 3] += f * v.w;
                        }
                    }
                }
                uint32_t v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = pack2<T>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
                store_64(v, d0 + q);
            }
        }
        if (!ok) {
            if (!*reinterpret_cast<volatile int*>(&s_abort)) {
                s_abort = 1;
                set_error(sh.err, KT_DEVERR_TIMEOUT_EPI);
            }
            // the run's pieces that have not been counted are, so that the counters are zero after the call
            if (row == 0)
                for (; more; more = w.next(sh, p.geo))
                    if (grp < w.groups(tpg) && !(w.t0 == 0 && w.t1 == w.it.tiles) && s_counted[grp] != w.first)
                        count_piece();
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tc_dealloc(s_tmem, 512);
    }
}

static int tile_ctas() { return std::min(sm_count(), static_cast<int>(kAttnMaxCounters / 2)); }

size_t attn_tile_workspace_bytes() {
    const size_t c = static_cast<size_t>(tile_ctas());
    return c * 2 * 256 * (128 * sizeof(float) + sizeof(float2));
}

template <typename T, int DP>
static kt_status launch_tile_typed(const AttnArgs& a, cudaStream_t s) {
    using Cfg = TileCfg<DP>;
    TileParams p{};
    p.sh = attn_shape(a);
    p.out = a.out.ptr;
    p.o_token = a.out.token_stride;
    p.o_head = a.out.head_stride;
    p.geo.tokens = 128 / p.sh.group;
    p.geo.box_slots = a.kv.page_size & -a.kv.page_size;
    if (p.geo.box_slots > kTileKeys) p.geo.box_slots = kTileKeys;
    CUtensorMap qmap, kmap, vmap;
    const uint64_t qd[3] = {static_cast<uint64_t>(a.kv.head_dim), static_cast<uint64_t>(a.q.heads),
                            static_cast<uint64_t>(a.batch.tokens)};
    const uint64_t qs[2] = {2 * static_cast<uint64_t>(a.q.head_stride), 2 * static_cast<uint64_t>(a.q.token_stride)};
    const uint32_t qb[3] = {64, static_cast<uint32_t>(p.sh.group), static_cast<uint32_t>(p.geo.tokens)};
    if (!encode_tiled_map(&qmap, a.kv.dtype, a.q.ptr, 3, qd, qs, qb, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
        !encode_kv_map(&kmap, a.kv, false, p.geo.box_slots) || !encode_kv_map(&vmap, a.kv, true, p.geo.box_slots))
        return report(KT_ERR_CUDA, "tensor map encoding failed");
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(attn_tile_kernel<T, DP>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e != cudaSuccess) return cuda_status(e);
        attr_set[dev] = true;
    }
    const size_t c = static_cast<size_t>(tile_ctas());
    p.counters = a.counters;
    p.part_o = reinterpret_cast<float4*>(a.ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + c * 2 * 256 * 32);
    count_launches(1);
    return cuda_status(launch_chained(attn_tile_kernel<T, DP>, dim3(static_cast<unsigned>(c)), dim3(kTileThreads),
                                      Cfg::kSmem, s, static_cast<const TileParams&>(p),
                                      static_cast<const CUtensorMap&>(qmap), static_cast<const CUtensorMap&>(kmap),
                                      static_cast<const CUtensorMap&>(vmap)));
}

kt_status launch_attn_tile(const AttnArgs& a, cudaStream_t s) {
    const bool wide = a.kv.head_dim > 64;
    if (a.kv.dtype == KT_DTYPE_BF16)
        return wide ? launch_tile_typed<__nv_bfloat16, 128>(a, s) : launch_tile_typed<__nv_bfloat16, 64>(a, s);
    return wide ? launch_tile_typed<__half, 128>(a, s) : launch_tile_typed<__half, 64>(a, s);
}

}  // namespace kt
