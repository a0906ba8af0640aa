// kt_attn_split.cu -- attention over a paged cache for few query rows: every
// warp streams its own keys and values and keeps its own softmax state.
//
// An item is (sequence, cache head, 16 query rows): row r of a sequence is its
// new token r / group under query head r % group of the cache head's group, so
// the heads that share a cache head share its loads.  The keys an item sees are
// cut into units of 64 keys; all items' units form one line that is dealt to
// the CTAs in equal contiguous runs, so that one long sequence and many short
// ones keep the GPU equally busy.  An item inside one run is finished by its
// CTA; one that is cut leaves partial sums (maximum, sum, unnormalised output)
// in the workspace, and the CTA that finishes last joins them in order, so the
// result does not depend on which one that was.
#include <algorithm>

#include "kt_attn_dev.cuh"

namespace kt {

#ifndef KT_MINU
#define KT_MINU 2
#endif
constexpr int kSplitWarps = 4;
constexpr int kSplitKeys = 16;                          // keys of one warp's block
constexpr int kSplitUnit = kSplitWarps * kSplitKeys;    // keys of one unit
constexpr int kSplitRows = 16;
constexpr int kSplitCtasPerSm = 2;
constexpr int kSplitMinUnits = KT_MINU;                       // least units of a CTA's run

template <int DP>
struct SplitCfg {
    static constexpr int kBlockBytes = kSplitKeys * DP * 2;          // one of K, V
    static constexpr int kStages = DP == 128 ? 3 : 6;
    static constexpr int kRing = kStages * 2 * kBlockBytes;          // per warp
    static constexpr int kSmem = kSplitWarps * kRing + 1024;
};

struct SplitParams {
    AttnShape sh;
    const void* q;
    void* out;
    long long q_token, q_head, o_token, o_head;
    float* part_o;       // [CTAs][2][16][DP]
    float* part_ml;      // [CTAs][2][16][2]
    unsigned* counters;  // [CTAs]
};

// Keys that the 16 rows of row tile rt see: [lo, hi); units of the item (at least one, so that its rows are written).
struct SplitItem {
    int lo, hi, unit0, units;
};
__device__ __forceinline__ SplitItem split_item(const AttnShape& s, const SeqInfo& q, int rt) {
    SplitItem it;
    const int t0 = rt * kSplitRows / s.group;
    const int t1 = min((rt * kSplitRows + kSplitRows - 1) / s.group, q.q_len - 1);
    it.hi = max(0, min(q.first_pos + t1 + 1, q.keys));
    it.lo = s.window > 0 ? max(0, q.first_pos + t0 - s.window + 1) : 0;
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.unit0 = it.lo / kSplitUnit;
    it.units = max(1, (it.hi + kSplitUnit - 1) / kSplitUnit - it.unit0);
    return it;
}
__device__ __forceinline__ int split_row_tiles(const AttnShape& s, const SeqInfo& q) {
    return (q.q_len * s.group + kSplitRows - 1) / kSplitRows;
}
__device__ __forceinline__ long long split_seq_units(const AttnShape& s, int b) {
    const SeqInfo q = seq_info(s, b);
    const int tiles = split_row_tiles(s, q);
    long long n = 0;
    for (int rt = 0; rt < tiles; ++rt) n += split_item(s, q, rt).units;
    return n * s.kv_heads;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kSplitWarps * 32, kSplitCtasPerSm)
    attn_split_kernel(const SplitParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Cfg = SplitCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kSplitWarps][Cfg::kStages];
    __shared__ int s_abort, s_last;
    __shared__ float s_ml[kSplitWarps][kSplitRows][2];
    __shared__ RunPlan s_plan;
    const AttnShape& sh = p.sh;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    uint8_t* ring_base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = ring_base + warp * Cfg::kRing;
    float* merge = reinterpret_cast<float*>(ring_base);   // [warps][16][DP], once every warp has left its ring

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
    const RunPlan plan = plan_run<kSplitWarps * 32>(
        sh.seqs, kSplitMinUnits, [&](int b) { return split_seq_units(sh, b); }, &s_plan);
    long long left = min(plan.per, plan.total - plan.begin);
    if (left <= 0) return;

    int b = plan.seq;
    long long at = plan.in_seq;              // unit inside the sequence
    long long global = plan.begin;
    uint32_t loads = 0;                      // blocks this warp has consumed so far
    while (left > 0 && b < sh.seqs) {
        const SeqInfo sq = seq_info(sh, b);
        const int tiles = split_row_tiles(sh, sq);
        // item of unit `at`: row tiles in order, each with its cache heads side by side
        int rt = 0;
        SplitItem it{};
        for (; rt < tiles; ++rt) {
            it = split_item(sh, sq, rt);
            const long long n = static_cast<long long>(it.units) * sh.kv_heads;
            if (at < n) break;
            at -= n;
        }
        if (rt == tiles) {
            ++b;
            at = 0;
            continue;
        }
        const int h = static_cast<int>(at / it.units);
        const int uo = static_cast<int>(at - static_cast<long long>(h) * it.units);
        const int take = static_cast<int>(min(static_cast<long long>(it.units - uo), left));
        const int32_t* pages = sh.block_table + b * sh.table_stride;

        // ---- this warp's blocks: keys base + 64 i, i in [i0, i1)
        const int base = (it.unit0 + uo) * kSplitUnit + warp * kSplitKeys;
        int i0 = 0, i1 = take;
        while (i0 < i1 && base + i0 * kSplitUnit + kSplitKeys <= it.lo) ++i0;
        while (i1 > i0 && base + (i1 - 1) * kSplitUnit >= it.hi) --i1;
        int page_batch = -1, my_page = -1;
        auto issue = [&](int i) {   // whole warp; block i into its stage
            const int batch = (i - i0) >> 5;
            if (batch != page_batch) {
                page_batch = batch;
                const int mine = i0 + batch * 32 + lane;
                my_page = mine < i1 ? checked_page(sh, pages, base + mine * kSplitUnit) : -1;
            }
            const int page = __shfl_sync(0xffffffffu, my_page, (i - i0) & 31);
            if (lane == 0) {
                const uint32_t st = (loads + static_cast<uint32_t>(i - i0)) % Cfg::kStages;
                const uint32_t bar = smem_u32(&s_full[warp][st]);
                const int slot = (base + i * kSplitUnit) % sh.page_size;
                uint8_t* k = ring + st * 2 * Cfg::kBlockBytes;
                mbar_arrive_expect_tx(bar, 2 * Cfg::kBlockBytes);
#pragma unroll
                for (int x = 0; x < DP; x += 64) {
                    tma_load_4d(smem_u32(k + x * 2 * kSplitKeys), &kmap, bar, x, slot, h, page);
                    tma_load_4d(smem_u32(k + Cfg::kBlockBytes + x * 2 * kSplitKeys), &vmap, bar, x, slot, h, page);
                }
            }
        };
        const int n_blocks = i1 - i0;
        for (int i = 0; i < min(n_blocks, Cfg::kStages); ++i) issue(i0 + i);

        // ---- queries: rows g and g + 8 of the tile in the MMA's A layout
        const int g = lane >> 2, t4 = lane & 3;
        uint32_t qa[DP / 16][4];
        int last_key[2], first_key[2];   // what the row sees; nothing for a row of no token
        {
            const T* qp[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = rt * kSplitRows + g + 8 * e;
                const int tok = row / sh.group;
                const bool ok = tok < sq.q_len;
                last_key[e] = ok ? min(sq.first_pos + tok, sq.keys - 1) : -1;
                first_key[e] = window_start(sq.first_pos + tok, sh.window);
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
            if (!mbar_wait(smem_u32(&s_full[warp][st]), (seq_no / Cfg::kStages) & 1u, &s_abort)) {
                s_abort = 1;
                set_error(sh.err, KT_DEVERR_TIMEOUT_LOAD);
            }
            const uint32_t kb = smem_u32(ring + st * 2 * Cfg::kBlockBytes);
            const uint32_t vb = kb + Cfg::kBlockBytes;
            const int key0 = base + i * kSplitUnit;

            // ---- S = Q K^T, 16 rows x 16 keys
            float s0[4] = {0, 0, 0, 0}, s1[4] = {0, 0, 0, 0};
            const int krow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                uint32_t kf[4];
                const int chunk = (ks & 3) * 2 + ((lane >> 3) & 1);
                ldmatrix_x4(kf, kb + (ks >> 2) * 2048 + krow * 128 + ((chunk ^ (krow & 7)) << 4));
                mma_16816<T>(s0, qa[ks], kf[0], kf[1]);
                mma_16816<T>(s1, qa[ks], kf[2], kf[3]);
            }
            // ---- scale, mask, running maximum (base-2 exponents)
            float x[2][4];
            const int k0 = key0 + t4 * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int keys[4] = {k0, k0 + 1, k0 + 8, k0 + 9};
                const float raw[4] = {s0[2 * e], s0[2 * e + 1], s1[2 * e], s1[2 * e + 1]};
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    x[e][f] = keys[f] <= last_key[e] && keys[f] >= first_key[e] ? raw[f] * sh.scale_log2 : -INFINITY;
                float top = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float mn = fmaxf(m[e], top);
                const float base_m = mn == -INFINITY ? 0.0f : mn;
                const float scale = ex2(m[e] - base_m);
                m[e] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    x[e][f] = ex2(x[e][f] - base_m);
                    sum += x[e][f];
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
            uint32_t pa[4] = {pack2<T>(x[0][0], x[0][1]), pack2<T>(x[1][0], x[1][1]), pack2<T>(x[0][2], x[0][3]),
                              pack2<T>(x[1][2], x[1][3])};
            const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3);
            const bool ragged = key0 + kSplitKeys > it.hi || key0 < it.lo;
#pragma unroll
            for (int n = 0; n < DP / 8; n += 2) {
                uint32_t vf[4];
                const int chunk = (n & 7) + (lane >> 4);
                ldmatrix_x4_trans(vf, vb + (n >> 3) * 2048 + vrow * 128 + ((chunk ^ (vrow & 7)) << 4));
                if (ragged) {
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const int key = k0 + (f & 1) * 8;
                        if (key >= it.hi || key < it.lo) vf[f] &= 0xffff0000u;
                        if (key + 1 >= it.hi || key + 1 < it.lo) vf[f] &= 0x0000ffffu;
                    }
                }
                mma_16816<T>(o[n], pa, vf[0], vf[1]);
                mma_16816<T>(o[n + 1], pa, vf[2], vf[3]);
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

        // ---- join the warps
        __syncthreads();
        {
            float* mo = merge + warp * kSplitRows * DP;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(mo + (g + 8 * e) * DP + n * 8 + t4 * 2) =
                        make_float2(o[n][2 * e], o[n][2 * e + 1]);
            if (t4 == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s_ml[warp][g + 8 * e][0] = m[e];
                    s_ml[warp][g + 8 * e][1] = l[e];
                }
            }
        }
        __syncthreads();
        const bool whole = uo == 0 && take == it.units;
        const int row = tid >> 3, d0 = (tid & 7) * (DP / 8);
        float mt = -INFINITY, lt = 0.0f, acc[DP / 8];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) mt = fmaxf(mt, s_ml[w][row][0]);
        const float mb = mt == -INFINITY ? 0.0f : mt;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
            const float f = ex2(s_ml[w][row][0] - mb);
            lt += f * s_ml[w][row][1];
            const float* mo = merge + (w * kSplitRows + row) * DP + d0;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) acc[i] += f * mo[i];
        }

        auto store = [&]() {   // acc, mt, lt -> the output row
            const int r = rt * kSplitRows + row;
            const int tok = r / sh.group;
            if (tok >= sq.q_len) return;
            const int head = h * sh.group + r - tok * sh.group;
            if (sh.sinks != nullptr) {
                const float sk = sh.sinks[head] * kLog2e;
                const float top = fmaxf(mt, sk);
                const float tb = top == -INFINITY ? 0.0f : top;
                const float f = ex2(mt - tb);
                lt = lt * f + ex2(sk - tb);
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) acc[i] *= f;
            }
            const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
            T* dst = static_cast<T*>(p.out) + static_cast<long long>(sq.first_token + tok) * p.o_token +
                     static_cast<long long>(head) * p.o_head;
#pragma unroll
            for (int i = 0; i < DP / 8; i += 8) {
                if (d0 + i >= sh.head_dim) break;
                uint4 v;
                v.x = pack2<T>(acc[i] * inv, acc[i + 1] * inv);
                v.y = pack2<T>(acc[i + 2] * inv, acc[i + 3] * inv);
                v.z = pack2<T>(acc[i + 4] * inv, acc[i + 5] * inv);
                v.w = pack2<T>(acc[i + 6] * inv, acc[i + 7] * inv);
                *reinterpret_cast<uint4*>(dst + d0 + i) = v;
            }
        };

        if (whole) {
            store();
        } else {
            // pieces of the item: the CTA where it begins (its slot 1), then the following ones (slot 0)
            const long long first_unit = global - uo;
            const int c0 = static_cast<int>(first_unit / plan.per);
            const int c1 = static_cast<int>((first_unit + it.units - 1) / plan.per);
            const int slot = 2 * static_cast<int>(blockIdx.x) + (uo == 0 ? 1 : 0);
            float* po = p.part_o + (static_cast<size_t>(slot) * kSplitRows + row) * DP + d0;
            const bool used = (rt * kSplitRows + row) / sh.group < sq.q_len;   // rows of no token are not joined
#pragma unroll
            for (int i = 0; i < DP / 8 && used; i += 4)
                *reinterpret_cast<float4*>(po + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            if ((tid & 7) == 0) {
                p.part_ml[(slot * kSplitRows + row) * 2] = mt;
                p.part_ml[(slot * kSplitRows + row) * 2 + 1] = lt;
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned seen = atomicAdd(&p.counters[c0], 1u);
                s_last = seen == static_cast<unsigned>(c1 - c0);
                if (s_last) p.counters[c0] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                // maxima and sums of all pieces into shared memory, then their outputs, several loads under way
                const int pieces = c1 - c0 + 1;
                float2* ml = reinterpret_cast<float2*>(merge + kSplitWarps * kSplitRows * DP);   // [pieces][16]
                for (int i = tid; i < pieces * kSplitRows; i += kSplitWarps * 32) {
                    const int sl = 2 * (c0 + i / kSplitRows) + (i < kSplitRows ? 1 : 0);
                    ml[i] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + sl * kSplitRows + i % kSplitRows);
                }
                __syncthreads();
                mt = -INFINITY;
                for (int k = 0; k < pieces; ++k) mt = fmaxf(mt, ml[k * kSplitRows + row].x);
                const float top = mt == -INFINITY ? 0.0f : mt;
                lt = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) acc[i] = 0.0f;
                if (used) {
#pragma unroll 4
                    for (int k = 0; k < pieces; ++k) {
                        const float2 e = ml[k * kSplitRows + row];
                        const float f = ex2(e.x - top);
                        lt += f * e.y;
                        const float* src = p.part_o +
                                           static_cast<size_t>((2 * (c0 + k) + (k == 0 ? 1 : 0)) * kSplitRows + row) * DP +
                                           d0;
#pragma unroll
                        for (int i = 0; i < DP / 8; i += 4) {
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + i));
                            acc[i] += f * v.x;
                            acc[i + 1] += f * v.y;
                            acc[i + 2] += f * v.z;
                            acc[i + 3] += f * v.w;
                        }
                    }
                }
                store();
            }
        }
        // generic reads and writes of the merge area come before the next item's loads into it
        fence_proxy_async_smem();
        __syncthreads();

        // ---- next unit of the run
        at = static_cast<long long>(h) * it.units + uo + take;
        for (int r = 0; r < rt; ++r) at += static_cast<long long>(split_item(sh, sq, r).units) * sh.kv_heads;
        left -= take;
        global += take;
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
    p.part_o = reinterpret_cast<float*>(a.ws);
    p.part_ml = p.part_o + c * 2 * kSplitRows * 128;
    count_launches(1);
    return cuda_status(launch_chained(attn_split_kernel<T, DP>, dim3(static_cast<unsigned>(c)), dim3(kSplitWarps * 32),
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
