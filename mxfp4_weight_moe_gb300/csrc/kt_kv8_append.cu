// kt_kv8_append.cu -- a step's keys (normed and rotated on the way) and values to
// the pages of an 8-bit key/value cache: e4m3 codes with a power of two for each
// block of 16 positions and head.
//
// A warp takes one block of one sequence, one head, keys or values: the scale needs
// all of the block's rows, and nobody else writes its codes or its scale, so there
// are no atomics and results are the same bits each time.  The block's new rows (at
// most 16 of at most 128 elements, 64 elements a lane) stay in registers as fp32
// from the loads to the codes.  Bound by memory (large steps) or by the chain of
// look-ups, cu_q -> block table -> old scale (decode steps).
//
// The step's queries go through the head-row kernel's code, in the same launch.
#include <algorithm>

#include "kt_head_rows_dev.cuh"
#include "kt_internal.h"

namespace kt {

constexpr int kBlk = KT_KV8_BLOCK;
constexpr int kAppendThreads = 128;
constexpr int kVec = 8;          // elements of a chunk; a lane owns two of a row
constexpr int kRowLanes = 8;     // lanes of a row of up to 128 elements
constexpr int kPassRows = 32 / kRowLanes;
constexpr int kPasses = kBlk / kPassRows;

// Blocks of sequence b are counted from here: a sequence of q tokens touches at most q / 16 + 2 of them.
__host__ __device__ __forceinline__ long long first_block(long long cu, int b) { return cu / kBlk + 2ll * b; }

// The last sequence whose blocks start at or before block u; the whole warp, 32 candidates at a time.
__device__ __forceinline__ int sequence_of_block(const Kv8AppendParams& p, long long u) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int lo = 0, n = p.seqs;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool before =
            at < n && first_block(min(max(p.cu_q[lo + at], 0), p.tokens), lo + at) <= u;
        const int last = max(__popc(__ballot_sync(0xffffffffu, before)) - 1, 0);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// e from -127 (a subnormal number) to 127.
__device__ __forceinline__ float power_of_two(int e) {
    return __uint_as_float(e < -126 ? 1u << 22 : static_cast<uint32_t>(e + 127) << 23);
}

// Four codes times 2^-shift, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float factor) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(w >> (16 * i))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        r |= static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(f.x * factor, f.y * factor)) << (16 * i);
    }
    return r;
}

template <typename T, int NORM>
__device__ __forceinline__ void kv8_append_block(const Kv8AppendParams& p, unsigned launch_block) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const unsigned blocks = static_cast<unsigned>(first_block(p.tokens, p.seqs));
    const int unit =
        static_cast<int>(launch_block / blocks) * (kAppendThreads / 32) + static_cast<int>(threadIdx.x >> 5);
    if (unit >= 2 * p.heads) return;
    const bool keys = unit < p.heads;
    const int h = keys ? unit : unit - p.heads;
    const Kv8Side& sd = p.side[keys ? 0 : 1];

    // ---- the block: positions [lo, hi) of it are new, tok0 + position its tokens
    const long long u = launch_block % blocks;
    const int b = sequence_of_block(p, u);
    const int t0 = min(max(p.cu_q[b], 0), p.tokens), t1 = min(max(p.cu_q[b + 1], t0), p.tokens);
    const int start = max(p.seq_lens[b], 0) - (t1 - t0);   // position of the first new token
    const long long j = u - first_block(t0, b);
    const int first = max(start, 0);
    if (j == 0 && start < 0 && t1 > t0 && lane == 0) set_error(p.err, KT_DEVERR_BAD_PAGE);
    const long long at = (static_cast<long long>(first / kBlk) + j) * kBlk;
    const long long end = static_cast<long long>(start) + (t1 - t0);
    if (j < 0 || at >= end) return;
    const int base = static_cast<int>(at);
    const int lo = max(first, base);
    int hi = static_cast<int>(min(end, at + kBlk));
    if (p.table != nullptr && hi > p.positions_end) {
        if (lane == 0) set_error(p.err, KT_DEVERR_BAD_POSITION);
        hi = p.positions_end;
    }
    // ---- new rows: lane c of a row owns the chunks that hold both halves of its rotated pairs
    const int c = lane % kRowLanes, r0 = lane / kRowLanes;
    const bool used = c * 2 * kVec < p.head_dim;
    const bool rotated = keys && c * 2 * kVec < p.rot;
    const bool apart = rotated && p.style == KT_ROPE_HALVES;
    const int half = p.rot / 2;
    const int e0 = apart ? kVec * c : 2 * kVec * c;
    const int e1 = apart ? half + kVec * c : 2 * kVec * c + kVec;
    uint4 x[kPasses][2];
    const T* src = static_cast<const T*>(sd.src) + h * sd.src_head;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int pos = base + i * kPassRows + r0;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (used && pos >= lo && pos < hi) {
            const T* row = src + (static_cast<long long>(t0) + (pos - start)) * sd.src_token;
            x[i][0] = *reinterpret_cast<const uint4*>(row + e0);
            x[i][1] = *reinterpret_cast<const uint4*>(row + e1);
        }
    }
    // ---- its place in the cache, looked up while the rows come
    const int index = base / p.page_size;
    int page = -1;
    if (index < p.max_pages) page = p.block_table[b * p.table_stride + index];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) set_error(p.err, KT_DEVERR_BAD_PAGE);
        return;
    }
    if (lo >= hi) return;
    const int slot = base - index * p.page_size;
    uint8_t* const scale_at =
        sd.scales + (static_cast<long long>(page) * (p.page_size / kBlk) + slot / kBlk) * p.heads + h;
    uint8_t* const block = sd.codes + page * sd.page + slot * sd.slot + h * sd.head;
    const int older = lo - base;   // rows of the block that were there before
    int exponent = p.least;
    const int old_byte = older > 0 ? *scale_at : p.least + 127;

    uint64_t y[kPasses][2][kVec / 2];
    uint64_t w0[kVec / 2], w1[kVec / 2];
    const bool normed = NORM != kNoNorm && keys && p.weight != nullptr;   // the same for the whole warp
    if (normed && used) {
        if (NORM == kWeightsTyped) {
            const uint4 a = load_weights<T, kVec>(p.weight, e0, p.weight_vector);
            const uint4 d = load_weights<T, kVec>(p.weight, e1, p.weight_vector);
            widen<T, kVec>(a, w0);
            widen<T, kVec>(d, w1);
        } else {
            const float* w = static_cast<const float*>(p.weight);
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) {
                w0[i] = pair(w[e0 + 2 * i], w[e0 + 2 * i + 1]);
                w1[i] = pair(w[e1 + 2 * i], w[e1 + 2 * i + 1]);
            }
        }
    }
    uint32_t top = 0;
    bool odd = false;   // an element that is not finite
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int pos = base + i * kPassRows + r0;
        const bool fresh = used && pos >= lo && pos < hi;
        widen<T, kVec>(x[i][0], y[i][0]);
        widen<T, kVec>(x[i][1], y[i][1]);
        if (normed) {
            uint64_t s2 = 0;       // two zeros
#pragma unroll
            for (int k = 0; k < kVec / 2; ++k) s2 = fma2(y[i][1][k], y[i][1][k], fma2(y[i][0][k], y[i][0][k], s2));
            float a, d;
            unpair(s2, a, d);
            float sum = a + d;
#pragma unroll
            for (int o = kRowLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float inv = rsqrtf(sum * p.inv_dim + p.eps);
            const uint64_t inv2 = pair(inv, inv);
            if (fresh) {
#pragma unroll
                for (int k = 0; k < kVec / 2; ++k) {
                    y[i][0][k] = mul2(mul2(y[i][0][k], w0[k]), inv2);
                    y[i][1][k] = mul2(mul2(y[i][1][k], w1[k]), inv2);
                }
            }
        }
        if (fresh && rotated) {
            uint64_t cs[kVec / 2], sn[kVec / 2];
            const float* row = p.table + static_cast<long long>(pos) * p.rot + kVec * c;
            load_turn<kVec>(row, row + half, cs, sn);
            if (apart) turn_halves<kVec>(y[i][0], y[i][1], cs, sn);
            else turn_interleaved<kVec>(y[i][0], y[i][1], cs, sn);
        }
        if (fresh) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                float a, d;
                unpair(y[i][k / 4][k % 4], a, d);
                const uint32_t ua = __float_as_uint(a) & 0x7fffffffu, ud = __float_as_uint(d) & 0x7fffffffu;
                odd = odd || max(ua, ud) >= 0x7f800000u;
                top = max(top, ua < 0x7f800000u ? ua : 0u);
                top = max(top, ud < 0x7f800000u ? ud : 0u);
            }
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    odd = __any_sync(0xffffffffu, odd);
    // least X with top <= 448 * 2^X = 1.75 * 2^(X + 8): a mantissa past 1.75 carries into the exponent
    if (top > 0) exponent = static_cast<int>((top + 0x1fffffu) >> 23) - 127 - 8;
    // A larger power that older tokens have is kept, one past p.most (another program's) as well: their codes mean it.
    const int old_exponent = old_byte - 127;
    if (old_byte == 255) exponent = p.most;
    else exponent = max(min(max(exponent, p.least), p.most), old_exponent);
    // a block with an element that is not finite is NaN as a whole, and stays so while it fills
    const int byte = odd || old_byte == 255 ? 255 : exponent + 127;
    if (lane == 0 && (older == 0 || byte != old_byte)) *scale_at = static_cast<uint8_t>(byte);
    if (older > 0 && exponent > old_exponent) {
        const float factor = power_of_two(max(old_exponent - exponent, -126));
        const int pieces = p.head_dim / 16;
        for (int i = lane; i < older * pieces; i += 32) {
            uint4* at16 = reinterpret_cast<uint4*>(block + (i / pieces) * sd.slot) + i % pieces;
            uint4 v = *at16;
            v.x = rescale4(v.x, factor);
            v.y = rescale4(v.y, factor);
            v.z = rescale4(v.z, factor);
            v.w = rescale4(v.w, factor);
            *at16 = v;
        }
    }
    const float inv_scale = power_of_two(-exponent);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kPassRows + r0;
        if (!used || base + r < lo || base + r >= hi) continue;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            uint32_t q[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < kVec / 2; ++k) {
                float a, d;
                unpair(y[i][part][k], a, d);
                q[k / 2] |= static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(a * inv_scale, d * inv_scale))
                            << (16 * (k & 1));
            }
            *reinterpret_cast<uint2*>(block + r * sd.slot + (part == 0 ? e0 : e1)) = make_uint2(q[0], q[1]);
        }
    }
}

template <typename T, int NORM>
__global__ void __launch_bounds__(kAppendThreads, 5) kv8_append_kernel(const Kv8AppendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    kv8_append_block<T, NORM>(p, blockIdx.x);
}
// The same and the queries, R rows a group: blocks from `blocks` on are the head rows'.  Keys and values come first:
// their chains are the longer ones (three prompts, below: 40.3 us; last, 41.6; among the queries' blocks, 41.1).
template <typename T, int NORM, int R, bool STREAM>
__global__ void __launch_bounds__(kAppendThreads, R > 1 ? 5 : 1)
    kv8_append_queries_kernel(const Kv8AppendParams p, const HeadRowsParams q, unsigned blocks) {
    static_assert(kAppendThreads == kRowThreads, "one launch");
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x < blocks) kv8_append_block<T, NORM>(p, blockIdx.x);
    else head_rows_block<T, 8, R, NORM, STREAM>(q, blockIdx.x - blocks);
}

template <typename T, int R, bool STREAM>
static cudaError_t launch_kv8_queries(const Kv8AppendParams& p, HeadRowsParams& q, unsigned blocks, cudaStream_t s) {
    const unsigned rows = plan_head_rows<8, R>(q);
    const bool normed = p.weight != nullptr || q.seg[0].weight != nullptr;
    count_launches(1);
    return launch_chained(!normed          ? kv8_append_queries_kernel<T, kNoNorm, R, STREAM>
                          : p.weight_f32   ? kv8_append_queries_kernel<T, kWeightsF32, R, STREAM>
                                           : kv8_append_queries_kernel<T, kWeightsTyped, R, STREAM>,
                          dim3(blocks + rows), dim3(kAppendThreads), 0, s, p, static_cast<const HeadRowsParams&>(q),
                          blocks);
}

template <typename T>
static cudaError_t launch_kv8_typed(const Kv8AppendParams& p, HeadRowsParams* q, bool wide, int dtype, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>(first_block(p.tokens, p.seqs)) *
                            static_cast<unsigned>((2 * p.heads + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    if (q != nullptr && wide) {
        // One row at a time where there are few, four for the loads under way where there are many (128 tokens of 64 +
        // 8 heads of 128: 4.16 us one at a time, 3.66 four, with norms 4.2 and 4.6; 250 tokens: 4.2 and 3.9, with norms
        // 5.5 and 4.9; three prompts of up to 3500 with norms: 83 and 40.3). One border for both, by which 128 tokens
        // lose 0.5 us without norms and win 0.4 with them. Many rows are marked to leave L2 first, as in the head-row
        // kernel's launcher. In a launch of their own the prompts' take 43.5 us, those of 48 single tokens 4.9, 3.3
        // here. (Queries that 16-byte loads do not fit have one.)
        const long long rows = static_cast<long long>(q->tokens) * q->seg[0].heads;
        if (rows < 12288) return launch_kv8_queries<T, 1, false>(p, *q, blocks, s);
        if (rows * q->head_dim * 4 > (128ll << 20)) return launch_kv8_queries<T, 4, true>(p, *q, blocks, s);
        return launch_kv8_queries<T, 4, false>(p, *q, blocks, s);
    }
    count_launches(1);
    const cudaError_t e = launch_chained(!p.weight        ? kv8_append_kernel<T, kNoNorm>
                                         : p.weight_f32   ? kv8_append_kernel<T, kWeightsF32>
                                                          : kv8_append_kernel<T, kWeightsTyped>,
                                         dim3(blocks), dim3(kAppendThreads), 0, s, p);
    return e != cudaSuccess || q == nullptr ? e : launch_head_rows(*q, dtype, wide, s);
}

cudaError_t launch_kv8_append(const Kv8AppendParams& p, HeadRowsParams* q, bool wide, int dtype, cudaStream_t s) {
    return dtype == KT_DTYPE_BF16 ? launch_kv8_typed<__nv_bfloat16>(p, q, wide, dtype, s)
                                  : launch_kv8_typed<__half>(p, q, wide, dtype, s);
}

}  // namespace kt
