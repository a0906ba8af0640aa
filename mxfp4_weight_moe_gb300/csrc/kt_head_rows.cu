// kt_head_rows.cu -- per-head RMS norm and position rotation of query and key
// heads, to dense outputs or into the pages of a key/value cache, values copied
// along.  One launch per call; the operator is bound by memory traffic (large
// steps) or by launch latency (decode steps).
#include <type_traits>

#include "kt_attn_dev.cuh"
#include "kt_internal.h"

namespace kt {

template <int VEC>
struct RawVec;
template <>
struct RawVec<8> {
    using type = uint4;
};
template <>
struct RawVec<4> {
    using type = uint2;
};

template <typename T>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
    if (std::is_same<T, __nv_bfloat16>::value) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pair(f.x, f.y);
}
// Chunks of VEC 16-bit elements to fp32 pairs and back (one rounding).
template <typename T, int VEC>
__device__ __forceinline__ void widen(const typename RawVec<VEC>::type& raw, uint64_t (&v)[VEC / 2]) {
    const uint32_t* t = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) v[i] = widen2<T>(t[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ typename RawVec<VEC>::type narrow(const uint64_t (&v)[VEC / 2]) {
    typename RawVec<VEC>::type raw;
    uint32_t* t = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        float lo, hi;
        unpair(v[i], lo, hi);
        t[i] = pack2<T>(lo, hi);
    }
    return raw;
}
__device__ __forceinline__ float half_of(uint64_t v, int which) {
    float lo, hi;
    unpair(v, lo, hi);
    return which ? hi : lo;
}
// (x, y) turned by (c, s)
__device__ __forceinline__ uint64_t turn(uint64_t v, float c, float s) {
    float x, y;
    unpair(v, x, y);
    return pair(x * c - y * s, y * c + x * s);
}
// Keeps the compiler from carrying what it has computed from v past this point.
__device__ __forceinline__ void forget(uint4& v) { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }
__device__ __forceinline__ void forget(uint2& v) { asm volatile("" : "+r"(v.x), "+r"(v.y)); }

// A chunk of norm weights of the heads' type (`vector`: it may be loaded at once).
template <typename T, int VEC>
__device__ __forceinline__ typename RawVec<VEC>::type load_weights(const void* weight, int at, bool vector) {
    const T* src = static_cast<const T*>(weight) + at;
    if (vector) return *reinterpret_cast<const typename RawVec<VEC>::type*>(src);
    typename RawVec<VEC>::type raw;
    const uint16_t* bits = reinterpret_cast<const uint16_t*>(src);
    uint32_t* t = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) t[i] = bits[2 * i] | static_cast<uint32_t>(bits[2 * i + 1]) << 16;
    return raw;
}

// Rotation of the chunks by their cosines and sines.
template <int VEC>
__device__ __forceinline__ void turn_halves(uint64_t (&a)[VEC / 2], uint64_t (&b)[VEC / 2],
                                            const uint64_t (&cs)[VEC / 2], const uint64_t (&sn)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const uint64_t u = fma2(a[i], cs[i], mul2(b[i], sn[i]) ^ 0x8000000080000000ull);   // the product negated
        b[i] = fma2(b[i], cs[i], mul2(a[i], sn[i]));
        a[i] = u;
    }
}
// Pair i of the first chunk turns by element i of the cosines, of the second by element VEC/2 + i.
template <int VEC>
__device__ __forceinline__ void turn_interleaved(uint64_t (&a)[VEC / 2], uint64_t (&b)[VEC / 2],
                                                 const uint64_t (&cs)[VEC / 2], const uint64_t (&sn)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        a[i] = turn(a[i], half_of(cs[i / 2], i & 1), half_of(sn[i / 2], i & 1));
        b[i] = turn(b[i], half_of(cs[VEC / 4 + i / 2], i & 1), half_of(sn[VEC / 4 + i / 2], i & 1));
    }
}

// Cosines and sines of VEC pairs.
template <int VEC>
__device__ __forceinline__ void load_turn(const float* cos, const float* sin, uint64_t (&cs)[VEC / 2],
                                          uint64_t (&sn)[VEC / 2]) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const float4 c = reinterpret_cast<const float4*>(cos)[i];
        const float4 s = reinterpret_cast<const float4*>(sin)[i];
        cs[2 * i] = pair(c.x, c.y);
        cs[2 * i + 1] = pair(c.z, c.w);
        sn[2 * i] = pair(s.x, s.y);
        sn[2 * i + 1] = pair(s.z, s.w);
    }
}

// Where a token's rows go: rotation position (negative: nothing of the token is written, for it has none such or, with
// kNoToken, is of no sequence), page and slot of the cache (page -1: keys and values are not written).
struct TokenPlace {
    int pos, page, slot;
};
constexpr int kNoToken = -2;
// tells: the caller reports what is wrong (a position, but for values: queries and keys do); which: segment that asks.
__device__ __forceinline__ TokenPlace place_of(const HeadRowsParams& p, int token, bool tells, int which) {
    TokenPlace t{0, -1, 0};
    if (p.cu_q != nullptr) {
        const int b = sequence_of_token(p.cu_q, p.seqs, token);
        if (b < 0) return TokenPlace{kNoToken, -1, 0};
        t.pos = p.seq_lens[b] - p.cu_q[b + 1] + token;
        if (which != 0) {
            const int index = t.pos >= 0 ? t.pos / p.page_size : -1;
            if (index >= 0 && index < p.max_pages) t.page = p.block_table[b * p.table_stride + index];
            if (t.page < 0 || t.page >= p.num_pages) {
                if (tells) set_error(p.err, KT_DEVERR_BAD_PAGE);
                t.page = -1;
            }
            t.slot = t.pos - index * p.page_size;
        }
    } else if (p.table != nullptr) {
        t.pos = p.positions[token];
    }
    if (p.table != nullptr && (t.pos < 0 || t.pos >= p.positions_end)) {
        if (tells && which != 2) set_error(p.err, KT_DEVERR_BAD_POSITION);
        t.pos = -1;
    } else if (p.table == nullptr) {
        t.pos = 0;
    }
    return t;
}

// Four heads a group and six blocks of 128 threads on an SM: measured on 8192 tokens of 64 + 8 heads of 128 (302 MB of
// rows) with norms, 54.1 us (49.9 us, 6.1 TB/s, with the rows marked to leave L2); two heads 58 to 62 us, three 56.3,
// six 56.7, fewer blocks 57.6.  (With norms, six blocks cost 44 bytes of spills a thread.)
constexpr int kRowThreads = 128, kRowBlocks = 6, kRowHeads = 4;
constexpr int kNoNorm = 0, kWeightsTyped = 1, kWeightsF32 = 2;

// A head row of D elements is handled by D / (2 VEC) lanes.  Lane j owns two
// chunks of VEC elements chosen so that both halves of every rotated pair are
// its own: for the halves style the chunks at VEC j and rot/2 + VEC j, for the
// interleaved one (and for elements past rot) the 2 VEC consecutive elements
// from 2 VEC j; in both, its pairs use the VEC cosines from VEC j.  So the
// rotation needs no exchange between lanes, the sum of squares one butterfly
// over the row's lanes (a power of two; those past the row idle), and an output
// may overwrite its input.
//
// A group of lanes takes R consecutive heads of one token and one of q, k, v:
// it issues the 2R loads at once, before it looks up the position and the page,
// and reads the cosines and the weights once for the R heads.
template <typename T, int VEC, int R, int NORM, bool STREAM>
__global__ void __launch_bounds__(kRowThreads, kRowBlocks) head_rows_kernel(const HeadRowsParams p) {
    using Raw = typename RawVec<VEC>::type;
    constexpr int kPairs = VEC / 2;
    griddep_wait();
    griddep_launch_dependents();
    const int lanes = p.lanes;
    const int j = static_cast<int>(threadIdx.x) & (lanes - 1);
    const unsigned unit = (blockIdx.x * static_cast<unsigned>(kRowThreads) + threadIdx.x) >> p.lanes_log2;
    const unsigned token = unit / static_cast<unsigned>(p.units_per_token);
    const int c = static_cast<int>(unit - token * static_cast<unsigned>(p.units_per_token));
    const int which = c >= p.seg[2].first_unit ? 2 : c >= p.seg[1].first_unit ? 1 : 0;
    const HeadSegment& sg = p.seg[which];
    const int h0 = (c - sg.first_unit) * R;
    const bool inside = token < static_cast<unsigned>(p.tokens);
    const int nh = inside && j < p.row_lanes ? min(R, sg.heads - h0) : 0;   // rows of this lane
    const int half = p.rot / 2;
    const bool rotated = j * 2 * VEC < p.rot;
    const bool apart = p.style == KT_ROPE_HALVES && rotated;
    const int e0 = apart ? VEC * j : 2 * VEC * j;
    const int e1 = apart ? half + VEC * j : 2 * VEC * j + VEC;

    Raw x[R][2];
    {
        const T* src = static_cast<const T*>(sg.src) + static_cast<long long>(token) * sg.src_token + h0 * sg.src_head;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r][0] = x[r][1] = Raw{};
            if (r < nh) {
                const Raw* s0 = reinterpret_cast<const Raw*>(src + e0);
                const Raw* s1 = reinterpret_cast<const Raw*>(src + e1);
                x[r][0] = STREAM ? __ldcs(s0) : *s0;
                x[r][1] = STREAM ? __ldcs(s1) : *s1;
            }
            src += sg.src_head;
        }
    }
    Raw w0{}, w1{};
    if (NORM == kWeightsTyped && sg.weight != nullptr && nh > 0) {
        w0 = load_weights<T, VEC>(sg.weight, e0, p.weight_vector);
        w1 = load_weights<T, VEC>(sg.weight, e1, p.weight_vector);
    }
    // position, and for a paged destination the rows' place in the cache
    T* dst = static_cast<T*>(sg.dst) + h0 * sg.dst_head;
    bool ok = nh > 0, turned = false;
    uint64_t cs[kPairs], sn[kPairs];
    if (inside) {
        const TokenPlace t = place_of(p, static_cast<int>(token), j == 0, which);
        ok = ok && t.pos >= 0 && (!sg.paged || t.page >= 0);
        dst += sg.paged ? t.page * sg.dst_page + t.slot * sg.dst_token : static_cast<long long>(token) * sg.dst_token;
        turned = ok && rotated && which != 2 && p.table != nullptr;
        if (turned) {
            const float* row = p.table + static_cast<long long>(t.pos) * p.rot + VEC * j;
            load_turn<VEC>(row, row + half, cs, sn);
        }
    }
    float inv[R];
    if (NORM != kNoNorm) {   // the whole warp, for its shuffles
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t a[kPairs], b[kPairs], s2 = 0;   // s2: two zeros
            widen<T, VEC>(x[r][0], a);
            widen<T, VEC>(x[r][1], b);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) s2 = fma2(b[i], b[i], fma2(a[i], a[i], s2));
            float lo, hi;
            unpair(s2, lo, hi);
            inv[r] = lo + hi;
        }
        for (int o = lanes / 2; o > 0; o >>= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) inv[r] += __shfl_xor_sync(0xffffffffu, inv[r], o);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            inv[r] = rsqrtf(inv[r] * p.inv_dim + p.eps);
            forget(x[r][0]);   // widened again below: the fp32 of all rows would take 16 R registers
            forget(x[r][1]);
        }
    }
    if (!ok) return;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= nh) break;
        if (which != 2) {
            uint64_t a[kPairs], b[kPairs];
            widen<T, VEC>(x[r][0], a);
            widen<T, VEC>(x[r][1], b);
            if (NORM != kNoNorm && sg.weight != nullptr) {
                const uint64_t inv2 = pair(inv[r], inv[r]);
                uint64_t u0[kPairs], u1[kPairs];
                if (NORM == kWeightsTyped) {
                    forget(w0);
                    forget(w1);
                    widen<T, VEC>(w0, u0);
                    widen<T, VEC>(w1, u1);
                } else {
                    const float* w = static_cast<const float*>(sg.weight);
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        u0[i] = pair(w[e0 + 2 * i], w[e0 + 2 * i + 1]);
                        u1[i] = pair(w[e1 + 2 * i], w[e1 + 2 * i + 1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < kPairs; ++i) {
                    a[i] = mul2(mul2(a[i], u0[i]), inv2);
                    b[i] = mul2(mul2(b[i], u1[i]), inv2);
                }
            }
            if (turned) {
                if (p.style == KT_ROPE_HALVES) turn_halves<VEC>(a, b, cs, sn);
                else turn_interleaved<VEC>(a, b, cs, sn);
            }
            x[r][0] = narrow<T, VEC>(a);
            x[r][1] = narrow<T, VEC>(b);
        }
        if (STREAM) {
            __stcs(reinterpret_cast<Raw*>(dst + e0), x[r][0]);
            __stcs(reinterpret_cast<Raw*>(dst + e1), x[r][1]);
        } else {
            *reinterpret_cast<Raw*>(dst + e0) = x[r][0];
            *reinterpret_cast<Raw*>(dst + e1) = x[r][1];
        }
        dst += sg.dst_head;
    }
}

template <typename T, int VEC, int R, bool STREAM>
static cudaError_t launch_rows(HeadRowsParams& p, cudaStream_t s) {
    int units = 0;
    for (HeadSegment& sg : p.seg) {
        sg.first_unit = units;
        units += (sg.heads + R - 1) / R;
    }
    p.units_per_token = units;
    p.row_lanes = p.head_dim / (2 * VEC);
    for (p.lanes_log2 = 0; (1 << p.lanes_log2) < p.row_lanes;) ++p.lanes_log2;
    p.lanes = 1 << p.lanes_log2;
    p.weight_vector = 1;
    for (const HeadSegment& sg : p.seg)
        if (reinterpret_cast<uintptr_t>(sg.weight) % (2 * VEC)) p.weight_vector = 0;
    const long long threads = static_cast<long long>(p.tokens) * units * p.lanes;
    const dim3 grid(static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads));
    count_launches(1);
    const bool norm = p.seg[0].weight != nullptr || p.seg[1].weight != nullptr;
    return launch_chained(!norm            ? head_rows_kernel<T, VEC, R, kNoNorm, STREAM>
                          : p.weight_f32   ? head_rows_kernel<T, VEC, R, kWeightsF32, STREAM>
                                           : head_rows_kernel<T, VEC, R, kWeightsTyped, STREAM>,
                          grid, dim3(kRowThreads), 0, s, static_cast<const HeadRowsParams&>(p));
}

template <typename T>
static cudaError_t launch_typed(HeadRowsParams& p, bool wide, cudaStream_t s) {
    const long long rows = static_cast<long long>(p.tokens) * (p.seg[0].heads + p.seg[1].heads + p.seg[2].heads);
    if (!wide) return launch_rows<T, 4, 1, false>(p, s);
    // few rows: one per group, so that they spread over the GPU; many: several, for the loads in flight
    if (rows < 16384) return launch_rows<T, 8, 1, false>(p, s);
    // Rows that pass through L2 (in and out, 128 MB of it) are marked to leave it first: 8192 tokens of 64 + 8 heads of
    // 128 in 49.4 us against 54.1.  What fits stays as it is: the projection has left it there, and attention reads it
    // next (2000 such tokens read and written in place of themselves: 11.4 us against 13.8 marked).
    if (rows * p.head_dim * 4 > (128ll << 20)) return launch_rows<T, 8, kRowHeads, true>(p, s);
    return launch_rows<T, 8, kRowHeads, false>(p, s);
}

cudaError_t launch_head_rows(HeadRowsParams& p, int dtype, bool wide, cudaStream_t s) {
    return dtype == KT_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(p, wide, s) : launch_typed<__half>(p, wide, s);
}

}  // namespace kt
