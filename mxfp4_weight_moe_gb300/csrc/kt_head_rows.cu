// kt_head_rows.cu -- per-head RMS norm and position rotation of query and key
// heads, to dense outputs or into the pages of a key/value cache, values copied
// along.  One launch per call; the operator is bound by memory traffic (large
// steps) or by launch latency (decode steps).
#include "kt_attn_internal.h"
#include "kt_common.cuh"
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

// A head row of D elements is handled by D / (2 VEC) lanes.  Lane j owns two
// chunks of VEC elements chosen so that both halves of every rotated pair are
// its own: for the halves style the chunks at VEC j and rot/2 + VEC j, for the
// interleaved one (and for elements past rot) the 2 VEC consecutive elements
// from 2 VEC j; in both, its pairs use the VEC cosines from VEC j.  So the
// rotation needs no exchange between lanes, the sum of squares one butterfly
// over the row's lanes (a power of two, `lanes`; those past the row idle), and
// an output may overwrite its input.
//
// A group of `lanes` lanes takes R consecutive heads of one token and one of
// q, k, v: it issues the 2R loads at once, before it looks up the position and
// the page, and reads the cosines once for the R heads.
template <typename T, int VEC, int R>
__global__ void __launch_bounds__(256) head_rows_kernel(const HeadRowsParams p) {
    using Raw = typename RawVec<VEC>::type;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = static_cast<int>(threadIdx.x) & (p.lanes - 1);
    const unsigned unit = (blockIdx.x * 256u + threadIdx.x) >> p.lanes_log2;
    const unsigned token = unit / static_cast<unsigned>(p.units_per_token);
    if (token >= static_cast<unsigned>(p.tokens)) return;   // whole groups
    const int c = static_cast<int>(unit - token * static_cast<unsigned>(p.units_per_token));
    const int which = c >= p.seg[2].first_unit ? 2 : c >= p.seg[1].first_unit ? 1 : 0;
    const HeadSegment& sg = p.seg[which];
    const int h0 = (c - sg.first_unit) * R;
    const int nh = min(R, sg.heads - h0);
    const int j = lane;
    const bool mine = j < p.row_lanes;
    const int half = p.rot / 2;
    const bool turned = p.table != nullptr && which != 2 && j * 2 * VEC < p.rot;
    const bool halves = p.style == KT_ROPE_HALVES && j * 2 * VEC < p.rot;
    const int e0 = halves ? VEC * j : 2 * VEC * j;
    const int e1 = halves ? half + VEC * j : 2 * VEC * j + VEC;

    Raw x[R][2];
    const T* src = static_cast<const T*>(sg.src) + static_cast<long long>(token) * sg.src_token + h0 * sg.src_head;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (mine && r < nh) {
            x[r][0] = *reinterpret_cast<const Raw*>(src + r * sg.src_head + e0);
            x[r][1] = *reinterpret_cast<const Raw*>(src + r * sg.src_head + e1);
        } else {
            x[r][0] = Raw{};
            x[r][1] = Raw{};
        }
    }

    // position, and for a paged destination the row's place in the cache
    long long dst_off = static_cast<long long>(token) * sg.dst_token;
    int pos = 0;
    bool ok = true;
    if (p.cu_q != nullptr) {
        const int b = sequence_of_token(p.cu_q, p.seqs, static_cast<int>(token));
        if (b < 0) return;   // belongs to no sequence
        pos = p.seq_lens[b] - p.cu_q[b + 1] + static_cast<int>(token);
        if (sg.paged) {
            const int page_index = pos >= 0 ? pos / p.page_size : -1;
            const int page = page_index >= 0 && page_index < p.max_pages
                                 ? p.block_table[b * p.table_stride + page_index]
                                 : -1;
            if (page < 0 || page >= p.num_pages) {
                if (lane == 0) set_error(p.err, KT_DEVERR_BAD_PAGE);
                ok = false;
            }
            dst_off = page * sg.dst_page + (pos - page_index * p.page_size) * sg.dst_token;
        }
    } else if (p.table != nullptr) {
        pos = p.positions[token];
    }
    if (p.table != nullptr && which != 2 && (pos < 0 || pos >= p.positions_end)) {
        if (lane == 0) set_error(p.err, KT_DEVERR_BAD_POSITION);
        ok = false;
    }
    if (!ok) return;   // the same for every lane of the group

    T* dst = static_cast<T*>(sg.dst) + dst_off + h0 * sg.dst_head;
    if (which == 2) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (mine && r < nh) {
                *reinterpret_cast<Raw*>(dst + r * sg.dst_head + e0) = x[r][0];
                *reinterpret_cast<Raw*>(dst + r * sg.dst_head + e1) = x[r][1];
            }
        }
        return;
    }

    float cs[VEC], sn[VEC];
    if (turned && mine) {
        const float* row = p.table + static_cast<long long>(pos) * p.rot + VEC * j;
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(row + i);
            *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(row + half + i);
        }
    }
    float w0[VEC], w1[VEC];
    if (sg.weight != nullptr && mine) {
        if (p.weight_f32) {
            const float* w = static_cast<const float*>(sg.weight);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                w0[i] = w[e0 + i];
                w1[i] = w[e1 + i];
            }
        } else {
            const T* w = static_cast<const T*>(sg.weight);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                w0[i] = to_f32(w[e0 + i]);
                w1[i] = to_f32(w[e1 + i]);
            }
        }
    }
    const unsigned group_mask = p.lanes == 32 ? 0xffffffffu
                                              : ((1u << p.lanes) - 1u) << ((threadIdx.x & 31u) & ~(p.lanes - 1u));
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float a[VEC], b[VEC];
        const T* t0 = reinterpret_cast<const T*>(&x[r][0]);
        const T* t1 = reinterpret_cast<const T*>(&x[r][1]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            a[i] = to_f32(t0[i]);
            b[i] = to_f32(t1[i]);
        }
        if (sg.weight != nullptr) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss += a[i] * a[i] + b[i] * b[i];
            for (int o = p.lanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group_mask, ss, o);
            const float inv = rsqrtf(ss * p.inv_dim + p.eps);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                a[i] *= inv * w0[i];
                b[i] *= inv * w1[i];
            }
        }
        if (!mine || r >= nh) continue;
        Raw y0, y1;
        T* o0 = reinterpret_cast<T*>(&y0);
        T* o1 = reinterpret_cast<T*>(&y1);
        if (turned) {
            if (p.style == KT_ROPE_HALVES) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = a[i] * cs[i] - b[i] * sn[i];
                    b[i] = b[i] * cs[i] + a[i] * sn[i];
                    a[i] = u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {   // pairs i/2 of the first chunk, VEC/2 + i/2 of the second
                    const float u = a[i] * cs[i / 2] - a[i + 1] * sn[i / 2];
                    a[i + 1] = a[i + 1] * cs[i / 2] + a[i] * sn[i / 2];
                    a[i] = u;
                    const float v = b[i] * cs[VEC / 2 + i / 2] - b[i + 1] * sn[VEC / 2 + i / 2];
                    b[i + 1] = b[i + 1] * cs[VEC / 2 + i / 2] + b[i] * sn[VEC / 2 + i / 2];
                    b[i] = v;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            o0[i] = from_f32<T>(a[i]);
            o1[i] = from_f32<T>(b[i]);
        }
        *reinterpret_cast<Raw*>(dst + r * sg.dst_head + e0) = y0;
        *reinterpret_cast<Raw*>(dst + r * sg.dst_head + e1) = y1;
    }
}

template <typename T, int VEC, int R>
static cudaError_t launch_rows(HeadRowsParams& p, cudaStream_t s) {
    int units = 0;
    for (int i = 0; i < 3; ++i) {
        p.seg[i].first_unit = units;
        units += (p.seg[i].heads + R - 1) / R;
    }
    p.units_per_token = units;
    p.row_lanes = p.head_dim / (2 * VEC);
    p.lanes_log2 = 0;
    while ((1 << p.lanes_log2) < p.row_lanes) ++p.lanes_log2;
    p.lanes = 1 << p.lanes_log2;
    const long long threads = static_cast<long long>(p.tokens) * units * p.lanes;
    count_launches(1);
    return launch_chained(head_rows_kernel<T, VEC, R>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256),
                          0, s, static_cast<const HeadRowsParams&>(p));
}

template <typename T>
static cudaError_t launch_typed(HeadRowsParams& p, bool wide, cudaStream_t s) {
    const long long rows = static_cast<long long>(p.tokens) * (p.seg[0].heads + p.seg[1].heads + p.seg[2].heads);
    if (!wide) return launch_rows<T, 4, 1>(p, s);
    // few rows: one per group, so that they spread over the GPU; many: four, for the loads in flight
    return rows < 16384 ? launch_rows<T, 8, 1>(p, s) : launch_rows<T, 8, 4>(p, s);
}

cudaError_t launch_head_rows(HeadRowsParams& p, int dtype, bool wide, cudaStream_t s) {
    return dtype == KT_DTYPE_BF16 ? launch_typed<__nv_bfloat16>(p, wide, s) : launch_typed<__half>(p, wide, s);
}

}  // namespace kt
