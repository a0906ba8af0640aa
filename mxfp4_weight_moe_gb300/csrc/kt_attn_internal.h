// kt_attn_internal.h -- declarations shared by the attention operators'
// translation units: kernel parameters, launchers and small device helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kt_attn.h"
#include "kt_internal.h"

namespace kt {

// ------------------------------------------------------------- head rows
struct HeadSegment {
    const void* src;
    void* dst;
    long long src_token, src_head;            // strides in elements
    long long dst_page, dst_token, dst_head;  // dst_token: slot stride of a paged destination
    const void* weight;
    int heads;
    int first_unit;
    int paged;
};
struct HeadRowsParams {
    HeadSegment seg[3];   // q, k (transformed) and v (copied)
    int tokens, head_dim;
    float inv_dim, eps;
    const float* table;
    int positions_end, rot, style;
    int weight_f32;
    const int32_t* positions;   // dense form
    const int32_t* cu_q;        // paged form (NULL otherwise)
    const int32_t* seq_lens;
    const int32_t* block_table;
    long long table_stride;
    int seqs, max_pages, page_size, num_pages;
    int* err;
    int units_per_token, lanes, lanes_log2, row_lanes, weight_vector;   // set by the launcher
};
// wide: every pointer is 16-byte aligned, every stride a multiple of 8 and head_dim and rotary_dim multiples of 16.
cudaError_t launch_head_rows(HeadRowsParams& p, int dtype, bool wide, cudaStream_t s);

// ------------------------------------------------------------- append to an 8-bit cache
struct Kv8Side {   // keys or values
    const void* src;
    long long src_token, src_head;
    uint8_t* codes;
    uint8_t* scales;
    long long page, slot, head;   // strides of the codes in bytes
};
struct Kv8AppendParams {
    Kv8Side side[2];
    int tokens, head_dim, heads;
    float inv_dim, eps;
    const float* table;
    int positions_end, rot, style;
    const void* weight;   // of the keys
    int weight_f32, weight_vector;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    const int32_t* block_table;
    long long table_stride;
    int seqs, max_pages, page_size, num_pages;
    int least, most;      // scale exponents
    int* err;
};
// q: the step's queries (NULL for none), `wide` as launch_head_rows's of them.
cudaError_t launch_kv8_append(const Kv8AppendParams& p, HeadRowsParams* q, bool wide, int dtype, cudaStream_t s);

// ------------------------------------------------------------- attention
struct AttnArgs {
    kt_paged_kv kv;       // of an 8-bit cache: strides in bytes, which are its elements
    const uint8_t* k_scales;   // NULL for a 16-bit cache
    const uint8_t* v_scales;
    kt_paged_batch batch;
    kt_heads q, out;
    float scale;
    int window;
    const float* sinks;
    int* err;
    unsigned* counters;   // KT_PAGED_ATTENTION_ZEROED bytes
    uint8_t* ws;          // partial results
};
constexpr size_t kAttnMaxCounters = KT_PAGED_ATTENTION_ZEROED / sizeof(unsigned);
size_t attn_split_workspace_bytes();
// rows: at most so many query rows a sequence and cache head are likely (picks the form, not the result)
kt_status launch_attn_split(const AttnArgs& a, int rows, cudaStream_t s);
size_t attn_tile_workspace_bytes();
kt_status launch_attn_tile(const AttnArgs& a, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
    return __float2half_rn(x);
}

// Sequence of token t, -1 for a token of none: the last b with cu_q[b] <= t (a
// decode step's token t is usually that of sequence t, which is tried first).
__device__ __forceinline__ int sequence_of_token(const int32_t* cu_q, int seqs, int t) {
    if (t < seqs && cu_q[t] <= t && t < cu_q[t + 1]) return t;
    int lo = 0, hi = seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_q[mid] <= t) lo = mid;
        else hi = mid;
    }
    return seqs > 0 && cu_q[lo] <= t && t < cu_q[lo + 1] ? lo : -1;
}
#endif

}  // namespace kt
