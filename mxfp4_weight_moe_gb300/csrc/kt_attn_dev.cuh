// kt_attn_dev.cuh -- device helpers of the paged-attention kernels: sequence
// geometry, the even division of all sequences' work among the CTAs, page
// look-up and the loads and matrix instructions both kernels use.
#pragma once

#include <math.h>

#include <type_traits>

#include "kt_attn_internal.h"
#include "kt_common.cuh"

namespace kt {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnShape {
    const int32_t* block_table;
    long long table_stride;
    const int32_t* cu_q;
    const int32_t* seq_lens;
    const float* sinks;
    int* err;
    int seqs, tokens, max_pages, num_pages, page_size;
    int kv_heads, group, head_dim, window;
    float scale_log2;   // scale * log2(e): the softmax runs on powers of two
    int withhold;       // test hook: the first CTA withholds its first load
    unsigned long long wait_limit_ns;
};

inline AttnShape attn_shape(const AttnArgs& a) {
    AttnShape s{};
    s.block_table = a.batch.block_table;
    s.table_stride = a.batch.table_stride;
    s.cu_q = a.batch.cu_q;
    s.seq_lens = a.batch.seq_lens;
    s.sinks = a.sinks;
    s.err = a.err;
    s.seqs = a.batch.seqs;
    s.tokens = a.batch.tokens;
    s.max_pages = a.batch.max_pages;
    s.num_pages = a.kv.num_pages;
    s.page_size = a.kv.page_size;
    s.kv_heads = a.kv.heads;
    s.group = a.q.heads / a.kv.heads;
    s.head_dim = a.kv.head_dim;
    s.window = a.window;
    s.scale_log2 = a.scale * kLog2e;
    const DebugSettings dbg = debug_settings();
    s.withhold = (dbg.flags & KT_DEBUG_WITHHOLD_STAGE) != 0;
    s.wait_limit_ns = dbg.wait_limit_ns;
    return s;
}

// Tiled tensor map of 16-bit elements (dims and box innermost first; strides in
// bytes for dims 1..rank-1, rank up to 4) in the 128-byte swizzle; false when it
// cannot be encoded.
bool encode_tiled_map(CUtensorMap* m, int dtype, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box, CUtensorMapL2promotion promotion);

// 4-D map (element, slot, head, page) of the cache's keys or values; a box is
// 64 elements x box_slots slots of one head and page in the 128-byte swizzle.
// Elements past head_dim and pages outside the cache read as zeros.
bool encode_kv_map(CUtensorMap* m, const kt_paged_kv& kv, bool values, int box_slots);

#ifdef __CUDACC__
// Sequence b of the step.  Nothing here goes past the step's tokens or the
// block table, whatever the arrays hold.
struct SeqInfo {
    int first_token, q_len;
    int first_pos;   // position of its first new token (negative: before the sequence)
    int keys;        // keys that can be read
};
__device__ __forceinline__ SeqInfo seq_info(const AttnShape& s, int b) {
    SeqInfo q;
    const int t0 = min(max(s.cu_q[b], 0), s.tokens), t1 = min(max(s.cu_q[b + 1], t0), s.tokens);
    const int len = max(s.seq_lens[b], 0);
    q.first_token = t0;
    q.q_len = t1 - t0;
    q.first_pos = len - q.q_len;
    const long long room = static_cast<long long>(s.max_pages) * s.page_size;
    q.keys = static_cast<int>(min(static_cast<long long>(len), room));
    if (q.keys < len && q.q_len > 0) set_error(s.err, KT_DEVERR_BAD_PAGE);
    return q;
}

// First key that a row at position pos sees (no difference that an int may not hold: pos can be negative).
__device__ __forceinline__ int window_start(int pos, int window) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// Page of key `key`, -1 (reads as zeros, and says so in the error word) when the table has none there.
__device__ __forceinline__ int checked_page(const AttnShape& s, const int32_t* pages, int key) {
    const int page = pages[key / s.page_size];
    if (page >= 0 && page < s.num_pages) return page;
    set_error(s.err, KT_DEVERR_BAD_PAGE);
    return -1;
}

// mbar_wait with one answer for the whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                          unsigned long long limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, limit_ns)) != 0;
}
constexpr uint64_t kDrainLimitNs = 1000000;   // for loads in flight to land, after a wait has run out

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}],"
        " [%2];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// The same, its lines the first to leave L2: for what is read once.
__device__ __forceinline__ uint64_t l2_policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_4d_once(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                                 int z, int w, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x),
        "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// D (16 x 8, fp32) += A (16 x 16, row-major) x B (16 x 8, column-major)
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma_16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x; -inf gives 0, results below the normal range are flushed.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats rounded to T, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The two halves of such a pair as floats.
template <typename T>
__device__ __forceinline__ float low_of(uint32_t v) {
    if (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(v << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(v)));
}
template <typename T>
__device__ __forceinline__ float high_of(uint32_t v) {
    if (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(v & 0xffff0000u);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(v >> 16)));
}
// A pair of T, what is larger than T's largest number (infinity) replaced by that, signs kept.
template <typename T>
__device__ __forceinline__ uint32_t finite_pair(uint32_t v);
template <>
__device__ __forceinline__ uint32_t finite_pair<__nv_bfloat16>(uint32_t v) {
    uint32_t r;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7f7f7f7fu));
    return r;
}
template <>
__device__ __forceinline__ uint32_t finite_pair<__half>(uint32_t v) {
    uint32_t r;
    asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7bff7bffu));
    return r;
}
#endif

}  // namespace kt
