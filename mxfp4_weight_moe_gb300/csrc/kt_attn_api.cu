// kt_attn_api.cu -- the C ABI declared in include/kt_attn.h: argument checks
// and the choice of kernel.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <cudaTypedefs.h>

#include "kt_attn_dev.cuh"

namespace kt {

static kt_status refuse(kt_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
static kt_status refuse(kt_status st, const char* fmt, ...) {
    char text[200];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return report(st, text);
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static bool is_16bit(int dtype) { return dtype == KT_DTYPE_BF16 || dtype == KT_DTYPE_FP16; }

// cuTensorMapEncodeTiled by way of the runtime, so that the library needs no link to the driver's; NULL without one.
static PFN_cuTensorMapEncodeTiled_v12000 find_encode() {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
               : nullptr;
}

static bool encode_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank, const uint64_t* dims,
                       const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle,
                       CUtensorMapL2promotion promotion) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = find_encode();
    if (!encode) return false;
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    cuuint64_t size[4] = {}, pitch[3] = {};
    cuuint32_t part[4] = {};
    for (int i = 0; i < rank; ++i) {
        size[i] = dims[i];
        part[i] = box[i];
        if (i > 0) pitch[i - 1] = strides[i - 1];
    }
    return encode(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), size, pitch, part, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_tiled_map(CUtensorMap* m, int dtype, const void* base, int rank, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box, CUtensorMapL2promotion promotion) {
    return encode_map(m, dtype == KT_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      base, rank, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, promotion);
}

bool encode_kv_map(CUtensorMap* m, const kt_paged_kv& kv, bool values, int box_slots) {
    const uint64_t dims[4] = {static_cast<uint64_t>(kv.head_dim), static_cast<uint64_t>(kv.page_size),
                              static_cast<uint64_t>(kv.heads), static_cast<uint64_t>(kv.num_pages)};
    const uint64_t strides[3] = {2 * static_cast<uint64_t>(values ? kv.v_slot_stride : kv.k_slot_stride),
                                 2 * static_cast<uint64_t>(values ? kv.v_head_stride : kv.k_head_stride),
                                 2 * static_cast<uint64_t>(values ? kv.v_page_stride : kv.k_page_stride)};
    const uint32_t box[4] = {64, static_cast<uint32_t>(box_slots), 1, 1};
    // L2 fetches in units that divide a row: what follows it in memory may be another head's, read much later
    const int row = 2 * kv.head_dim;
    const CUtensorMapL2promotion promotion = row % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                             : row % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                             : row % 64 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                              : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    return encode_tiled_map(m, kv.dtype, values ? kv.v : kv.k, 4, dims, strides, box, promotion);
}

bool encode_kv8_map(CUtensorMap* m, const kt_paged_kv& kv, bool values, int width, int box_slots,
                    CUtensorMapSwizzle swizzle) {
    const uint64_t dims[4] = {static_cast<uint64_t>(kv.head_dim), static_cast<uint64_t>(kv.page_size),
                              static_cast<uint64_t>(kv.heads), static_cast<uint64_t>(kv.num_pages)};
    const uint64_t strides[3] = {static_cast<uint64_t>(values ? kv.v_slot_stride : kv.k_slot_stride),
                                 static_cast<uint64_t>(values ? kv.v_head_stride : kv.k_head_stride),
                                 static_cast<uint64_t>(values ? kv.v_page_stride : kv.k_page_stride)};
    const uint32_t box[4] = {static_cast<uint32_t>(width), static_cast<uint32_t>(box_slots), 1, 1};
    const int row = kv.head_dim;   // L2 fetches as in encode_kv_map
    const CUtensorMapL2promotion promotion = row % 128 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                             : row % 64 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                             : CU_TENSOR_MAP_L2_PROMOTION_NONE;
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, values ? kv.v : kv.k, 4, dims, strides, box, swizzle, promotion);
}

static kt_status check_heads(const kt_heads* h, const char* name, size_t align, int64_t step) {
    if (h->heads <= 0 || h->heads > 65536) return refuse(KT_ERR_INVALID_ARG, "%s: %d heads", name, h->heads);
    if (!h->ptr) return refuse(KT_ERR_INVALID_ARG, "%s is a null pointer", name);
    if (h->token_stride < 0 || h->head_stride < 0) return refuse(KT_ERR_INVALID_ARG, "%s: negative stride", name);
    if (!aligned(h->ptr, align) || h->token_stride % step || h->head_stride % step)
        return refuse(KT_ERR_ALIGNMENT, "%s: pointer must be %zu-byte aligned, strides multiples of %d elements", name,
                      align, static_cast<int>(step));
    return KT_OK;
}

static kt_status check_cache(const kt_paged_kv* c) {
    if (!c) return refuse(KT_ERR_INVALID_ARG, "null cache descriptor");
    if (!is_16bit(c->dtype)) return refuse(KT_ERR_INVALID_ARG, "cache dtype %d is not bf16 or fp16", c->dtype);
    if (c->num_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
        return refuse(KT_ERR_INVALID_ARG, "cache sizes must be positive");
    if (c->page_size % 16 || c->page_size > 65536 || c->head_dim % 8 || c->head_dim > 128)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE,
                      "page_size=%d must be a multiple of 16 and head_dim=%d a multiple of 8 up to 128", c->page_size,
                      c->head_dim);
    if (!c->k || !c->v) return refuse(KT_ERR_INVALID_ARG, "null cache pointer");
    const int64_t st[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                           c->v_page_stride, c->v_slot_stride, c->v_head_stride};
    for (int64_t x : st) {
        if (x <= 0) return refuse(KT_ERR_INVALID_ARG, "cache strides must be positive");
        if (x % 8) return refuse(KT_ERR_ALIGNMENT, "cache strides must be multiples of 8 elements");
        if (x >= (int64_t(1) << 38)) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "cache stride too large");
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return refuse(KT_ERR_ALIGNMENT, "cache pointers must be 16-byte aligned");
    return KT_OK;
}

static kt_status check_cache8(const kt_paged_kv8* c) {
    if (!c) return refuse(KT_ERR_INVALID_ARG, "null cache descriptor");
    if (!is_16bit(c->dtype)) return refuse(KT_ERR_INVALID_ARG, "cache dtype %d is not bf16 or fp16", c->dtype);
    if (c->num_pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
        return refuse(KT_ERR_INVALID_ARG, "cache sizes must be positive");
    if (c->page_size % KT_KV8_BLOCK || c->page_size > 65536 || c->head_dim % 16 || c->head_dim > 128 ||
        c->heads > 65535)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE,
                      "page_size=%d must be a multiple of %d, head_dim=%d a multiple of 16 up to 128", c->page_size,
                      KT_KV8_BLOCK, c->head_dim);
    if (!c->k || !c->v || !c->k_scales || !c->v_scales) return refuse(KT_ERR_INVALID_ARG, "null cache pointer");
    const int64_t st[6] = {c->k_page_stride, c->k_slot_stride, c->k_head_stride,
                           c->v_page_stride, c->v_slot_stride, c->v_head_stride};
    for (int64_t x : st) {
        if (x <= 0) return refuse(KT_ERR_INVALID_ARG, "cache strides must be positive");
        if (x % 16) return refuse(KT_ERR_ALIGNMENT, "cache strides must be multiples of 16 bytes");
        if (x >= (int64_t(1) << 39)) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "cache stride too large");
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return refuse(KT_ERR_ALIGNMENT, "cache pointers must be 16-byte aligned");
    return KT_OK;
}

static kt_status check_batch(const kt_paged_batch* b) {
    if (!b) return refuse(KT_ERR_INVALID_ARG, "null batch descriptor");
    if (b->seqs < 0 || b->tokens < 0 || b->max_pages < 0 || b->table_stride < 0)
        return refuse(KT_ERR_INVALID_ARG, "negative batch size");
    if (b->seqs > 65536) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "%d sequences: at most 65536", b->seqs);
    if (b->seqs == 0 || b->tokens == 0) return KT_OK;
    if (!b->cu_q || !b->seq_lens || (b->max_pages > 0 && !b->block_table))
        return refuse(KT_ERR_INVALID_ARG, "null batch pointer");
    if (!aligned(b->cu_q, 4) || !aligned(b->seq_lens, 4) || !aligned(b->block_table, 4))
        return refuse(KT_ERR_ALIGNMENT, "batch arrays must be 4-byte aligned");
    return KT_OK;
}

static kt_status check_transform(const kt_head_transform* t, int head_dim, int dtype) {
    if (!t) return KT_OK;
    if (t->table) {
        if (t->style != KT_ROPE_HALVES && t->style != KT_ROPE_INTERLEAVED)
            return refuse(KT_ERR_INVALID_ARG, "style=%d is not a KT_ROPE_* value", t->style);
        if (t->positions <= 0 || t->rotary_dim <= 0)
            return refuse(KT_ERR_INVALID_ARG, "positions=%d and rotary_dim=%d must be positive", t->positions,
                          t->rotary_dim);
        if (t->rotary_dim % 8 || t->rotary_dim > head_dim)
            return refuse(KT_ERR_UNSUPPORTED_SHAPE, "rotary_dim=%d must be a multiple of 8 up to head_dim=%d",
                          t->rotary_dim, head_dim);
        if (!aligned(t->table, 16)) return refuse(KT_ERR_ALIGNMENT, "the rotation table must be 16-byte aligned");
    }
    if (t->q_weight || t->k_weight) {
        if (t->weight_dtype != dtype && t->weight_dtype != KT_DTYPE_F32)
            return refuse(KT_ERR_INVALID_ARG, "weight dtype must be the heads' or f32");
        if (!(std::isfinite(t->eps) && t->eps >= 0.0f))
            return refuse(KT_ERR_INVALID_ARG, "eps must be finite and >= 0");
        const size_t a = t->weight_dtype == KT_DTYPE_F32 ? 4 : 2;
        if (!aligned(t->q_weight, a) || !aligned(t->k_weight, a))
            return refuse(KT_ERR_ALIGNMENT, "norm weights must be aligned to their element");
    }
    return KT_OK;
}

static void fill_transform(HeadRowsParams& p, const kt_head_transform* t, int head_dim) {
    p.head_dim = head_dim;
    p.inv_dim = 1.0f / static_cast<float>(head_dim);
    if (!t) return;
    p.eps = t->eps;
    p.weight_f32 = t->weight_dtype == KT_DTYPE_F32;
    p.seg[0].weight = t->q_weight;
    p.seg[1].weight = t->k_weight;
    if (t->table) {
        p.table = t->table;
        p.positions_end = t->positions;
        p.rot = t->rotary_dim;
        p.style = t->style;
    }
}

static void dense(HeadSegment& s, const kt_heads* src, const kt_heads* dst) {
    s.src = src->ptr;
    s.src_token = src->token_stride;
    s.src_head = src->head_stride;
    s.heads = src->heads;
    if (dst) {
        s.dst = dst->ptr;
        s.dst_token = dst->token_stride;
        s.dst_head = dst->head_stride;
    }
}

// 16-byte accesses: every pointer and stride in use allows them, and chunk pairs of 16 elements tile the head.
static bool wide_rows(const HeadRowsParams& p) {
    bool ok = p.head_dim % 16 == 0 && p.rot % 16 == 0;
    for (const HeadSegment& s : p.seg) {
        if (!s.heads) continue;
        ok = ok && aligned(s.src, 16) && aligned(s.dst, 16) && s.src_token % 8 == 0 && s.src_head % 8 == 0 &&
             s.dst_token % 8 == 0 && s.dst_head % 8 == 0 && s.dst_page % 8 == 0;
    }
    return ok;
}

static bool too_many_rows(const HeadRowsParams& p) {
    // 32 lanes at most a row, and 31 bits of threads
    return static_cast<long long>(p.tokens) * (p.seg[0].heads + p.seg[1].heads + p.seg[2].heads) > INT_MAX / 32;
}

}  // namespace kt

using namespace kt;

extern "C" {

kt_status kt_qk_norm_rope(const kt_heads* q, const kt_heads* k, const kt_heads* q_out, const kt_heads* k_out,
                          const int32_t* positions, int tokens, int head_dim, int dtype,
                          const kt_head_transform* transform, int* err, void* stream) {
    report(KT_OK, "");
    if (!q || !q_out || !transform || (k && !k_out)) return refuse(KT_ERR_INVALID_ARG, "null descriptor");
    if (!is_16bit(dtype)) return refuse(KT_ERR_INVALID_ARG, "dtype %d is not bf16 or fp16", dtype);
    if (tokens < 0 || head_dim <= 0)
        return refuse(KT_ERR_INVALID_ARG, "tokens=%d must be >= 0 and head_dim=%d positive", tokens, head_dim);
    if (head_dim % 8 || head_dim > 256)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "head_dim=%d must be a multiple of 8 up to 256", head_dim);
    kt_status st = check_transform(transform, head_dim, dtype);
    if (st != KT_OK || tokens == 0) return st;
    if ((st = check_heads(q, "q", 8, 4)) != KT_OK || (st = check_heads(q_out, "q_out", 8, 4)) != KT_OK) return st;
    if (k && ((st = check_heads(k, "k", 8, 4)) != KT_OK || (st = check_heads(k_out, "k_out", 8, 4)) != KT_OK))
        return st;
    if (q_out->heads != q->heads || (k && k_out->heads != k->heads))
        return refuse(KT_ERR_INVALID_ARG, "outputs must have their inputs' heads");
    if (transform->table && !positions) return refuse(KT_ERR_INVALID_ARG, "a rotation needs positions");
    if (!aligned(positions, 4) || !aligned(err, 4)) return refuse(KT_ERR_ALIGNMENT, "positions and err: 4 bytes");
    HeadRowsParams p{};
    dense(p.seg[0], q, q_out);
    if (k) dense(p.seg[1], k, k_out);
    fill_transform(p, transform, head_dim);
    p.tokens = tokens;
    p.positions = positions;
    p.err = err;
    if (too_many_rows(p)) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "too many head rows");
    return cuda_status(launch_head_rows(p, dtype, wide_rows(p), static_cast<cudaStream_t>(stream)));
}

kt_status kt_kv_append(const kt_paged_kv* cache, const kt_paged_batch* batch, const kt_heads* k, const kt_heads* v,
                       const kt_heads* q, const kt_heads* q_out, const kt_head_transform* transform, int* err,
                       void* stream) {
    report(KT_OK, "");
    kt_status st;
    if ((st = check_cache(cache)) != KT_OK || (st = check_batch(batch)) != KT_OK) return st;
    if (!k || !v || (q && !q_out)) return refuse(KT_ERR_INVALID_ARG, "null descriptor");
    if ((st = check_transform(transform, cache->head_dim, cache->dtype)) != KT_OK) return st;
    if (batch->seqs == 0 || batch->tokens == 0) return KT_OK;
    if ((st = check_heads(k, "k", 8, 4)) != KT_OK || (st = check_heads(v, "v", 8, 4)) != KT_OK) return st;
    if (q && ((st = check_heads(q, "q", 8, 4)) != KT_OK || (st = check_heads(q_out, "q_out", 8, 4)) != KT_OK))
        return st;
    if (k->heads != cache->heads || v->heads != cache->heads || (q && q_out->heads != q->heads))
        return refuse(KT_ERR_INVALID_ARG, "k and v must have the cache's heads, q_out q's");
    if (!aligned(err, 4)) return refuse(KT_ERR_ALIGNMENT, "err must be 4-byte aligned");
    HeadRowsParams p{};
    if (q) dense(p.seg[0], q, q_out);
    dense(p.seg[1], k, nullptr);
    dense(p.seg[2], v, nullptr);
    fill_transform(p, transform, cache->head_dim);
    p.seg[1].dst = cache->k;
    p.seg[1].dst_page = cache->k_page_stride;
    p.seg[1].dst_token = cache->k_slot_stride;
    p.seg[1].dst_head = cache->k_head_stride;
    p.seg[1].paged = 1;
    p.seg[2].dst = cache->v;
    p.seg[2].dst_page = cache->v_page_stride;
    p.seg[2].dst_token = cache->v_slot_stride;
    p.seg[2].dst_head = cache->v_head_stride;
    p.seg[2].paged = 1;
    p.tokens = batch->tokens;
    p.cu_q = batch->cu_q;
    p.seq_lens = batch->seq_lens;
    p.block_table = batch->block_table;
    p.table_stride = batch->table_stride;
    p.seqs = batch->seqs;
    p.max_pages = batch->max_pages;
    p.page_size = cache->page_size;
    p.num_pages = cache->num_pages;
    p.err = err;
    if (too_many_rows(p)) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "too many head rows");
    return cuda_status(launch_head_rows(p, cache->dtype, wide_rows(p), static_cast<cudaStream_t>(stream)));
}

kt_status kt_kv8_append(const kt_paged_kv8* cache, const kt_paged_batch* batch, const kt_heads* k, const kt_heads* v,
                        const kt_heads* q, const kt_heads* q_out, const kt_head_transform* transform, int* err,
                        void* stream) {
    report(KT_OK, "");
    kt_status st;
    if ((st = check_cache8(cache)) != KT_OK || (st = check_batch(batch)) != KT_OK) return st;
    if (!k || !v || (q && !q_out)) return refuse(KT_ERR_INVALID_ARG, "null descriptor");
    if ((st = check_transform(transform, cache->head_dim, cache->dtype)) != KT_OK) return st;
    if (transform && transform->table && transform->rotary_dim % 16)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "rotary_dim=%d must be a multiple of 16", transform->rotary_dim);
    if (batch->seqs == 0 || batch->tokens == 0) return KT_OK;
    if ((st = check_heads(k, "k", 16, 8)) != KT_OK || (st = check_heads(v, "v", 16, 8)) != KT_OK) return st;
    if (q && ((st = check_heads(q, "q", 8, 4)) != KT_OK || (st = check_heads(q_out, "q_out", 8, 4)) != KT_OK))
        return st;
    if (k->heads != cache->heads || v->heads != cache->heads || (q && q_out->heads != q->heads))
        return refuse(KT_ERR_INVALID_ARG, "k and v must have the cache's heads, q_out q's");
    if (!aligned(err, 4)) return refuse(KT_ERR_ALIGNMENT, "err must be 4-byte aligned");
    if ((batch->tokens / KT_KV8_BLOCK + 2ll * batch->seqs) * (cache->heads / 2 + 1) > INT_MAX / 2)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "too many blocks");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Kv8AppendParams p{};
    p.side[0] = Kv8Side{k->ptr, k->token_stride, k->head_stride, cache->k, cache->k_scales, cache->k_page_stride,
                        cache->k_slot_stride, cache->k_head_stride};
    p.side[1] = Kv8Side{v->ptr, v->token_stride, v->head_stride, cache->v, cache->v_scales, cache->v_page_stride,
                        cache->v_slot_stride, cache->v_head_stride};
    p.tokens = batch->tokens;
    p.head_dim = cache->head_dim;
    p.heads = cache->heads;
    p.inv_dim = 1.0f / static_cast<float>(cache->head_dim);
    if (transform) {
        p.eps = transform->eps;
        p.weight = transform->k_weight;
        p.weight_f32 = transform->weight_dtype == KT_DTYPE_F32;
        p.weight_vector = aligned(transform->k_weight, 16);
        if (transform->table) {
            p.table = transform->table;
            p.positions_end = transform->positions;
            p.rot = transform->rotary_dim;
            p.style = transform->style;
        }
    }
    p.cu_q = batch->cu_q;
    p.seq_lens = batch->seq_lens;
    p.block_table = batch->block_table;
    p.table_stride = batch->table_stride;
    p.seqs = batch->seqs;
    p.max_pages = batch->max_pages;
    p.page_size = cache->page_size;
    p.num_pages = cache->num_pages;
    p.least = cache->dtype == KT_DTYPE_BF16 ? -117 : -14;
    // bf16: attention's fp32 sums hold 2^24 keys of 448 * 2^87 under weights of up to 2^8
    p.most = cache->dtype == KT_DTYPE_BF16 ? 87 : 7;
    p.err = err;
    HeadRowsParams h{};
    if (q) {
        dense(h.seg[0], q, q_out);
        fill_transform(h, transform, cache->head_dim);
        h.seg[1].weight = nullptr;
        h.tokens = batch->tokens;
        h.cu_q = batch->cu_q;
        h.seq_lens = batch->seq_lens;
        h.seqs = batch->seqs;
        h.max_pages = batch->max_pages;
        h.page_size = cache->page_size;
        h.num_pages = cache->num_pages;
        h.err = err;
        if (too_many_rows(h)) return refuse(KT_ERR_UNSUPPORTED_SHAPE, "too many head rows");
    }
    return cuda_status(launch_kv8_append(p, q ? &h : nullptr, q && wide_rows(h), cache->dtype, s));
}

size_t kt_paged_attention_workspace_bytes(void) {
    const size_t a = attn_split_workspace_bytes(), b = attn_tile_workspace_bytes();
    return KT_PAGED_ATTENTION_ZEROED + (a > b ? a : b);
}

// kt_paged_attention and kt_paged_attention8 after the checks of the cache (an 8-bit one has scales).
static kt_status attention_impl(const kt_paged_kv* cache, const uint8_t* k_scales, const uint8_t* v_scales,
                                const kt_paged_batch* batch, const kt_heads* q, const kt_heads* out, int max_q_len,
                                float scale, int window, const float* sinks, int* err, void* ws, size_t ws_bytes,
                                void* stream) {
    kt_status st;
    if ((st = check_batch(batch)) != KT_OK) return st;
    if (!q || !out) return refuse(KT_ERR_INVALID_ARG, "null descriptor");
    if (max_q_len < 0 || window < 0)
        return refuse(KT_ERR_INVALID_ARG, "max_q_len=%d and window=%d must be >= 0", max_q_len, window);
    if (!(std::isfinite(scale) && scale > 0.0f)) return refuse(KT_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (batch->seqs == 0 || batch->tokens == 0) return KT_OK;
    if ((st = check_heads(q, "q", 16, 8)) != KT_OK || (st = check_heads(out, "out", 16, 8)) != KT_OK) return st;
    if (out->heads != q->heads || q->heads % cache->heads)
        return refuse(KT_ERR_INVALID_ARG, "%d query heads (out: %d) over %d cache heads", q->heads, out->heads,
                      cache->heads);
    if (q->heads / cache->heads > 128)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "%d query heads per cache head: at most 128",
                      q->heads / cache->heads);
    if (static_cast<long long>(batch->tokens) * q->heads > INT_MAX / 2)
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "too many query rows");
    if (!aligned(sinks, 4) || !aligned(err, 4)) return refuse(KT_ERR_ALIGNMENT, "sinks and err: 4 bytes");
    if (!ws) return refuse(KT_ERR_INVALID_ARG, "null workspace");
    if (!aligned(ws, 256)) return refuse(KT_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < kt_paged_attention_workspace_bytes())
        return refuse(KT_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws_bytes,
                      kt_paged_attention_workspace_bytes());
    AttnArgs a{*cache, k_scales, v_scales, *batch, *q, *out, scale, window, sinks, err, static_cast<unsigned*>(ws),
               static_cast<uint8_t*>(ws) + KT_PAGED_ATTENTION_ZEROED};
    // The split kernel's tiles hold 16 query rows: it reads the keys once for chunks of up to so many. Over an 8-bit
    // cache it takes up to 32, which reads them twice, for what it keeps: weights in 11 bits or more (the tile kernel
    // rounds them to the element type) and NaN values with the tokens that see them. Its times at 32 rows (4 tokens of
    // 8 heads a cache head) and the tile kernel's, us: 64 sequences after 8191, heads of 128: 445 and 355, of 64: 290
    // and 296; 16 after 3000: 54.7 and 47.0; one after 16000: 29.0 and 28.5. At 16 rows: 231 and 355, 153 and 296, 37.2
    // and 47.1, 25.7 and 30.0; at 48, heads of 128: 657 and 358. The tile kernel loads its queries by TMA, which needs
    // strides.
    const long long rows = static_cast<long long>(max_q_len) * (q->heads / cache->heads);
    if (rows <= (k_scales != nullptr ? 32 : 16) || q->token_stride == 0 || q->head_stride == 0)
        return launch_attn_split(a, static_cast<int>(std::min(rows, 1024ll)), static_cast<cudaStream_t>(stream));
    return launch_attn_tile(a, static_cast<cudaStream_t>(stream));
}

kt_status kt_paged_attention(const kt_paged_kv* cache, const kt_paged_batch* batch, const kt_heads* q,
                             const kt_heads* out, int max_q_len, float scale, int window, const float* sinks, int* err,
                             void* ws, size_t ws_bytes, void* stream) {
    report(KT_OK, "");
    const kt_status st = check_cache(cache);
    if (st != KT_OK) return st;
    return attention_impl(cache, nullptr, nullptr, batch, q, out, max_q_len, scale, window, sinks, err, ws, ws_bytes,
                          stream);
}

kt_status kt_paged_attention8(const kt_paged_kv8* cache, const kt_paged_batch* batch, const kt_heads* q,
                              const kt_heads* out, int max_q_len, float scale, int window, const float* sinks,
                              int* err, void* ws, size_t ws_bytes, void* stream) {
    report(KT_OK, "");
    const kt_status st = check_cache8(cache);
    if (st != KT_OK) return st;
    const kt_paged_kv kv{cache->k,             cache->v,             cache->k_page_stride, cache->k_slot_stride,
                         cache->k_head_stride, cache->v_page_stride, cache->v_slot_stride, cache->v_head_stride,
                         cache->num_pages,     cache->page_size,     cache->heads,         cache->head_dim,
                         cache->dtype};
    return attention_impl(&kv, cache->k_scales, cache->v_scales, batch, q, out, max_q_len, scale, window, sinks, err, ws,
                          ws_bytes, stream);
}

}  // extern "C"
