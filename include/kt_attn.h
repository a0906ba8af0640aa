/*
 * kt_attn.h -- C ABI of the attention operators that stand in front of the MoE
 * layer (kt_moe.h) in a decoder layer's serving path: the norm and rotation of
 * query and key heads, the append to a paged key/value cache, and the attention
 * of each sequence's new tokens over its pages.
 *
 * Conventions are those of kt_moe.h: device pointers unless stated otherwise,
 * buffers owned by the caller, calls asynchronous on `stream`, arguments checked
 * before anything is launched, no device memory allocated, sm_103a only.  The
 * descriptor structs are HOST structs, read during the call.  Element types are
 * KT_DTYPE_BF16 or KT_DTYPE_FP16; all arithmetic is fp32, rounded once to the
 * element type where a result is stored.  For the matrix product with the values,
 * attention holds its softmax weights in two parts of the element type where a
 * call has few query rows (max_q_len x group up to 16), and rounds them to the
 * element type, once, for chunks of more.
 */
#ifndef KT_ATTN_H
#define KT_ATTN_H

#include "kt_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KT_DTYPE_BF16 0
#define KT_DTYPE_FP16 1
#define KT_DTYPE_F32 2 /* norm weights only */

/* Further bits of a device error word (`err` below: an optional int32 that the
 * kernels OR bits into and never clear). */
#define KT_DEVERR_BAD_PAGE 0x20     /* a needed block-table entry was outside [0, num_pages), or a length
                                       outside the block table: nothing is written there; it reads as zeros */
#define KT_DEVERR_BAD_POSITION 0x40 /* a rotation position outside the table: that token is not written */
/* KT_DEVERR_TIMEOUT_* (kt_moe.h): a wait inside kt_paged_attention ran out; that call's results are undefined. */

/* [tokens, heads, head_dim]: element (t, h, d) at ptr + t*token_stride + h*head_stride + d (strides in elements). */
typedef struct kt_heads {
    void* ptr;
    int64_t token_stride;
    int64_t head_stride;
    int heads;
} kt_heads;

/*
 * A paged cache: slot s of page p of head h is the row k + p*k_page_stride +
 * s*k_slot_stride + h*k_head_stride (elements; v likewise), head_dim contiguous
 * elements.  page_size is a multiple of 16, head_dim a multiple of 8 up to 128;
 * pointers are 16-byte aligned and strides positive multiples of 8 elements.
 */
typedef struct kt_paged_kv {
    void* k;
    void* v;
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int num_pages, page_size, heads, head_dim;
    int dtype;
} kt_paged_kv;

/*
 * One step's sequences.  Sequence b has the tokens [cu_q[b], cu_q[b+1]) of the
 * step (possibly none) and seq_lens[b] keys in all, the step's own included:
 * its token t has position seq_lens[b] - cu_q[b+1] + t.  Position p lies in slot
 * p % page_size of page block_table[b*table_stride + p / page_size].  Entries
 * past a sequence's last page are not read as pages.  Tokens from cu_q[seqs] on
 * belong to no sequence and are left alone.
 */
typedef struct kt_paged_batch {
    const int32_t* block_table; /* [seqs, max_pages], rows table_stride apart */
    int64_t table_stride;
    int max_pages;
    const int32_t* cu_q;     /* [seqs + 1], cu_q[0] = 0, ascending */
    const int32_t* seq_lens; /* [seqs] */
    int seqs;
    int tokens; /* rows of q, k, v and out */
} kt_paged_batch;

/*
 * What happens to a query or key head before it is stored: the RMS norm
 * x * weight / sqrt(mean(x^2) + eps) where the weight (head_dim elements of
 * weight_dtype) is not NULL, then the rotation of the first rotary_dim elements
 * by the token's position where the table is not NULL:
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * for the pairs (i, i + rotary_dim/2) (KT_ROPE_HALVES) or (2i, 2i+1)
 * (KT_ROPE_INTERLEAVED), with cos = table[p][i], sin = table[p][rotary_dim/2 + i]
 * (f32 [positions, rotary_dim], rows contiguous, 16-byte aligned).
 */
#define KT_ROPE_HALVES 0
#define KT_ROPE_INTERLEAVED 1
typedef struct kt_head_transform {
    const float* table;
    int positions;
    int rotary_dim; /* multiple of 8, at most head_dim */
    int style;
    const void* q_weight;
    const void* k_weight;
    int weight_dtype; /* the heads' dtype or KT_DTYPE_F32 */
    float eps;
} kt_head_transform;

/*
 * Norm and rotation of q and k (k may be NULL) in one pass and one launch:
 * q_out = transform(q), k_out = transform(k).  An output may be its input (same
 * pointer and strides) and shares no memory otherwise.  positions: i32 [tokens], required with a table.
 * head_dim: multiple of 8 up to 256; pointers 8-byte aligned, strides multiples
 * of 4 elements.  tokens == 0 is a no-op.
 * Errors: KT_ERR_INVALID_ARG, KT_ERR_UNSUPPORTED_SHAPE, KT_ERR_ALIGNMENT, KT_ERR_CUDA.
 */
kt_status kt_qk_norm_rope(const kt_heads* q, const kt_heads* k, const kt_heads* q_out, const kt_heads* k_out,
                          const int32_t* positions, int tokens, int head_dim, int dtype,
                          const kt_head_transform* transform, int* err, void* stream);

/*
 * Append the step's keys (transformed; transform may be NULL) and values to the
 * cache, and, where q is not NULL, write q_out = transform(q), all in one
 * launch.  The rotation position is the position in the sequence.  q_out may be q
 * and shares no memory otherwise.
 */
kt_status kt_kv_append(const kt_paged_kv* cache, const kt_paged_batch* batch, const kt_heads* k, const kt_heads* v,
                       const kt_heads* q, const kt_heads* q_out, const kt_head_transform* transform, int* err,
                       void* stream);

/* Workspace bytes of kt_paged_attention on the current device (40 MB on 152 SMs:
 * partial results of two pieces of 256 query rows for each; the same for every
 * call).  Its first KT_PAGED_ATTENTION_ZEROED bytes are counters.  Calls of one
 * stream can share one. */
#define KT_PAGED_ATTENTION_ZEROED 4096
size_t kt_paged_attention_workspace_bytes(void);

/*
 * Attention of every sequence's new tokens over its pages (appended before):
 *   out[t, h] = sum_j softmax_j(scale * q[t, h] . k[j, h / group]) v[j, h / group]
 * over the keys j <= position(t), and j > position(t) - window where window > 0;
 * group = q heads / cache heads (a whole number, at most 128).  sinks (f32 [q
 * heads], may be NULL; finite or -inf) adds exp(sinks[h]) to the softmax's sum.
 * A token that sees no key gets zeros.  Pages that lie before every token's window
 * are not read, whatever their entries say.
 *   max_q_len  upper bound of the sequences' new tokens (picks the kernel form
 *              only; results hold for any value)
 *   scale      finite, > 0
 *   ws         >= kt_paged_attention_workspace_bytes() bytes, 256-byte aligned,
 *              its first KT_PAGED_ATTENTION_ZEROED bytes zeroed before the first
 *              use; every call leaves them zero
 * q and out: 16-byte aligned, strides multiples of 8 elements.  out may be q (same
 * pointer and strides) and shares no memory otherwise.
 */
kt_status kt_paged_attention(const kt_paged_kv* cache, const kt_paged_batch* batch, const kt_heads* q,
                             const kt_heads* out, int max_q_len, float scale, int window, const float* sinks, int* err,
                             void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KT_ATTN_H */
