/*
 * kt_norm.h -- C ABI of the norm between the blocks of a decoder layer: the
 * residual's addition and the RMS norm of the hidden states, in front of the
 * attention's projection and of the MoE layer (kt_moe.h), whose tokens it can
 * write in MXFP8.
 *
 * Conventions are those of kt_moe.h.  Element types are KT_DTYPE_* (kt_attn.h).
 */
#ifndef KT_NORM_H
#define KT_NORM_H

#include "kt_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KT_NORM_MAX_HIDDEN 32768

/* [tokens, hidden]: element (t, i) at ptr + t*token_stride + i (elements of the
 * call's dtype); a NULL ptr leaves the operand out. */
typedef struct kt_token_rows {
    void* ptr;
    int64_t token_stride;
} kt_token_rows;

/*
 * s = x + residual (s = x without one) and y = s * weight / sqrt(mean(s^2) + eps)
 * of every token, in one pass and one launch:
 *   residual_out  s, rounded once to dtype (needs a residual)
 *   out           y, rounded once to dtype
 *   codes, scales y in MXFP8: e4m3 [tokens, hidden] and one e8m0 byte for each 32
 *                 elements [tokens, hidden / 32], by the rule of the MoE layer's
 *                 own quantisation (exponent floor(log2 amax) - 8,
 *                 rounded to nearest even, saturating), from the fp32 y
 * Any output may be NULL, but not all.  A token's bits do not depend on the call's
 * other tokens.  The sums are fp32, of the unrounded s: a token whose squares' sum
 * passes fp32's range (3.4e38) has zeros for y, and with eps 0 one whose squares
 * vanish below that range has no finite y.
 * dtype KT_DTYPE_BF16 or KT_DTYPE_FP16; weight [hidden] of dtype or KT_DTYPE_F32.
 * hidden: a multiple of 8 (of 32 for codes) up to KT_NORM_MAX_HIDDEN.  Pointers of
 * rows, weight and codes are 16-byte aligned, strides multiples of 8 elements.
 * out and residual_out may be x or residual (same pointer and stride) and share no
 * memory otherwise.  tokens == 0 is a no-op.
 * Errors: KT_ERR_INVALID_ARG, KT_ERR_UNSUPPORTED_SHAPE, KT_ERR_ALIGNMENT, KT_ERR_CUDA.
 */
kt_status kt_add_rms_norm(const kt_token_rows* x, const kt_token_rows* residual, const void* weight, int weight_dtype,
                          float eps, int tokens, int hidden, int dtype, const kt_token_rows* residual_out,
                          const kt_token_rows* out, uint8_t* codes, uint8_t* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KT_NORM_H */
