// kt_add_rms_norm.cu -- the residual's addition and the RMS norm of token rows,
// results in 16 bits and in MXFP8 (the C ABI of include/kt_norm.h).
//
// y = s w / sqrt(mean(s^2) + eps), s = x + residual.  One pass: a row stays in
// registers as fp32 between its sum of squares and its outputs, so that x and the
// residual are read once.  A chunk of 8 elements (16 bytes) belongs to one thread;
// the 32 elements of an MXFP8 scale to four neighbouring lanes.  Bound by memory
// for many rows (8192 tokens of 7168 in 78.0 us, the measured copy rate), by latency
// for few.
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "kt_attn_dev.cuh"
#include "kt_internal.h"
#include "kt_norm.h"

namespace kt {

struct NormParams {
    const void* x;
    const void* residual;
    const void* weight;
    void* residual_out;
    void* out;
    uint8_t* codes;
    uint8_t* scales;
    long long x_stride, r_stride, ro_stride, o_stride;
    int tokens, hidden;
    float eps;
    int weight_f32;
};

template <typename T>
__device__ __forceinline__ void widen8(const uint4& raw, float (&v)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = low_of<T>(w[i]);
        v[2 * i + 1] = high_of<T>(w[i]);
    }
}
template <typename T>
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

constexpr int kSmallRows = 4;   // rows a block where a row is one warp's

// CHUNKS chunks of 8 elements a thread; a row is a block's (as many warps as it takes), or a warp's (SMALL).
//
// A row's squares are summed in an order that its length alone decides, so that a token's bits do not depend on how
// many others are in the step.  Of a block's row: the eight of a chunk; the chunks of each group of 32 neighbouring
// ones, which a warp holds in both forms, by a butterfly; the groups i, i + 32, .. by lane i; the lanes by a butterfly.
template <typename T, int CHUNKS, bool SMALL>
__global__ void __launch_bounds__(SMALL ? kSmallRows * 32 : 1024) add_rms_norm_kernel(const NormParams p) {
    __shared__ float s_sum[32 * CHUNKS];   // of the groups of chunks
    griddep_wait();
    griddep_launch_dependents();
    const int kThreads = SMALL ? 32 : static_cast<int>(blockDim.x);   // of a row
    const int tid = SMALL ? static_cast<int>(threadIdx.x) % 32 : static_cast<int>(threadIdx.x);
    const long long token =
        SMALL ? static_cast<long long>(blockIdx.x) * kSmallRows + threadIdx.x / 32 : static_cast<long long>(blockIdx.x);
    const bool row = token < p.tokens;
    const int chunks = p.hidden >> 3;
    const T* x = static_cast<const T*>(p.x) + token * p.x_stride;
    const T* r = static_cast<const T*>(p.residual) + token * p.r_stride;
    uint4 rx[CHUNKS], rr[CHUNKS];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int at = tid + c * kThreads;
        rx[c] = rr[c] = make_uint4(0, 0, 0, 0);
        if (row && at < chunks) {
            rx[c] = reinterpret_cast<const uint4*>(x)[at];
            if (p.residual != nullptr) rr[c] = reinterpret_cast<const uint4*>(r)[at];
        }
    }
    float s[CHUNKS][8];
    constexpr int kSums = SMALL ? 1 : CHUNKS;
    float sums[kSums] = {};
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        float b[8];
        widen8<T>(rx[c], s[c]);
        widen8<T>(rr[c], b);
        float& q = sums[c % kSums];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[c][i] += b[i];
            q = fmaf(s[c][i], s[c][i], q);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int c = 0; c < kSums; ++c) sums[c] += __shfl_xor_sync(0xffffffffu, sums[c], o);
    float sum = sums[0];
    if (!SMALL) {
        const int warps = kThreads / 32, groups = warps * CHUNKS;
        if ((tid & 31) == 0) {
#pragma unroll
            for (int c = 0; c < kSums; ++c) s_sum[(tid >> 5) + c * warps] = sums[c];
        }
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if ((tid & 31) + 32 * c < groups) sum += s_sum[(tid & 31) + 32 * c];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    // The root to half a unit, by a Newton-Raphson step on 1 / r^2 - v (r + r (1 - v r^2) / 2): its error would move every
    // rounding of the row the same way.  Roots of 0 and of infinity are as they are: the step would make them NaN.
    const float v = sum / static_cast<float>(p.hidden) + p.eps;
    const float near = rsqrtf(v);
    const float inv = v > 0.0f && v < INFINITY ? fmaf(0.5f * near, fmaf(-v * near, near, 1.0f), near) : near;
    if (!row) return;   // a whole warp
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
        const int at = tid + c * kThreads;
        const bool mine = at < chunks;
        float y[8];
        if (mine) {
            if (p.residual_out != nullptr)
                reinterpret_cast<uint4*>(static_cast<T*>(p.residual_out) + token * p.ro_stride)[at] = narrow8<T>(s[c]);
            float w[8];
            if (p.weight_f32) {
                const float4 a = reinterpret_cast<const float4*>(p.weight)[2 * at];
                const float4 b = reinterpret_cast<const float4*>(p.weight)[2 * at + 1];
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
            } else {
                widen8<T>(reinterpret_cast<const uint4*>(p.weight)[at], w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = s[c][i] * inv * w[i];
            if (p.out != nullptr)
                reinterpret_cast<uint4*>(static_cast<T*>(p.out) + token * p.o_stride)[at] = narrow8<T>(y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        }
        if (p.codes != nullptr) {   // hidden is a multiple of 32: four lanes are inside or outside together
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(y[i]) & 0x7fffffffu);
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int X = mx_e4m3_block_exponent(amax);
            const float sc = exp2_neg(X);
            if (mine) {
                uint32_t q[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    q[i] = f32x2_to_e4m3x2_satfinite(y[4 * i] * sc, y[4 * i + 1] * sc) |
                           static_cast<uint32_t>(f32x2_to_e4m3x2_satfinite(y[4 * i + 2] * sc, y[4 * i + 3] * sc)) << 16;
                reinterpret_cast<uint2*>(p.codes + token * p.hidden)[at] = make_uint2(q[0], q[1]);
                if ((at & 3) == 0)
                    p.scales[token * (p.hidden >> 5) + (at >> 2)] = static_cast<uint8_t>(X + 127);
            }
        }
    }
}

template <typename T, int CHUNKS, bool SMALL>
static cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
    count_launches(1);
    const int chunks = p.hidden / 8;
    const int threads = SMALL ? kSmallRows * 32 : (chunks + 32 * CHUNKS - 1) / (32 * CHUNKS) * 32;
    const int blocks = SMALL ? (p.tokens + kSmallRows - 1) / kSmallRows : p.tokens;
    return launch_chained(add_rms_norm_kernel<T, CHUNKS, SMALL>, dim3(static_cast<unsigned>(blocks)),
                          dim3(static_cast<unsigned>(threads)), 0, s, p);
}

template <typename T>
static cudaError_t launch_norm_typed(const NormParams& p, cudaStream_t s) {
    const int chunks = p.hidden / 8;
    if (chunks <= 32) return launch_norm<T, 1, true>(p, s);
    if (chunks <= 128) return launch_norm<T, 4, true>(p, s);
    // Small steps: a chunk a thread (1 token of 7168: 2.3 us, 2.9 with four; 600 tokens of 2048: 2.4 and 3.3).  Large
    // ones: four, for the loads under way (8192 tokens of 7168, all outputs, 531 MB: 78.0 us, 6.8 TB/s, and 89.9 with
    // one).  They meet at 2 to 4 million elements (450 tokens of 7168: 5.0 and 5.2; 600: 5.8 and 5.0; 2000 of 2048: 5.0
    // and 5.4).
    if (static_cast<long long>(p.tokens) * chunks <= (1 << 19) && chunks <= 1024) return launch_norm<T, 1, false>(p, s);
    return launch_norm<T, 4, false>(p, s);
}

static bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static kt_status refuse(kt_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
static kt_status refuse(kt_status st, const char* fmt, ...) {
    char text[200];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return report(st, text);
}

static kt_status check_rows(const kt_token_rows* r, const char* name) {
    if (!r || !r->ptr) return KT_OK;
    if (r->token_stride < 0) return refuse(KT_ERR_INVALID_ARG, "%s: negative stride", name);
    if (!aligned(r->ptr, 16) || r->token_stride % 8)
        return refuse(KT_ERR_ALIGNMENT, "%s: pointer must be 16-byte aligned, the stride a multiple of 8 elements", name);
    return KT_OK;
}

}  // namespace kt

using namespace kt;

extern "C" kt_status kt_add_rms_norm(const kt_token_rows* x, const kt_token_rows* residual, const void* weight,
                                     int weight_dtype, float eps, int tokens, int hidden, int dtype,
                                     const kt_token_rows* residual_out, const kt_token_rows* out, uint8_t* codes,
                                     uint8_t* scales, void* stream) {
    report(KT_OK, "");
    if (dtype != KT_DTYPE_BF16 && dtype != KT_DTYPE_FP16)
        return refuse(KT_ERR_INVALID_ARG, "dtype %d is not bf16 or fp16", dtype);
    if (weight_dtype != dtype && weight_dtype != KT_DTYPE_F32)
        return refuse(KT_ERR_INVALID_ARG, "weight dtype must be the rows' or f32");
    if (tokens < 0 || hidden <= 0)
        return refuse(KT_ERR_INVALID_ARG, "tokens=%d must be >= 0 and hidden=%d positive", tokens, hidden);
    if (hidden % 8 || hidden > KT_NORM_MAX_HIDDEN || ((codes || scales) && hidden % 32))
        return refuse(KT_ERR_UNSUPPORTED_SHAPE, "hidden=%d must be a multiple of 8 (of 32 for codes) up to %d", hidden,
                      KT_NORM_MAX_HIDDEN);
    if (!(std::isfinite(eps) && eps >= 0.0f)) return refuse(KT_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!codes != !scales) return refuse(KT_ERR_INVALID_ARG, "codes and scales come together");
    const bool has_out = out && out->ptr, has_ro = residual_out && residual_out->ptr, has_r = residual && residual->ptr;
    if (tokens == 0) return KT_OK;
    if (!has_out && !has_ro && !codes) return refuse(KT_ERR_INVALID_ARG, "no output");
    if (has_ro && !has_r) return refuse(KT_ERR_INVALID_ARG, "residual_out needs a residual");
    if (!x || !x->ptr || !weight) return refuse(KT_ERR_INVALID_ARG, "null pointer argument");
    kt_status st;
    if ((st = check_rows(x, "x")) != KT_OK || (st = check_rows(residual, "residual")) != KT_OK ||
        (st = check_rows(residual_out, "residual_out")) != KT_OK || (st = check_rows(out, "out")) != KT_OK)
        return st;
    if (!aligned(weight, 16) || !aligned(codes, 16))
        return refuse(KT_ERR_ALIGNMENT, "weight and codes must be 16-byte aligned");
    NormParams p{};
    p.x = x->ptr;
    p.x_stride = x->token_stride;
    if (has_r) {
        p.residual = residual->ptr;
        p.r_stride = residual->token_stride;
    }
    if (has_ro) {
        p.residual_out = residual_out->ptr;
        p.ro_stride = residual_out->token_stride;
    }
    if (has_out) {
        p.out = out->ptr;
        p.o_stride = out->token_stride;
    }
    p.weight = weight;
    p.weight_f32 = weight_dtype == KT_DTYPE_F32;
    p.codes = codes;
    p.scales = scales;
    p.tokens = tokens;
    p.hidden = hidden;
    p.eps = eps;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == KT_DTYPE_BF16 ? launch_norm_typed<__nv_bfloat16>(p, s) : launch_norm_typed<__half>(p, s));
}
