// kt_head_dev.cuh -- device helpers of the kernels that norm and rotate head
// rows: chunks of 16-bit elements as fp32 pairs, norm weights, rotations.
#pragma once

#include <type_traits>

#include "kt_attn_dev.cuh"

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

}  // namespace kt
