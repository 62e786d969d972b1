// Vectors of V activations of type T (bf16, fp16 or fp32) in registers: raw
// words as loaded, widened to fp32 for arithmetic, rounded once (to nearest
// even) when stored.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace mhc {

typedef __nv_bfloat16 bf16;
typedef __half fp16;

template <class T, int V>
struct Vec {
    static constexpr int kBytes = int(sizeof(T)) * V;
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];
};

// Loads keep out of L1 (every element is used once) but are ordinary global
// loads, not read-only ones: an operator may be called in place.
template <class T, int V>
__device__ __forceinline__ void ld_vec(Vec<T, V> &v, const T *p)
{
    constexpr int B = Vec<T, V>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v.w[4 * i]), "=r"(v.w[4 * i + 1]), "=r"(v.w[4 * i + 2]),
                           "=r"(v.w[4 * i + 3])
                         : "l"(reinterpret_cast<const char *>(p) + 16 * i));
    } else if constexpr (B == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v.w[0] = u.x;
        v.w[1] = u.y;
    } else if constexpr (B == 4) {
        v.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        v.w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
}

// The same, kept in L1 for a second look.
template <class T, int V>
__device__ __forceinline__ void ld_vec_keep(Vec<T, V> &v, const T *p)
{
    constexpr int B = Vec<T, V>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            v.w[4 * i] = u.x;
            v.w[4 * i + 1] = u.y;
            v.w[4 * i + 2] = u.z;
            v.w[4 * i + 3] = u.w;
        }
    } else {
        ld_vec(v, p);
    }
}

template <class T, int V>
__device__ __forceinline__ void st_vec(T *p, const Vec<T, V> &v)
{
    constexpr int B = Vec<T, V>::kBytes;
    if constexpr (B >= 16) {
#pragma unroll
        for (int i = 0; i < B / 16; ++i)
            st_stream(reinterpret_cast<char *>(p) + 16 * i,
                      make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]));
    } else if constexpr (B == 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(v.w[0], v.w[1]);
    } else if constexpr (B == 4) {
        *reinterpret_cast<uint32_t *>(p) = v.w[0];
    } else {
        *reinterpret_cast<uint16_t *>(p) = uint16_t(v.w[0]);
    }
}

template <class T, int V>
__device__ __forceinline__ void zero_vec(Vec<T, V> &v)
{
#pragma unroll
    for (int i = 0; i < Vec<T, V>::kWords; ++i) v.w[i] = 0u;
}

__device__ __forceinline__ void widen2(uint32_t w, float &lo, float &hi, const bf16 *)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void widen2(uint32_t w, float &lo, float &hi, const fp16 *)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x;
    hi = f.y;
}
__device__ __forceinline__ uint32_t round2(float lo, float hi, const bf16 *) { return pack2(lo, hi); }
__device__ __forceinline__ uint32_t round2(float lo, float hi, const fp16 *)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <class T, int V>
__device__ __forceinline__ void widen(const Vec<T, V> &v, float (&f)[V])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(v.w[i]);
    } else if constexpr (V == 1) {
        float hi;
        widen2(v.w[0], f[0], hi, static_cast<const T *>(nullptr));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            widen2(v.w[i], f[2 * i], f[2 * i + 1], static_cast<const T *>(nullptr));
    }
}

template <class T, int V>
__device__ __forceinline__ void narrow(const float (&f)[V], Vec<T, V> &v)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) v.w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
        v.w[0] = round2(f[0], 0.f, static_cast<const T *>(nullptr));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            v.w[i] = round2(f[2 * i], f[2 * i + 1], static_cast<const T *>(nullptr));
    }
}

// V values for arithmetic: packed fp32 pairs (one instruction works on two
// values), or a single fp32 where V = 1.
__device__ __forceinline__ f32x2 e_mul(f32x2 a, f32x2 b) { return f2_mul(a, b); }
__device__ __forceinline__ float e_mul(float a, float b) { return a * b; }
__device__ __forceinline__ f32x2 e_fma(f32x2 a, f32x2 b, f32x2 c) { return f2_fma(a, b, c); }
__device__ __forceinline__ float e_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ void e_set(f32x2 &a, float v) { a = f2_make(v, v); }
__device__ __forceinline__ void e_set(float &a, float v) { a = v; }
__device__ __forceinline__ f32x2 e_neg(f32x2 a) { return a ^ 0x8000000080000000ull; }
__device__ __forceinline__ float e_neg(float a) { return -a; }
__device__ __forceinline__ float e_sum(f32x2 a)
{
    float lo, hi;
    f2_split(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ float e_sum(float a) { return a; }
// (lo, hi) -> (hi, lo)
__device__ __forceinline__ f32x2 e_swap(f32x2 a)
{
    float lo, hi;
    f2_split(a, lo, hi);
    return f2_make(hi, lo);
}
__device__ __forceinline__ float e_swap(float a) { return a; }

template <int V>
struct Elems {
    typedef f32x2 E;
    static constexpr int N = V / 2;
};
template <>
struct Elems<1> {
    typedef float E;
    static constexpr int N = 1;
};

template <class T, int V>
__device__ __forceinline__ void widen_e(const Vec<T, V> &v, typename Elems<V>::E (&x)[Elems<V>::N])
{
    float f[V];
    widen(v, f);
    if constexpr (V == 1) {
        x[0] = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) x[i] = f2_make(f[2 * i], f[2 * i + 1]);
    }
}

template <class T, int V>
__device__ __forceinline__ void narrow_e(const typename Elems<V>::E (&x)[Elems<V>::N], Vec<T, V> &v)
{
    float f[V];
    if constexpr (V == 1) {
        f[0] = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) f2_split(x[i], f[2 * i], f[2 * i + 1]);
    }
    narrow(f, v);
}

}  // namespace mhc
