// Device helpers of the 8-bit floating-point operators: a block's scale, the
// conversions, the gated activation.
#pragma once

#include "common.cuh"

namespace mhc {

constexpr uint32_t kLeastBits = 0x0d800000u;  // 2^-100, the least amax of a block

// FMT 0: e4m3, 1: e5m2.  Round to nearest even, saturating; NaN stays NaN.
template <int FMT>
__device__ __forceinline__ uint32_t f8_cvt2(float lo, float hi)
{
    uint16_t r;
    if constexpr (FMT == 0)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t f8_cvt4(float a, float b, float c, float d)
{
    return f8_cvt2<FMT>(a, b) | f8_cvt2<FMT>(c, d) << 16;
}

template <int FMT>
__device__ __forceinline__ float f8_top()
{
    return FMT == 0 ? 448.f : 57344.f;
}
// A magnitude's bits: they are ordered as the magnitudes, inf and NaN above all numbers.
__device__ __forceinline__ uint32_t f8_mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Scale and multiplier of a block whose largest magnitude has these bits.
template <int FMT>
__device__ __forceinline__ float f8_scale(uint32_t amax)
{
    return amax < 0x7f800000u ? __fdiv_rn(__uint_as_float(amax), f8_top<FMT>())
                              : __uint_as_float(0x7fc00000u);
}
template <int FMT>
__device__ __forceinline__ float f8_up(uint32_t amax)
{
    return __fdiv_rn(f8_top<FMT>(), __uint_as_float(amax));
}

// Of two scales r and c and a sum d of products of 8-bit values (2^-32 <= |d| < 2^40, or 0):
// whether r c is no normal number though neither is 0.  d is then multiplied by the larger
// and that by the smaller: where |r c| > fp32's largest both are above 1, where it is below
// its least normal number the larger is below 2^23, so no step overflows or loses bits
// unless d r c does.
__device__ __forceinline__ bool f8_apart(float r, float c)
{
    return f8_mag(r * c) - 0x00800000u >= 0x7f000000u && r != 0.f && c != 0.f;
}
// d r c so
__device__ __forceinline__ float f8_scaled(float d, float r, float c)
{
    if (!f8_apart(r, c)) return d * (r * c);
    return fabsf(r) > fabsf(c) ? d * r * c : d * c * r;
}
// Whether d r may be no normal number: |r| < 2^-94 or > 2^88.
__device__ __forceinline__ bool f8_far(float r)
{
    return f8_mag(r) - 0x10800000u > 0x5b000000u && r != 0.f;
}

// 1 / (1 + exp(-g)): 0 where exp(-g) is inf.  An exp(-g) that is no normal number may be
// zero beside 1.  Two approximations of a unit or two of fp32 each, and the rounding of ex2's
// argument, which is 1.2 |g| 2^-24 of exp(-g): silu(g) is off by 1.1 2^-24 (rms; 5.6 at
// most) for gates within 4, by 10 2^-24 at most to -10, 60 2^-24 at -60, where silu is 5e-25.
// Over normal gates the gradient is off by 5.6e-8 (rms), with expf and a divide by 5.8e-8.
// (Carrying the rounding takes four instructions more, where the gradient is bound by them.)
__device__ __forceinline__ float sigm(float g)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    return rcp_approx(1.f + e);
}
// g p for p = sigm(g), 0 at -inf; NaN comes with p
__device__ __forceinline__ float silu_bound(float g) { return fmaxf(g, -3.4028234e38f); }
__device__ __forceinline__ float silu(float g, float p) { return silu_bound(g) * p; }

}  // namespace mhc
