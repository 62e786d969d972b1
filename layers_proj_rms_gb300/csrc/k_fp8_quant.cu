// Quantisation to 8-bit floating point (e4m3 or e5m2) with a scale for each
// block of 128 elements along the rows, along the columns (stored transposed),
// both, or for each tile of 128 x 128; of the values themselves, of
// silu(gate) up, or of that product's gradient, formed in fp32 on the way:
//
//   amax = max(largest |v| of the block, 2^-100), scale = amax / top,
//   q = round(v * (top / amax)),   top = 448 (e4m3), 57344 (e5m2),
//
// both quotients as IEEE divides.  A block that holds an infinity or a NaN has
// the scale NaN: the largest magnitude is found on the bit patterns, where a
// NaN is above all numbers.  The least amax keeps 1/amax finite and gives a
// block of zeros a scale.
//
// A block of 512 threads takes a tile of 128 x 128: a thread holds 4 rows x 8
// columns in registers, so a row's 128 values are in 16 lanes and a column's in 32
// threads of one place each.  Three steps, a barrier after each: the largest
// magnitudes of rows (shuffles) and columns (shared memory); the quotients, one
// thread a row or column; the bytes.  Those along the rows leave from the
// registers, 128 a row; those along the columns go through shared memory, 4 a
// store, swizzled so that neither side has bank conflicts.  16-bit values stay as
// they came: their magnitudes are compared as pairs of 16-bit numbers.
#include <algorithm>

#include "elem.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "launch.h"

namespace mhc {

namespace {

constexpr int B = kFp8Block;
constexpr int kRows = 4, kThreads = B / kRows * 16, kWarps = kThreads / 32;
// What a thread holds of the tile: 4 rows x 8 columns.
template <class T, int SRC>
struct Held {
    // 16-bit values as they came, or fp32
    static constexpr bool PACKED = SRC == kFp8Plain && sizeof(T) == 2;
    Vec<T, 8> w[PACKED ? kRows : 1];
    float v[PACKED ? 1 : kRows][8];

    // the 8 values of row i as pairs
    __device__ __forceinline__ void row(int i, f32x2 (&p)[4]) const
    {
        if constexpr (PACKED) {
            float f[8];
            widen<T, 8>(w[i], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = f2_make(f[2 * k], f[2 * k + 1]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = f2_make(v[i][2 * k], v[i][2 * k + 1]);
        }
    }
};

// The magnitude of a 16-bit value as that of the same fp32.
__device__ __forceinline__ uint32_t mag_bits(uint32_t h, const bf16 *) { return h << 16; }
__device__ __forceinline__ uint32_t mag_bits(uint32_t h, const fp16 *)
{
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

// 8 values of a row: x points at them (of gate, where there are two halves), u at
// those of up, d at the upstream gradient's.
template <class T, int SRC>
__device__ __forceinline__ void values(Held<T, SRC> &h, int i, const T *x, const T *u, const T *d,
                                       bool up_part)
{
    if constexpr (Held<T, SRC>::PACKED) {
        ld_vec<T, 8>(h.w[i], x);
    } else if constexpr (SRC == kFp8Plain) {
        Vec<T, 8> w;
        ld_vec<T, 8>(w, x);
        widen<T, 8>(w, h.v[i]);
    } else {
        Vec<T, 8> wg, wu, wd;
        ld_vec<T, 8>(wg, x);
        if (!up_part) ld_vec<T, 8>(wu, u);
        if constexpr (SRC == kFp8SwigluGrad) ld_vec<T, 8>(wd, d);
        float gv[8], uv[8], dv[8];
        widen<T, 8>(wg, gv);
        if constexpr (SRC == kFp8SwigluGrad) widen<T, 8>(wd, dv);
        if (up_part) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h.v[i][j] = dv[j] * silu(gv[j], sigm(gv[j]));
            return;
        }
        widen<T, 8>(wu, uv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = sigm(gv[j]), a = silu(gv[j], p);
            h.v[i][j] = SRC == kFp8Swiglu ? a * uv[j] : dv[j] * uv[j] * (p + a * (1.f - p));
        }
    }
}

template <class T, int FMT, int SRC, bool TILES>
__global__ void __launch_bounds__(kThreads, 2) k_fp8_quant(const Fp8QuantArgs a, int halves)
{
    typedef Held<T, SRC> H;
    __shared__ __align__(16) uint8_t tile[B * B];
    __shared__ __align__(16) uint32_t col_part[kWarps][B];
    __shared__ __align__(16) uint32_t row_m[B];
    __shared__ __align__(16) float row_up[B], col_up[B];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tx = tid & 15, ty = tid >> 4;
    // the gate and the up tile of the same columns, which read the same rows, are neighbours
    const int bx = int(blockIdx.x % a.ncb);
    const int cb = halves ? (bx >> 1) + (bx & 1) * halves : bx;
    const int64_t rb = blockIdx.x / a.ncb, g = blockIdx.y;
    const int64_t r0 = rb * B + ty * kRows, c0 = int64_t(cb) * B + tx * 8;
    const int64_t R = a.R, C = a.C;
    const int64_t nrb = (R + B - 1) / B, ncb = a.ncb;
    const bool in_c = c0 < C;  // C is a multiple of 8
    const int rows = in_c ? int(min(int64_t(kRows), R - r0)) : 0;  // of this thread's

    pdl_wait();
    H held;
    {
        const bool up_part = SRC == kFp8SwigluGrad && c0 >= a.F;
        const int64_t step = SRC == kFp8Plain ? C : 2 * a.F, j = up_part ? c0 - a.F : c0;
        const T *x = static_cast<const T *>(a.x) + (g * R + r0) * step + j;
        const T *d = SRC == kFp8SwigluGrad ? static_cast<const T *>(a.da) + r0 * a.F + j : nullptr;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i < rows) {
                values<T, SRC>(held, i, x + i * step, x + i * step + a.F, d + i * a.F, up_part);
            } else if constexpr (H::PACKED) {
                zero_vec<T, 8>(held.w[i]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) held.v[i][k] = 0.f;
            }
        }
    }
    if (a.y) {
        T *y = static_cast<T *>(a.y) + (g * R + r0) * C + c0;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (i < rows) {
                if constexpr (!H::PACKED) {
                    Vec<T, 8> w;
                    narrow<T, 8>(held.v[i], w);
                    st_vec<T, 8>(y + i * C, w);
                }
            }
        if (!a.q && !a.qt) return;
    }

    // the largest magnitudes: of the thread's rows and columns, then of the lanes'
    uint32_t rm[kRows], cm[8];
    if constexpr (H::PACKED) {
        uint32_t c2[4] = {0, 0, 0, 0}, r2[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t x = held.w[i].w[k] & 0x7fff7fffu;
                m = __vmaxu2(m, x);
                c2[k] = __vmaxu2(c2[k], x);
            }
            r2[i] = max(m & 0xffffu, m >> 16);
        }
        if (a.q && !TILES) {  // two rows a word
            uint32_t p = r2[0] | r2[1] << 16, q = r2[2] | r2[3] << 16;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
                p = __vmaxu2(p, __shfl_xor_sync(kFull, p, d));
                q = __vmaxu2(q, __shfl_xor_sync(kFull, q, d));
            }
            r2[0] = p & 0xffffu;
            r2[1] = p >> 16;
            r2[2] = q & 0xffffu;
            r2[3] = q >> 16;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) rm[i] = mag_bits(r2[i], static_cast<const T *>(nullptr));
        if (a.qt && !TILES) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c2[k] = __vmaxu2(c2[k], __shfl_xor_sync(kFull, c2[k], 16));
                cm[2 * k] = mag_bits(c2[k] & 0xffffu, static_cast<const T *>(nullptr));
                cm[2 * k + 1] = mag_bits(c2[k] >> 16, static_cast<const T *>(nullptr));
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) cm[k] = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            rm[i] = 0;
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const uint32_t x = f8_mag(held.v[i][k]), y = f8_mag(held.v[i][k + 1]);
                rm[i] = __vimax3_u32(rm[i], x, y);
                cm[k] = max(cm[k], x);
                cm[k + 1] = max(cm[k + 1], y);
            }
        }
        if (a.q && !TILES) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) rm[i] = max(rm[i], __shfl_xor_sync(kFull, rm[i], d));
        }
        if (a.qt && !TILES) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cm[k] = max(cm[k], __shfl_xor_sync(kFull, cm[k], 16));
        }
    }
    float up_tile = 0.f;
    if constexpr (TILES) {
        const uint32_t m = __reduce_max_sync(kFull, max(max(rm[0], rm[1]), max(rm[2], rm[3])));
        if (lane == 0) row_m[warp] = m;
        __syncthreads();
        uint32_t k = kLeastBits;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) k = max(k, row_m[w]);
        up_tile = f8_up<FMT>(k);
        if (tid == 0) {
            const float s = f8_scale<FMT>(k);
            if (a.s) a.s[(g * ncb + cb) * nrb + rb] = s;
            if (a.st) a.st[(g * nrb + rb) * ncb + cb] = s;
        }
    } else {
        if (a.q && tx == 0)
            *reinterpret_cast<uint4 *>(&row_m[ty * kRows]) = make_uint4(rm[0], rm[1], rm[2], rm[3]);
        if (a.qt && lane < 16) {
            *reinterpret_cast<uint4 *>(&col_part[warp][tx * 8]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
            *reinterpret_cast<uint4 *>(&col_part[warp][tx * 8 + 4]) =
                make_uint4(cm[4], cm[5], cm[6], cm[7]);
        }
        __syncthreads();
        if (tid < B) {
            if (a.q) {
                const uint32_t k = max(kLeastBits, row_m[tid]);
                row_up[tid] = f8_up<FMT>(k);
                if (rb * B + tid < R) a.s[(g * ncb + cb) * R + rb * B + tid] = f8_scale<FMT>(k);
            }
        } else if (tid < 2 * B && a.qt) {
            const int c = tid - B;
            uint32_t k = kLeastBits;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) k = max(k, col_part[w][c]);
            col_up[c] = f8_up<FMT>(k);
            if (int64_t(cb) * B + c < C) a.st[(g * nrb + rb) * C + int64_t(cb) * B + c] = f8_scale<FMT>(k);
        }
        __syncthreads();
    }

    if (a.q) {
        float4 ru = make_float4(up_tile, up_tile, up_tile, up_tile);
        if (!TILES) ru = *reinterpret_cast<const float4 *>(&row_up[ty * kRows]);
        const float up[kRows] = {ru.x, ru.y, ru.z, ru.w};
        uint8_t *q = a.q + (g * R + r0) * C + c0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i < rows) {
                f32x2 p[4];
                held.row(i, p);
                float f[8];
                const f32x2 m = f2_make(up[i], up[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) f2_split(f2_mul(p[k], m), f[2 * k], f[2 * k + 1]);
                *reinterpret_cast<uint2 *>(q + i * C) =
                    make_uint2(f8_cvt4<FMT>(f[0], f[1], f[2], f[3]), f8_cvt4<FMT>(f[4], f[5], f[6], f[7]));
            }
        }
    }
    if (!a.qt) return;
    float t[kRows][8];  // the columns' values
    {
        f32x2 cu[4];
        if (TILES) {
#pragma unroll
            for (int k = 0; k < 4; ++k) cu[k] = f2_make(up_tile, up_tile);
        } else {
            const float4 x = *reinterpret_cast<const float4 *>(&col_up[tx * 8]);
            const float4 y = *reinterpret_cast<const float4 *>(&col_up[tx * 8 + 4]);
            cu[0] = f2_make(x.x, x.y);
            cu[1] = f2_make(x.z, x.w);
            cu[2] = f2_make(y.x, y.y);
            cu[3] = f2_make(y.z, y.w);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            f32x2 p[4];
            held.row(i, p);
#pragma unroll
            for (int k = 0; k < 4; ++k) f2_split(f2_mul(p[k], cu[k]), t[i][2 * k], t[i][2 * k + 1]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)  // column tx*8 + j, rows ty*4 .. ty*4 + 3
        *reinterpret_cast<uint32_t *>(tile + (tx * 8 + j) * B + (ty ^ (2 * tx)) * 4) =
            f8_cvt4<FMT>(t[0][j], t[1][j], t[2][j], t[3][j]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < B * 8 / kThreads; ++k) {
        const int c = k * (kThreads / 8) + (tid >> 3), m = tid & 7, sw = c >> 3;  // 16 rows from 16 m
        uint4 w = *reinterpret_cast<const uint4 *>(tile + c * B + (m ^ (sw >> 1)) * 16);
        if (sw & 1) w = make_uint4(w.z, w.w, w.x, w.y);
        const int64_t col = int64_t(cb) * B + c, row = rb * B + m * 16;
        if (col < C && row < R)  // R is a multiple of 16
            *reinterpret_cast<uint4 *>(a.qt + (g * C + col) * R + row) = w;
    }
}

template <class T, int FMT>
cudaError_t by_source(const Fp8QuantArgs &a, int source, cudaStream_t s)
{
    const dim3 grid{unsigned(a.ncb * fp8_blocks(a.R)), unsigned(a.G)};
    const int halves = source == kFp8SwigluGrad && a.F % B == 0 ? int(a.F / B) : 0;
    if (source == kFp8Swiglu) {
        MHC_PROF("k_fp8_swiglu_fwd", s);
        return launch_k(k_fp8_quant<T, FMT, kFp8Swiglu, false>, grid, dim3(kThreads), 0, s, a, halves);
    }
    if (source == kFp8SwigluGrad) {
        MHC_PROF("k_fp8_swiglu_bwd", s);
        return launch_k(k_fp8_quant<T, FMT, kFp8SwigluGrad, false>, grid, dim3(kThreads), 0, s, a,
                        halves);
    }
    MHC_PROF("k_fp8_quant", s);
    if (a.tiles)
        return launch_k(k_fp8_quant<T, FMT, kFp8Plain, true>, grid, dim3(kThreads), 0, s, a, halves);
    return launch_k(k_fp8_quant<T, FMT, kFp8Plain, false>, grid, dim3(kThreads), 0, s, a, halves);
}

template <class T>
cudaError_t by_format(const Fp8QuantArgs &a, int source, int format, cudaStream_t s)
{
    return format == 0 ? by_source<T, 0>(a, source, s) : by_source<T, 1>(a, source, s);
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8QuantArgs &a, int source, int dtype, int format,
                             cudaStream_t s)
{
    if (dtype == 0) return by_format<bf16>(a, source, format, s);
    if (dtype == 1) return by_format<fp16>(a, source, format, s);
    return by_format<float>(a, source, format, s);
}

}  // namespace mhc
