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
// A block of 256 threads takes a tile of 128 x 128: a thread holds 8 rows x 8
// columns in registers, so a row's 128 values are in 16 lanes (maximum by four
// shuffles) and a column's in 16 threads of one place each (through shared
// memory).  The bytes along the rows leave from the registers, 128 a row; those
// along the columns go through shared memory, 8 a store, swizzled so that
// neither side has bank conflicts.
#include <algorithm>

#include "elem.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "launch.h"

namespace mhc {

namespace {

constexpr int B = kFp8Block;
// 8 values of row r, columns c .. c + 7
template <class T, int SRC>
__device__ __forceinline__ void values(const Fp8QuantArgs &a, const T *x, int64_t r, int64_t c,
                                       float (&v)[8])
{
    Vec<T, 8> w;
    if constexpr (SRC == kFp8Plain) {
        ld_vec<T, 8>(w, x + r * a.C + c);
        widen<T, 8>(w, v);
    } else {
        const int64_t F = a.F;
        const bool up_part = SRC == kFp8SwigluGrad && c >= F;
        const int64_t j = up_part ? c - F : c;
        float g[8];
        ld_vec<T, 8>(w, x + r * 2 * F + j);
        widen<T, 8>(w, g);
        if constexpr (SRC == kFp8Swiglu) {
            float u[8];
            ld_vec<T, 8>(w, x + r * 2 * F + F + j);
            widen<T, 8>(w, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = silu(g[i], sigm(g[i])) * u[i];
        } else {
            float d[8];
            ld_vec<T, 8>(w, static_cast<const T *>(a.da) + r * F + j);
            widen<T, 8>(w, d);
            if (up_part) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = d[i] * silu(g[i], sigm(g[i]));
            } else {
                float u[8];
                ld_vec<T, 8>(w, x + r * 2 * F + F + j);
                widen<T, 8>(w, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = sigm(g[i]);
                    v[i] = d[i] * u[i] * (p + silu(g[i], p) * (1.f - p));
                }
            }
        }
    }
}

template <class T, int FMT, int SRC, bool TILES>
__global__ void __launch_bounds__(256, 2) k_fp8_quant(const Fp8QuantArgs a, int halves)
{
    pdl_wait();
    __shared__ __align__(16) uint8_t tile[B * B];
    __shared__ uint32_t col_part[8][B];
    __shared__ float row_s[B], col_s[B], col_up[B];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tx = tid & 15, ty = tid >> 4;
    // the gate and the up tile of the same columns, which read the same rows, are neighbours
    const int bx = int(blockIdx.x % a.ncb);
    const int cb = halves ? (bx >> 1) + (bx & 1) * halves : bx;
    const int64_t rb = blockIdx.x / a.ncb, g = blockIdx.y;
    const int64_t r0 = rb * B + ty * 8, c0 = int64_t(cb) * B + tx * 8;
    const int64_t R = a.R, C = a.C;
    const int64_t nrb = (R + B - 1) / B, ncb = a.ncb;
    const T *x = static_cast<const T *>(a.x) + g * R * C;
    const bool in_c = c0 < C;  // C is a multiple of 8

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (in_c && r0 + i < R) {
            values<T, SRC>(a, x, r0 + i, c0, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
    }
    if (a.y && in_c) {
        T *y = static_cast<T *>(a.y) + g * R * C;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + i < R) {
                Vec<T, 8> w;
                narrow<T, 8>(v[i], w);
                st_vec<T, 8>(y + (r0 + i) * C + c0, w);
            }
    }

    float up_tile = 0.f;
    if (TILES) {
        uint32_t m = kLeastBits;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, f8_mag(v[i][j]));
        m = __reduce_max_sync(kFull, m);
        if (lane == 0) col_part[0][warp] = m;
        __syncthreads();
        m = col_part[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max(m, col_part[0][w]);
        up_tile = f8_up<FMT>(m);
        if (tid == 0) {
            const float s = f8_scale<FMT>(m);
            if (a.s) a.s[(g * ncb + cb) * nrb + rb] = s;
            if (a.st) a.st[(g * nrb + rb) * ncb + cb] = s;
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float up = up_tile;
            if (!TILES) {
                uint32_t m = kLeastBits;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, f8_mag(v[i][j]));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
                up = f8_up<FMT>(m);
                if (tx == 0) row_s[ty * 8 + i] = f8_scale<FMT>(m);
            }
            if (in_c && r0 + i < R) {
                uint2 w;
                w.x = f8_cvt4<FMT>(v[i][0] * up, v[i][1] * up, v[i][2] * up, v[i][3] * up);
                w.y = f8_cvt4<FMT>(v[i][4] * up, v[i][5] * up, v[i][6] * up, v[i][7] * up);
                *reinterpret_cast<uint2 *>(a.q + (g * R + r0 + i) * C + c0) = w;
            }
        }
    }
    if (a.qt && !TILES) {
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            m[j] = kLeastBits;
#pragma unroll
            for (int i = 0; i < 8; ++i) m[j] = max(m[j], f8_mag(v[i][j]));
            m[j] = max(m[j], __shfl_xor_sync(kFull, m[j], 16));
        }
        if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<uint4 *>(&col_part[warp][tx * 8 + j]) =
                    make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
        }
        __syncthreads();
        if (tid < B) {
            uint32_t k = col_part[0][tid];
#pragma unroll
            for (int w = 1; w < 8; ++w) k = max(k, col_part[w][tid]);
            col_s[tid] = f8_scale<FMT>(k);
            col_up[tid] = f8_up<FMT>(k);
        }
    }
    __syncthreads();
    if (!TILES) {
        if (a.q && tid < B && rb * B + tid < R)
            a.s[(g * ncb + cb) * R + rb * B + tid] = row_s[tid];
        if (a.qt && tid >= B && int64_t(cb) * B + tid - B < C)
            a.st[(g * nrb + rb) * C + int64_t(cb) * B + tid - B] = col_s[tid - B];
    }
    if (!a.qt) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float up = TILES ? up_tile : col_up[tx * 8 + j];
        uint2 w;
        w.x = f8_cvt4<FMT>(v[0][j] * up, v[1][j] * up, v[2][j] * up, v[3][j] * up);
        w.y = f8_cvt4<FMT>(v[4][j] * up, v[5][j] * up, v[6][j] * up, v[7][j] * up);
        // column tx*8 + j, rows ty*8 .. ty*8 + 7
        *reinterpret_cast<uint2 *>(tile + (tx * 8 + j) * B + (ty ^ tx) * 8) = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = k * 32 + (tid >> 3), m = tid & 7, sw = c >> 3;  // 16 rows from 16 m
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
        return launch_k(k_fp8_quant<T, FMT, kFp8Swiglu, false>, grid, dim3(256), 0, s, a, halves);
    }
    if (source == kFp8SwigluGrad) {
        MHC_PROF("k_fp8_swiglu_bwd", s);
        return launch_k(k_fp8_quant<T, FMT, kFp8SwigluGrad, false>, grid, dim3(256), 0, s, a,
                        halves);
    }
    MHC_PROF("k_fp8_quant", s);
    if (a.tiles)
        return launch_k(k_fp8_quant<T, FMT, kFp8Plain, true>, grid, dim3(256), 0, s, a, halves);
    return launch_k(k_fp8_quant<T, FMT, kFp8Plain, false>, grid, dim3(256), 0, s, a, halves);
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
