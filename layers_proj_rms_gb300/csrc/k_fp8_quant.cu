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

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void cp_async16(uint32_t to, const void *from, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void sts128(uint32_t to, float x, float y, float z, float w)
{
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to), "f"(x), "f"(y), "f"(z), "f"(w)
                 : "memory");
}

constexpr int kRows = 4, kThreads = B / kRows * 16, kWarps = kThreads / 32;
// What a thread holds of the tile: 4 rows x 8 columns.
template <class T, int SRC>
struct Held {
    // 16-bit values as they came, or fp32
    static constexpr bool PACKED = SRC == kFp8Plain && sizeof(T) == 2;
    Vec<T, 8> w[PACKED ? kRows : 1];
    float v[PACKED ? 1 : kRows][8];

    __device__ __forceinline__ void zero(int i)
    {
        if constexpr (PACKED) {
            zero_vec<T, 8>(w[i]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
        }
    }
    // the 8 values of row i
    __device__ __forceinline__ void row(int i, float (&f)[8]) const
    {
        if constexpr (PACKED) {
            widen<T, 8>(w[i], f);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = v[i][k];
        }
    }
};

// The magnitude of a 16-bit value as that of the same fp32.
__device__ __forceinline__ uint32_t mag_bits(uint32_t h, const bf16 *) { return h << 16; }
__device__ __forceinline__ uint32_t mag_bits(uint32_t h, const fp16 *)
{
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}

// Rows of 8 values that a thread reads for one of its own: gate and up, the
// upstream gradient, gate and up.
template <int SRC>
constexpr int kSources = SRC == kFp8Plain ? 1 : SRC == kFp8Swiglu ? 2 : 3;
// Whether a block walks over tiles and brings the next one to shared memory while it
// works on this one.  16384 x 4096 in fp32 took 96 us so and 74 a block a tile, the
// activation in fp32 85 and 66, 73664 x 4096 in bf16 220 and 238, the activation in
// bf16 168 and 214, its gradient (32768 x 2048) 190 and 198.
template <class T>
constexpr bool kStaged = sizeof(T) == 2;

// c = a b
__device__ __forceinline__ void mul8(const float (&a)[8], const float (&b)[8], float (&c)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2)
        f2_split(f2_mul(f2_make(a[j], a[j + 1]), f2_make(b[j], b[j + 1])), c[j], c[j + 1]);
}

// c = du (p + a (1 - p))
__device__ __forceinline__ void gate_grad(const float (&du)[8], const float (&a)[8],
                                          const float (&p)[8], float (&c)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const f32x2 pp = f2_make(p[j], p[j + 1]);
        const f32x2 q = f2_fma(pp, f2_make(-1.f, -1.f), f2_make(1.f, 1.f));
        f2_split(f2_mul(f2_make(du[j], du[j + 1]), f2_fma(f2_make(a[j], a[j + 1]), q, pp)), c[j],
                 c[j + 1]);
    }
}

// The thread's row i from its 8 values of each source.
template <class T, int SRC>
__device__ __forceinline__ void hold(Held<T, SRC> &h, int i, const Vec<T, 8> &wg, const Vec<T, 8> &wu,
                                     const Vec<T, 8> &wd, bool up_part)
{
    if constexpr (Held<T, SRC>::PACKED) {
        h.w[i] = wg;
    } else if constexpr (SRC == kFp8Plain) {
        widen<T, 8>(wg, h.v[i]);
    } else {
        float gv[8], uv[8], dv[8], p[8], a[8];
        widen<T, 8>(wg, gv);
        if constexpr (SRC == kFp8SwigluGrad) widen<T, 8>(wd, dv);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = sigm(gv[j]);
        // silu(gate), then pairs: up's gradient d a, gate's d u (p + a (1 - p)), the product a u
#pragma unroll
        for (int j = 0; j < 8; ++j) gv[j] = silu_bound(gv[j]);
        mul8(gv, p, a);
        if (up_part) {
            mul8(dv, a, h.v[i]);
            return;
        }
        widen<T, 8>(wu, uv);
        if constexpr (SRC == kFp8Swiglu) {
            mul8(a, uv, h.v[i]);
        } else {
            mul8(dv, uv, uv);
            gate_grad(uv, a, p, h.v[i]);
        }
    }
}

// Row i of the gate's gradient, and of up's beside it.
template <class T>
__device__ __forceinline__ void hold_both(Held<T, kFp8SwigluGrad> &h, float (&up)[8], int i,
                                          const Vec<T, 8> &wg, const Vec<T, 8> &wu,
                                          const Vec<T, 8> &wd)
{
    float gv[8], uv[8], dv[8], p[8];
    widen<T, 8>(wg, gv);
    widen<T, 8>(wu, uv);
    widen<T, 8>(wd, dv);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = sigm(gv[j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) gv[j] = silu_bound(gv[j]);
    mul8(gv, p, gv);
    mul8(dv, gv, up);
    mul8(dv, uv, uv);
    gate_grad(uv, gv, p, h.v[i]);
}

// A thread's part of a tile: where it stands.
template <class T, int SRC>
struct Part {
    int cb, rows;  // the tile's block of columns; rows that are there
    int64_t rb, g, r0, c0;
    bool up_part;
    const T *x, *u, *d;  // the first row's 8 values of each source
    int64_t step, dstep;

    __device__ __forceinline__ Part(const Fp8QuantArgs &a, int halves, uint32_t t)
    {
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
        // the gate and the up tile of the same columns, which read the same rows, are neighbours
        const uint32_t all = t / a.ncb;  // tiles are below 2^31
        const int bx = int(t - all * a.ncb);
        g = all / a.nrb;
        rb = all - uint32_t(g) * a.nrb;
        cb = halves ? (bx >> 1) + (bx & 1) * halves : bx;
        r0 = rb * B + ty * kRows;
        c0 = int64_t(cb) * B + tx * 8;
        rows = c0 < a.C ? int(max(int64_t(0), min(int64_t(kRows), a.R - r0))) : 0;  // C a multiple of 8
        up_part = SRC == kFp8SwigluGrad && c0 >= a.F;
        step = SRC == kFp8Plain ? a.C : 2 * a.F;
        dstep = a.F;
        const int64_t j = up_part ? c0 - a.F : c0;
        x = static_cast<const T *>(a.x) + (g * a.R + r0) * step + j;
        u = x + a.F;
        d = SRC == kFp8SwigluGrad ? static_cast<const T *>(a.da) + r0 * dstep + j : x;
    }
};

// PAIRS: the gate's tile and the up tile of the same columns one after the other, from one
// reading and one sigm; up's values wait in the thread's staging places, in fp32.  Where the
// blocks of 128 end with the gate's columns (32768 x 2048: 134 us, one by one 169; along the
// rows alone 104 and 143); elsewhere up's blocks begin inside the gate's.
template <class T, int FMT, int SRC, bool TILES, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) k_fp8_quant(const Fp8QuantArgs a, int halves)
{
    typedef Held<T, SRC> H;
    // A row's magnitude stands where its quotient comes after, the columns' magnitudes by warps
    // where the bytes along them do: with three sources two blocks fill the SM's 228 KB, and
    // where nothing is staged the L1 is the larger (73 -> 70 us).  Elsewhere the barrier between
    // the tiles would cost 1%.
    constexpr bool ALIAS = !kStaged<T> || kSources<SRC> == 3;
    __shared__ __align__(16) uint8_t tile[B * B];
    __shared__ __align__(16) uint32_t col_own[ALIAS ? 1 : kWarps][B];
    uint32_t(*col_part)[B] = ALIAS ? reinterpret_cast<uint32_t(*)[B]>(tile) : col_own;
    static_assert(sizeof(uint32_t) * kWarps * B <= sizeof(tile), "columns' magnitudes");
    __shared__ __align__(16) float row_up[B], col_up[B];
    uint32_t *row_m = reinterpret_cast<uint32_t *>(row_up);
    extern __shared__ __align__(16) uint8_t next[];  // [source][row][half of it][thread] 16 bytes
    constexpr int PER = int(sizeof(T)) / 2;           // 16-byte pieces of 8 values
    constexpr bool STAGED = kStaged<T>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tx = tid & 15, ty = tid >> 4;
    const int64_t R = a.R, C = a.C;
    const int64_t nrb = a.nrb, ncb = a.ncb;
    const uint32_t tiles = uint32_t(a.G) * a.nrb * a.ncb;
    const uint32_t mine = uint32_t(__cvta_generic_to_shared(next)) + tid * 16;

    // a thread brings and reads its own 16 bytes only
    auto bring = [&](const Part<T, SRC> &q) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const uint32_t n = i < q.rows ? 16 : 0;
                const uint32_t at = mine + (i * PER + k) * kThreads * 16;
                constexpr int SLOT = kRows * PER * kThreads * 16;
                cp_async16(at, n ? q.x + i * q.step + k * 4 : a.x, n);
                if (SRC == kFp8Swiglu || (SRC == kFp8SwigluGrad && !q.up_part))
                    cp_async16(at + SLOT, n ? q.u + i * q.step + k * 4 : a.x, n);
                if constexpr (SRC == kFp8SwigluGrad)
                    cp_async16(at + 2 * SLOT, n ? q.d + i * q.dstep + k * 4 : a.x, n);
            }
    };
    auto take = [&](Vec<T, 8> &w, int source, int i) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint4 v = lds128(mine + ((source * kRows + i) * PER + k) * kThreads * 16);
            w.w[4 * k] = v.x;
            w.w[4 * k + 1] = v.y;
            w.w[4 * k + 2] = v.z;
            w.w[4 * k + 3] = v.w;
        }
    };

    pdl_wait();
    uint32_t t = PAIRS ? 2 * blockIdx.x : blockIdx.x, next_t;
    Part<T, SRC> coming(a, halves, t);
    if constexpr (STAGED) bring(coming);
    for (; t < tiles; t = next_t) {
    const bool second = PAIRS && t % 2;
    // (a block a tile where nothing is staged)
    next_t = !STAGED ? tiles : !PAIRS ? t + gridDim.x : second ? t - 1 + 2 * gridDim.x : t + 1;
    const Part<T, SRC> part = coming;
    const int cb = part.cb, rows = part.rows;
    const int64_t rb = part.rb, g = part.g, r0 = part.r0, c0 = part.c0;
    H held;
    if constexpr (STAGED) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        Vec<T, 8> wg, wu, wd;
        if constexpr (PAIRS) {
            const uint32_t lo = mine + i * kThreads * 16, hi = lo + kRows * kThreads * 16;
            if (second) {
                const uint4 v = lds128(lo), w = lds128(hi);
                const uint32_t b[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) held.v[i][j] = __uint_as_float(b[j]);
            } else {
                take(wg, 0, i);
                take(wu, 1, i);
                take(wd, 2, i);
                float up[8];
                hold_both(held, up, i, wg, wu, wd);
                sts128(lo, up[0], up[1], up[2], up[3]);
                sts128(hi, up[4], up[5], up[6], up[7]);
            }
        } else if constexpr (STAGED) {
            take(wg, 0, i);
            if (SRC == kFp8Swiglu || (SRC == kFp8SwigluGrad && !part.up_part)) take(wu, 1, i);
            if constexpr (SRC == kFp8SwigluGrad) take(wd, 2, i);
            hold<T, SRC>(held, i, wg, wu, wd, part.up_part);
        } else if (i < rows) {
            ld_vec<T, 8>(wg, part.x + i * part.step);
            if (SRC != kFp8Plain && !part.up_part) ld_vec<T, 8>(wu, part.u + i * part.step);
            if (SRC == kFp8SwigluGrad) ld_vec<T, 8>(wd, part.d + i * part.dstep);
            hold<T, SRC>(held, i, wg, wu, wd, part.up_part);
        } else {
            held.zero(i);
        }
    }
    if constexpr (STAGED)
        if (next_t < tiles) {
            coming = Part<T, SRC>(a, halves, next_t);
            if (!PAIRS || second) bring(coming);
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
        if (!a.q && !a.qt) continue;
    }

    // the largest magnitudes: of the thread's rows and columns, then of the lanes'
    uint32_t rm[kRows], cm[8];
    if constexpr (H::PACKED) {
        uint32_t c2[4] = {0, 0, 0, 0}, r2[kRows], last[4];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            uint32_t r4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                r4[k] = held.w[i].w[k] & 0x7fff7fffu;
                if (i % 2) c2[k] = __vimax3_u16x2(c2[k], last[k], r4[k]);
                last[k] = r4[k];
            }
            const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(r4[0], r4[1], r4[2]), r4[3], 0);
            r2[i] = max(m & 0xffffu, m >> 16);
        }
        if (a.q && !TILES) {  // two rows a word
            uint32_t p = r2[0] | r2[1] << 16, q = r2[2] | r2[3] << 16;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
                p = __vimax3_u16x2(p, __shfl_xor_sync(kFull, p, d), 0);
                q = __vimax3_u16x2(q, __shfl_xor_sync(kFull, q, d), 0);
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
                c2[k] = __vimax3_u16x2(c2[k], __shfl_xor_sync(kFull, c2[k], 16), 0);
                cm[2 * k] = mag_bits(c2[k] & 0xffffu, static_cast<const T *>(nullptr));
                cm[2 * k + 1] = mag_bits(c2[k] >> 16, static_cast<const T *>(nullptr));
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) cm[k] = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) rm[i] = 0;
#pragma unroll
        for (int i = 0; i < kRows; i += 2)
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const uint32_t x0 = f8_mag(held.v[i][k]), y0 = f8_mag(held.v[i][k + 1]);
                const uint32_t x1 = f8_mag(held.v[i + 1][k]), y1 = f8_mag(held.v[i + 1][k + 1]);
                rm[i] = __vimax3_u32(rm[i], x0, y0);
                rm[i + 1] = __vimax3_u32(rm[i + 1], x1, y1);
                cm[k] = __vimax3_u32(cm[k], x0, x1);
                cm[k + 1] = __vimax3_u32(cm[k + 1], y0, y1);
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
                const float ups[8] = {up[i], up[i], up[i], up[i], up[i], up[i], up[i], up[i]};
                float f[8];
                held.row(i, f);
                mul8(f, ups, f);
                *reinterpret_cast<uint2 *>(q + i * C) =
                    make_uint2(f8_cvt4<FMT>(f[0], f[1], f[2], f[3]), f8_cvt4<FMT>(f[4], f[5], f[6], f[7]));
            }
        }
    }
    if (!a.qt) {
        __syncthreads();
        continue;
    }
    float tc[kRows][8];  // the columns' values
    {
        float cu[8];
        if (TILES) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cu[k] = up_tile;
        } else {
            const float4 x = *reinterpret_cast<const float4 *>(&col_up[tx * 8]);
            const float4 y = *reinterpret_cast<const float4 *>(&col_up[tx * 8 + 4]);
            const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) cu[k] = z[k];
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            held.row(i, tc[i]);
            mul8(tc[i], cu, tc[i]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)  // column tx*8 + j, rows ty*4 .. ty*4 + 3
        *reinterpret_cast<uint32_t *>(tile + (tx * 8 + j) * B + (ty ^ (2 * tx)) * 4) =
            f8_cvt4<FMT>(tc[0][j], tc[1][j], tc[2][j], tc[3][j]);
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
    if (STAGED && ALIAS) __syncthreads();  // the next tile's magnitudes come where these bytes were
    }
}

template <class T, int FMT, int SRC, bool TILES, bool PAIRS>
cudaError_t run(const Fp8QuantArgs &a, const char *name, cudaStream_t s)
{
    auto *kernel = k_fp8_quant<T, FMT, SRC, TILES, PAIRS>;
    const int smem = kStaged<T> ? kSources<SRC> * kRows * int(sizeof(T)) * 8 * kThreads : 0;
    if (smem) {
        cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    const int halves = SRC == kFp8SwigluGrad && a.F % B == 0 ? int(a.F / B) : 0;
    // two blocks an SM that walk over the tiles, or a block a tile
    int64_t blocks = a.G * a.nrb * a.ncb / (PAIRS ? 2 : 1);
    if (kStaged<T>) blocks = std::min<int64_t>(blocks, 2 * num_sms());
    MHC_PROF(name, s);
    return launch_k(kernel, dim3(unsigned(blocks)), dim3(kThreads), smem, s,
                    a, halves);
}

template <class T, int FMT>
cudaError_t by_source(const Fp8QuantArgs &a, int source, cudaStream_t s)
{
    if (source == kFp8Swiglu) return run<T, FMT, kFp8Swiglu, false, false>(a, "k_fp8_swiglu_fwd", s);
    if (source == kFp8SwigluGrad) {
        if constexpr (kStaged<T>)
            if (a.F % B == 0)
                return run<T, FMT, kFp8SwigluGrad, false, true>(a, "k_fp8_swiglu_bwd", s);
        return run<T, FMT, kFp8SwigluGrad, false, false>(a, "k_fp8_swiglu_bwd", s);
    }
    return a.tiles ? run<T, FMT, kFp8Plain, true, false>(a, "k_fp8_quant", s)
                   : run<T, FMT, kFp8Plain, false, false>(a, "k_fp8_quant", s);
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
