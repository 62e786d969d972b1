// Token rows to their experts' segments and back.
//
//   dispatch:      xs[r] = x[slot_of[r] / k], padding rows 0
//   combine:       f[t] = sum_j w[t][j] ys[row_of[t][j]]     (w absent: 1; the
//                  gradient of dispatch), dropped slots (-1) add nothing
//   combine bwd:   dys[row] = w[t][j] df[t], padding rows 0;
//                  dw[t][j] = sum_c df[t][c] ys[row][c], dropped slots 0
//
// All three are bound by HBM (16384 x 4096, k = 4: dispatch 112 us, 97% of the
// measured copy bandwidth, combine backward 193 us, 97%; 8192 x 7168, k = 8,
// combine backward 365 us, 100%, once four blocks fit an SM: with two, 387).
// They walk over tokens, not over sorted rows: a token's row is read once and
// its k rows are whole, contiguous 2C-byte rows wherever they are, so every
// byte crosses HBM once.  Padding rows have no token; each block clears those
// of its share of the sorted rows.
// Sums over j are in ascending j and sums over c in an order fixed by C
// alone, so a token's results do not depend on T or on its place.
#include "elem.cuh"
#include "launch.h"
#include "moe.h"

namespace mhc {

constexpr int kFaultRow = 203;  // a row of the plan outside [-1, R)

namespace {

constexpr int kRowThreads = 256;

// The row of a slot: -1 if dropped, or if the plan is not one (a fault).
__device__ __forceinline__ int64_t plan_row(const int32_t *row_of, int64_t slot, int64_t R,
                                            int *fault)
{
    const int64_t r = __ldg(row_of + slot);
    if (r >= -1 && r < R) return r;
    report_fault(fault, kFaultRow);
    return -1;
}

// Zeroes the padding rows among the block's share of the sorted rows.
__device__ __forceinline__ void clear_padding(const int32_t *slot_of, int64_t R, int64_t chunks,
                                              uint4 *out)
{
    const int64_t per = (R + gridDim.x - 1) / gridDim.x;
    const int64_t r0 = per * blockIdx.x, r1 = r0 + per < R ? r0 + per : R;
    for (int64_t r = r0; r < r1; ++r)
        if (__ldg(slot_of + r) < 0)
            for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x)
                st_stream(out + r * chunks + q, make_uint4(0, 0, 0, 0));
}

// chunks: 16-byte pieces of a row
__global__ void __launch_bounds__(kRowThreads)
    k_moe_dispatch(const uint4 *__restrict__ x, const int32_t *__restrict__ row_of,
                   const int32_t *__restrict__ slot_of, int64_t T, int k, int64_t R,
                   int64_t chunks, uint4 *__restrict__ xs, int *fault)
{
    pdl_wait();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x)
        for (int64_t q = threadIdx.x; q < chunks; q += blockDim.x) {
            const uint4 v = ld_stream(x + t * chunks + q);
            for (int j = 0; j < k; ++j) {
                const int64_t r = plan_row(row_of, t * k + j, R, fault);
                if (r >= 0) st_stream(xs + r * chunks + q, v);
            }
        }
    clear_padding(slot_of, R, chunks, xs);
}

// sum_j w[t][j] ys[row][chunk q] for one token's chunk of V elements; KM rows
// at a time are on their way.
template <class T, int KM>
__device__ __forceinline__ void combine_chunk(const T *ys, const float *w, const int32_t *row_of,
                                              int64_t t, int64_t q, int k, int64_t R,
                                              int64_t chunks, T *f, int *fault)
{
    constexpr int V = 16 / int(sizeof(T));
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    for (int j0 = 0; j0 < k; j0 += KM) {
        Vec<T, V> v[KM];
        float wj[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            wj[j] = 0.f;
            zero_vec(v[j]);
            if (j0 + j < k) {
                const int64_t slot = t * k + j0 + j, r = plan_row(row_of, slot, R, fault);
                if (r >= 0) {
                    wj[j] = w ? __ldg(w + slot) : 1.f;
                    ld_vec(v[j], ys + (r * chunks + q) * V);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            float y[V];
            widen(v[j], y);
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(wj[j], y[e], acc[e]);
        }
    }
    Vec<T, V> o;
    narrow(acc, o);
    st_vec(f + (t * chunks + q) * V, o);
}

// BLOCK: a block on one token at a time (its rows are looked up once for all
// chunks); else one chunk of one token per thread (for few tokens, short rows).
template <class T, bool BLOCK, int KM>
__global__ void __launch_bounds__(kRowThreads)
    k_moe_combine(const T *__restrict__ ys, const float *__restrict__ w,
                  const int32_t *__restrict__ row_of, int64_t tokens, int k, int64_t R,
                  int64_t chunks, T *__restrict__ f, int *fault)
{
    pdl_wait();
    if constexpr (BLOCK) {
        for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x)
            for (int64_t q = threadIdx.x; q < chunks; q += kRowThreads)
                combine_chunk<T, KM>(ys, w, row_of, t, q, k, R, chunks, f, fault);
    } else {
        const int64_t i = int64_t(blockIdx.x) * kRowThreads + threadIdx.x;
        if (i >= tokens * chunks) return;
        const int64_t t = i / chunks;
        combine_chunk<T, KM>(ys, w, row_of, t, i - t * chunks, k, R, chunks, f, fault);
    }
}

// TPT threads of a block work on one token (32: a warp on its own, for rows of
// up to 192 chunks; else the whole block); the sums of dw of KM slots stay in
// registers over the row.
template <class T, int TPT, int KM>
__global__ void __launch_bounds__(kRowThreads, TPT == 32 && KM == 8 ? 3 : 4)
    k_moe_combine_bwd(const T *__restrict__ df, const T *__restrict__ ys,
                      const float *__restrict__ w, const int32_t *__restrict__ row_of,
                      const int32_t *__restrict__ slot_of, int64_t tokens, int k, int64_t R,
                      int64_t chunks, T *__restrict__ dys, float *__restrict__ dw, int *fault)
{
    constexpr int V = 16 / int(sizeof(T)), PER = kRowThreads / TPT;
    __shared__ float red[KM][kRowThreads / 32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = threadIdx.x % TPT;
    const int64_t step = int64_t(gridDim.x) * PER;
    for (int64_t t = int64_t(blockIdx.x) * PER + threadIdx.x / TPT; t < tokens; t += step)
        for (int j0 = 0; j0 < k; j0 += KM) {
            int64_t row[KM];
            float wj[KM], acc[KM];
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                acc[j] = wj[j] = 0.f;
                row[j] = -1;
                if (j0 + j < k) {
                    const int64_t slot = t * k + j0 + j;
                    row[j] = plan_row(row_of, slot, R, fault);
                    if (row[j] >= 0) wj[j] = w ? __ldg(w + slot) : 1.f;
                }
            }
            for (int64_t q = me; q < chunks; q += TPT) {
                Vec<T, V> dv, yv[KM];
                ld_vec(dv, df + (t * chunks + q) * V);
                if (dw)
#pragma unroll
                    for (int j = 0; j < KM; ++j)
                        if (row[j] >= 0) ld_vec(yv[j], ys + (row[j] * chunks + q) * V);
                float d[V];
                widen(dv, d);
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (row[j] >= 0) {
                        float o[V];
                        if (dw) {
                            float y[V];
                            widen(yv[j], y);
#pragma unroll
                            for (int e = 0; e < V; ++e) acc[j] = fmaf(d[e], y[e], acc[j]);
                        }
#pragma unroll
                        for (int e = 0; e < V; ++e) o[e] = wj[j] * d[e];
                        Vec<T, V> ov;
                        narrow(o, ov);
                        st_vec(dys + (row[j] * chunks + q) * V, ov);
                    }
            }
            if (!dw) continue;
            if constexpr (TPT == 32) {
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    const float s = warp_sum(acc[j]);
                    if (lane == j && j0 + j < k) dw[t * k + j0 + j] = s;
                }
            } else {
#pragma unroll
                for (int j = 0; j < KM; ++j) {
                    const float s = warp_sum(acc[j]);
                    if (lane == 0) red[j][warp] = s;
                }
                __syncthreads();
                if (threadIdx.x < KM && j0 + int(threadIdx.x) < k) {
                    float s = 0.f;
                    for (int i = 0; i < TPT / 32; ++i) s += red[threadIdx.x][i];
                    dw[t * k + j0 + threadIdx.x] = s;
                }
                __syncthreads();
            }
        }
    clear_padding(slot_of, R, chunks, reinterpret_cast<uint4 *>(dys));
}

// A block per token, and no more than eight sorted rows to look over for each.
unsigned row_blocks(int64_t T, int64_t R)
{
    const int64_t n = T > (R + 7) / 8 ? T : (R + 7) / 8, cap = int64_t(kSplitSms) * 64;
    return unsigned(n < cap ? n : cap);
}

int row_threads(int64_t chunks)
{
    const int64_t t = (chunks + 31) / 32 * 32;
    return int(t < kRowThreads ? t : kRowThreads);
}

template <class T>
cudaError_t combine_of(const void *ys, const float *w, const int32_t *row_of, int64_t tokens,
                       int k, int64_t R, int64_t C, void *f, int *fault, cudaStream_t s)
{
    const int64_t chunks = C * int64_t(sizeof(T)) / 16;
    // 1001 tokens of 1792 chunks, k = 6: a block a token 29.6 us, a chunk a thread
    // 31.5; 16384 of 512, k = 4: 105 and 116; 12598 of 305, k = 7: 83 and 79.  A
    // chunk's sum is the same either way.
    const bool block = chunks >= 512 && tokens >= kSplitSms * 4;
    const int64_t blocks = block ? row_blocks(tokens, 0)
                                 : (tokens * chunks + kRowThreads - 1) / kRowThreads;
    MHC_PROF("k_moe_combine", s);
    auto kernel = k <= 4 ? (block ? k_moe_combine<T, true, 4> : k_moe_combine<T, false, 4>)
                         : (block ? k_moe_combine<T, true, 8> : k_moe_combine<T, false, 8>);
    return launch_k(kernel, dim3(unsigned(blocks)), dim3(kRowThreads), 0, s, static_cast<const T *>(ys), w,
                    row_of, tokens, k, R, chunks, static_cast<T *>(f), fault);
}

template <class T>
cudaError_t combine_bwd_of(const void *df, const void *ys, const float *w, const int32_t *row_of,
                           const int32_t *slot_of, int64_t tokens, int k, int64_t R, int64_t C,
                           void *dys, float *dw, int *fault, cudaStream_t s)
{
    const int64_t chunks = C * int64_t(sizeof(T)) / 16;
    // a block on one token, or a warp: rows of 166 chunks, k = 5, 30.5 and 24.0 us
    // (3311 tokens); of 256 chunks, k = 6, 44.9 and 47.4 (4096 tokens).  The rule
    // looks at C alone, as the order of dw's sums goes by it.
    const bool one = chunks > 192;
    const int64_t per = one ? 1 : kRowThreads / 32, need = (tokens + per - 1) / per;
    MHC_PROF("k_moe_combine_bwd", s);
    auto kernel = k <= 4 ? (one ? k_moe_combine_bwd<T, kRowThreads, 4> : k_moe_combine_bwd<T, 32, 4>)
                         : (one ? k_moe_combine_bwd<T, kRowThreads, 8> : k_moe_combine_bwd<T, 32, 8>);
    return launch_k(kernel, dim3(row_blocks(need, R)), dim3(kRowThreads), 0, s, static_cast<const T *>(df),
                    static_cast<const T *>(ys), w, row_of, slot_of, tokens, k, R, chunks,
                    static_cast<T *>(dys), dw, fault);
}

}  // namespace

cudaError_t launch_moe_dispatch_fwd(const void *x, int dtype, const int32_t *row_of,
                                    const int32_t *slot_of, int64_t T, int k, int64_t R,
                                    int64_t C, void *xs, int *fault, cudaStream_t s)
{
    const int64_t chunks = C * (dtype == 2 ? 4 : 2) / 16;
    MHC_PROF("k_moe_dispatch", s);
    return launch_k(k_moe_dispatch, dim3(row_blocks(T, R)), dim3(row_threads(chunks)), 0, s,
                    static_cast<const uint4 *>(x), row_of, slot_of, T, k, R, chunks,
                    static_cast<uint4 *>(xs), fault);
}

cudaError_t launch_moe_combine_fwd(const void *ys, int dtype, const float *w,
                                   const int32_t *row_of, int64_t T, int k, int64_t R, int64_t C,
                                   void *f, int *fault, cudaStream_t s)
{
    return dtype == 0   ? combine_of<bf16>(ys, w, row_of, T, k, R, C, f, fault, s)
           : dtype == 1 ? combine_of<fp16>(ys, w, row_of, T, k, R, C, f, fault, s)
                        : combine_of<float>(ys, w, row_of, T, k, R, C, f, fault, s);
}

cudaError_t launch_moe_combine_bwd(const void *df, const void *ys, int dtype, const float *w,
                                   const int32_t *row_of, const int32_t *slot_of, int64_t T,
                                   int k, int64_t R, int64_t C, void *dys, float *dw, int *fault,
                                   cudaStream_t s)
{
    return dtype == 0 ? combine_bwd_of<bf16>(df, ys, w, row_of, slot_of, T, k, R, C, dys, dw, fault, s)
           : dtype == 1
               ? combine_bwd_of<fp16>(df, ys, w, row_of, slot_of, T, k, R, C, dys, dw, fault, s)
               : combine_bwd_of<float>(df, ys, w, row_of, slot_of, T, k, R, C, dys, dw, fault, s);
}

}  // namespace mhc
