// Top-k router: ids [T, k] of the k largest logits of each token (ties to the
// lowest index, NaN above everything) and their weights, and the gradient.
//
//   softmax:          w_j = scale p_j, p = softmax over all E logits
//   softmax, renorm:  w_j = scale softmax over the k chosen logits
//   sigmoid:          w_j = scale s(l_j), s the logistic function
//   sigmoid, renorm:  w_j = scale s_j / sum of the chosen s, formed as the
//                     softmax of log s over the chosen (no underflow)
//   a row whose chosen (softmax: whose all) logits are -inf has weights 0.
//   backward, a_j = scale dw_j:
//     softmax:          dl_e = p_e (sum_{j: id_j = e} a_j - sum_j a_j p_j)
//     softmax, renorm:  dl_j = v_j (a_j - sum_i a_i v_i), v = w / scale
//     sigmoid:          dl_j = a_j s_j (1 - s_j)
//     sigmoid, renorm:  dl_j = v_j (1 - s_j) (a_j - sum_i a_i v_i)
//   dlogits of the experts not chosen are 0 but for the plain softmax.  A slot
//   dropped after the choice (id -1) has a_j = 0; renormalised, its score stays
//   in the weights' sum, as in the forward, so a row with such a slot is chosen
//   again (the choice is exact) and its experts' dl_j have their share of it.
//
// One warp per token; lane l holds logits l, l + 32, ...  The choice compares
// logits as stored (monotone integer keys), never computed scores, so it is
// exact.  Chosen slot j lives in lane j (k <= 32).  What bounds this form: the
// warp's instructions (each round is one warp maximum and one step of a sorted
// list; 16384 x 256 fp32, k = 8: 420 a token, 8.3 us).  The backward of the same,
// renormalised, takes 8.7 us, and 12.1 with one slot in 64 dropped (12% of the
// rows are chosen again).
#include "elem.cuh"
#include "launch.h"
#include "moe.h"

namespace mhc {

// backward: an id outside [-1, E), or one that the forward did not choose in a
// row whose choice has to be found again
constexpr int kFaultChoice = 204;

namespace {

// Warps of a block, and blocks per SM that the registers leave room for:
// 16384 x 256 fp32, k = 8: 4, 12 take 8.3 us; 4, any 8.4; 8, 8 8.5; 16, any 10.6.
constexpr int kRouterWarps = 4, kRouterPerSm = 12;

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, m));
    return v;
}

__device__ __forceinline__ float widen1(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen1(fp16 v) { return __half2float(v); }
__device__ __forceinline__ float widen1(float v) { return v; }
__device__ __forceinline__ void narrow1(float f, bf16 &o) { o = __float2bfloat16_rn(f); }
__device__ __forceinline__ void narrow1(float f, fp16 &o) { o = __float2half_rn(f); }
__device__ __forceinline__ void narrow1(float f, float &o) { o = f; }

// Ascending integer key of a float; > 0; equal for -0 and 0; NaN the largest
// (the sum with 0 turns -0 into 0 and every NaN into the canonical 0x7fffffff).
__device__ __forceinline__ unsigned key_of(float f)
{
    const unsigned u = __float_as_uint(__fadd_rn(f, 0.f));
    return u ^ (unsigned(int(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float logistic(float l) { return 1.f / (1.f + expf(-l)); }
__device__ __forceinline__ float log_logistic(float l)
{
    return fminf(l, 0.f) - log1pf(expf(-fabsf(l)));
}

// Softmax of one value per lane over the lanes that are `on`; -inf everywhere
// (or no lane on) gives 0.
__device__ __forceinline__ float lane_softmax(float v, bool on)
{
    const float m = warp_max(on ? v : -INFINITY);  // a NaN is passed over here, not below
    const float p = on && (m != -INFINITY || v != v) ? expf(v - m) : 0.f;
    const float s = warp_sum(p);
    return s == 0.f ? 0.f : p / s;
}

// A lane's NV logits.  FULL (E = 32 NV): runs of up to eight neighbours, loaded
// as vectors; else one of every 32.
template <int NV, bool FULL>
__device__ __forceinline__ int expert_of(int lane, int i)
{
    constexpr int RUN = NV < 8 ? NV : 8;
    return FULL ? (i / RUN * 32 + lane) * RUN + i % RUN : lane + 32 * i;
}

template <class T, int NV, bool FULL>
__device__ __forceinline__ void load_row(const T *row, int E, int lane, float (&l)[NV])
{
    constexpr int RUN = NV < 8 ? NV : 8;
    if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < NV; i += RUN) {
            Vec<T, RUN> v;
            float f[RUN];
            ld_vec_keep(v, row + expert_of<NV, FULL>(lane, i));
            widen(v, f);
#pragma unroll
            for (int e = 0; e < RUN; ++e) l[i + e] = f[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            l[i] = e < E ? widen1(row[e]) : -INFINITY;
        }
    }
}

// max and sum of exp(l - max) over the row
template <int NV>
__device__ __forceinline__ void row_stats(const float (&l)[NV], float &m, float &sum)
{
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    sum = 0.f;
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) sum += expf(l[i] - m);
    sum = warp_sum(sum);
}

// Sorts NV (1, 2, 4, 8) registers in descending order: a merge network of
// compare-exchanges (19 for eight values).
template <int NV>
__device__ __forceinline__ void sort_desc(unsigned (&p)[NV])
{
    auto cx = [&](int a, int b) {
        const unsigned hi = max(p[a], p[b]), lo = min(p[a], p[b]);
        p[a] = hi;
        p[b] = lo;
    };
#pragma unroll
    for (int w = 1; w < NV; w *= 2)           // merge sorted runs of w
#pragma unroll
        for (int d = w; d >= 1; d /= 2)
#pragma unroll
            for (int i = d % w; i + d < NV; i += 2 * d)
#pragma unroll
                for (int q = 0; q < d; ++q)
                    if (i + q + d < NV && (i + q) / (2 * w) == (i + q + d) / (2 * w))
                        cx(i + q, i + q + d);
}

// The choice packs a logit's key and its index into one word: the key's upper
// 22 bits over 1023 - index, so that one integer maximum finds the
// largest logit and, among equal ones, the lowest index.  22 bits hold the
// whole of a bf16 or fp16 value (16 and 19 bits of its fp32 form).  Of a
// 32-bit logit they do not: the order is then certain unless two neighbours of
// the top k + 1 agree in them, and such a row (about 2 in 100 of normal logits
// at E = 256, k = 8) is chosen again, by whole keys.
__device__ __forceinline__ unsigned pack_of(float l, int e)
{
    return (key_of(l) & ~1023u) | unsigned(1023 - e);
}

// Exact choice by whole keys, one maximum at a time: lane j gets choice j.  The
// row is loaded again: an array handed to a function would keep every row's
// logits in local memory.
template <class T, int NV, bool FULL>
__device__ __noinline__ int choose_exact(const T *row, int E, int k)
{
    const int lane = threadIdx.x & 31;
    float l[NV];
    load_row<T, NV, FULL>(row, E, lane, l);
    unsigned key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = FULL || lane + 32 * i < E ? key_of(l[i]) : 0u;
    int mine = 0;
    for (int j = 0; j < k; ++j) {
        unsigned best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i] > best) {
                best = key[i];
                at = expert_of<NV, FULL>(lane, i);
            }
        const unsigned top = __reduce_max_sync(kFull, best);
        const int e = int(__reduce_min_sync(kFull, best == top ? unsigned(at) : ~0u));
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e == expert_of<NV, FULL>(lane, i)) key[i] = 0u;
        if (lane == j) mine = e;
    }
    return mine;
}

template <class T, int NV, bool FULL>
__global__ void __launch_bounds__(kRouterWarps * 32, NV <= 8 ? kRouterPerSm : 1)
    k_moe_router(const T *__restrict__ logits, int64_t tokens, int E, int k, int score,
                 int renorm, float scale, int32_t *__restrict__ ids, float *__restrict__ w)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
    if (t >= tokens) return;
    const T *row = logits + t * E;
    float l[NV];
    load_row<T, NV, FULL>(row, E, lane, l);
    unsigned p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        p[i] = FULL || lane + 32 * i < E ? pack_of(l[i], expert_of<NV, FULL>(lane, i)) : 0u;
    // up to eight values a lane are sorted, so that a round only looks at the
    // head; more are searched in every round
    constexpr bool kSorted = NV <= 8;
    if constexpr (kSorted) sort_desc<NV>(p);
    unsigned mine = 0u, last = 0u;  // choice `lane`; the last one
    const int rounds = sizeof(T) == 2 || k == E ? k : k + 1;
#pragma unroll 3
    for (int j = 0; j < rounds; ++j) {
        unsigned best = p[0];
        if constexpr (!kSorted)
#pragma unroll
            for (int i = 1; i < NV; ++i) best = max(best, p[i]);
        last = __reduce_max_sync(kFull, best);
        if constexpr (kSorted) {
            if (p[0] == last) {
#pragma unroll
                for (int i = 0; i + 1 < NV; ++i) p[i] = p[i + 1];
                p[NV - 1] = 0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (p[i] == last) p[i] = 0u;
        }
        if (lane == j) mine = last;
    }
    const bool on = lane < k;
    int my_id = 1023 - int(mine & 1023u);
    if constexpr (sizeof(T) == 4) {
        // neighbours in order: lanes 0 .. k - 1, then the one after them
        const unsigned next = __shfl_down_sync(kFull, mine, 1);
        const bool near = on && (mine ^ (lane == k - 1 ? last : next)) < 1024u;
        if (__any_sync(kFull, near && !(lane == k - 1 && rounds == k)))
            my_id = choose_exact<T, NV, FULL>(row, E, k);
    }
    const float my_l = on ? widen1(row[my_id]) : -INFINITY;
    float v;
    if (renorm) {
        // lane 0 has the largest
        const float s = score == 0 ? my_l : log_logistic(my_l);
        const float m = __shfl_sync(kFull, s, 0);
        v = on && m != -INFINITY ? expf(s - m) : 0.f;
        const float sum = warp_sum(v);
        v = sum == 0.f ? 0.f : v / sum;
    } else if (score == 0) {
        float m, sum;
        row_stats<NV>(l, m, sum);
        v = sum == 0.f ? 0.f : expf(my_l - m) / sum;
    } else {
        v = logistic(my_l);
    }
    if (on) {
        ids[t * k + lane] = my_id;
        w[t * k + lane] = scale * v;
    }
}

template <class T, int NV>
__global__ void __launch_bounds__(kRouterWarps * 32)
    k_moe_router_bwd(const float *__restrict__ dw, const T *__restrict__ logits,
                     const int32_t *__restrict__ ids, int64_t tokens, int E, int k, int score,
                     int renorm, float scale, T *__restrict__ dlogits, int *fault)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = int64_t(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
    if (t >= tokens) return;
    const T *row = logits + t * E;
    int id = lane < k ? __ldg(ids + t * k + lane) : -1;
    if (id < -1 || id >= E) {
        report_fault(fault, kFaultChoice);
        id = -1;
    }
    float a = id >= 0 ? scale * __ldg(dw + t * k + lane) : 0.f;
    if (renorm && __any_sync(kFull, lane < k && id < 0)) {
        // lane j takes choice j, and the gradient of the slot that kept it
        const int found = choose_exact<T, NV, false>(row, E, k), chosen = lane < k ? found : -1;
        float kept = 0.f;
        for (int j = 0; j < k; ++j) {
            const int e = __shfl_sync(kFull, id, j);
            const float v = __shfl_sync(kFull, a, j);
            if (e < 0) continue;
            if (e == chosen) kept += v;
            if (!__any_sync(kFull, e == chosen)) report_fault(fault, kFaultChoice);
        }
        id = chosen;
        a = kept;
    }
    const bool on = id >= 0;
    const float lj = on ? widen1(row[id]) : -INFINITY;
    float d;         // this lane's slot's gradient
    float out[NV];   // dlogits of experts lane, lane + 32, ...
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = 0.f;
    if (renorm) {
        const float v = lane_softmax(score == 0 ? lj : log_logistic(lj), on);
        d = v * (a - warp_sum(a * v));
        if (score != 0) d *= logistic(-lj);
    } else if (score == 0) {
        float l[NV], m, sum;
        load_row<T, NV, false>(row, E, lane, l);
        row_stats<NV>(l, m, sum);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float v = on ? expf(lj - m) * inv : 0.f;
        const float inner = warp_sum(a * v);
#pragma unroll
        for (int i = 0; i < NV; ++i) out[i] = -(expf(l[i] - m) * inv * inner);
        d = a * v;
    } else {
        const float v = logistic(lj);
        d = a * v * logistic(-lj);
    }
    if (!on) d = 0.f;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kFull, id, j);
        const float v = __shfl_sync(kFull, d, j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e == lane + 32 * i) out[i] += v;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e < E) narrow1(out[i], dlogits[t * E + e]);
    }
}

#define MHC_ROUTER_NV(NV_, ...)                          \
    if (E <= 32) { constexpr int NV_ = 1; __VA_ARGS__; } \
    else if (E <= 64) { constexpr int NV_ = 2; __VA_ARGS__; } \
    else if (E <= 128) { constexpr int NV_ = 4; __VA_ARGS__; } \
    else if (E <= 256) { constexpr int NV_ = 8; __VA_ARGS__; } \
    else if (E <= 512) { constexpr int NV_ = 16; __VA_ARGS__; } \
    else { constexpr int NV_ = 32; __VA_ARGS__; }

template <class T>
cudaError_t fwd_of(const void *logits, int64_t tokens, int E, int k, int score, int renorm,
                   float scale, int32_t *ids, float *w, cudaStream_t s)
{
    const dim3 g(unsigned((tokens + kRouterWarps - 1) / kRouterWarps));
    MHC_ROUTER_NV(NV, return launch_k(E == 32 * NV ? k_moe_router<T, NV, true>
                                                   : k_moe_router<T, NV, false>,
                                      g, dim3(kRouterWarps * 32), 0, s,
                                      static_cast<const T *>(logits), tokens, E, k, score, renorm,
                                      scale, ids, w));
}

template <class T>
cudaError_t bwd_of(const float *dw, const void *logits, const int32_t *ids, int64_t tokens, int E,
                   int k, int score, int renorm, float scale, void *dlogits, int *fault,
                   cudaStream_t s)
{
    const dim3 g(unsigned((tokens + kRouterWarps - 1) / kRouterWarps));
    MHC_ROUTER_NV(NV, return launch_k(k_moe_router_bwd<T, NV>, g, dim3(kRouterWarps * 32), 0, s,
                                      dw, static_cast<const T *>(logits), ids, tokens, E, k, score,
                                      renorm, scale, static_cast<T *>(dlogits), fault));
}

}  // namespace

cudaError_t launch_moe_router_fwd(const void *logits, int dtype, int64_t T, int E, int k,
                                  int score, int renorm, float scale, int32_t *ids, float *w,
                                  cudaStream_t s)
{
    MHC_PROF("k_moe_router", s);
    return dtype == 0   ? fwd_of<bf16>(logits, T, E, k, score, renorm, scale, ids, w, s)
           : dtype == 1 ? fwd_of<fp16>(logits, T, E, k, score, renorm, scale, ids, w, s)
                        : fwd_of<float>(logits, T, E, k, score, renorm, scale, ids, w, s);
}

cudaError_t launch_moe_router_bwd(const float *dw, const void *logits, int dtype,
                                  const int32_t *ids, int64_t T, int E, int k, int score,
                                  int renorm, float scale, void *dlogits, int *fault,
                                  cudaStream_t s)
{
    MHC_PROF("k_moe_router_bwd", s);
    return dtype == 0 ? bwd_of<bf16>(dw, logits, ids, T, E, k, score, renorm, scale, dlogits, fault, s)
           : dtype == 1
               ? bwd_of<fp16>(dw, logits, ids, T, E, k, score, renorm, scale, dlogits, fault, s)
               : bwd_of<float>(dw, logits, ids, T, E, k, score, renorm, scale, dlogits, fault, s);
}

}  // namespace mhc
