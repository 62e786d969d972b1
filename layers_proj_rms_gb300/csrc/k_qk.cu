// RMS norm of every query and key head with the position rotation in the
// same pass, forward and backward.
//
//   rho = (sum_d x_d^2 / D + eps)^-1/2,  a = x rho gamma
//   rotated pairs (i, j), p = pair index, c = cos[pos][p], s = sin[pos][p]:
//     y_i = a_i c - a_j s,   y_j = a_j c + a_i s;   y_d = a_d for d >= R
//   backward: b = the inverse rotation of dy (b_i = dy_i c + dy_j s,
//     b_j = dy_j c - dy_i s), g = b gamma, xh = x rho,
//     dx = rho (g - xh (sum_d g xh) / D),  dgamma_d = sum_{t, h} b_d xh_d.
//
// Layout of the work.  The two elements of a rotated pair are R/2 apart (or
// neighbours, interleaved), so a lane owns a unit of two chunks of V elements
// that hold whole pairs: chunks u and u + R/(2V) of the rotated part, or two
// neighbouring chunks.  No element crosses lanes; a head is G lanes (a power
// of two) and its sums are log2(G) butterflies.  A warp keeps one tensor (q
// or k) and one set of heads for its life, so gamma stays in registers, and
// walks over tokens; the token's cos and sin serve all heads of the set.
//
// V = 8 (16-byte vectors for 16-bit types) needs R a multiple of 16, D of 8,
// and strides and pointers on 16 bytes; V = 2 needs R a multiple of 4 and D
// of 2; V = 1 takes anything.  The result of a head does not depend on V's
// vectorised loads, the grid or T: the order of its sums is fixed by D and R.
#include "qk.h"

#include "elem.cuh"
#include "launch.h"

namespace mhc {

constexpr int kFaultPosition = 201;  // a position outside the table

namespace {

constexpr int kQkWarps = 8;  // warps of a block

struct QkGeom {
    int lg;         // log2 of the lanes of a head
    int nb[2];      // head sets of q, k
    int64_t t_step; // tokens advanced per iteration of a warp
};

__device__ __forceinline__ float group_sum(float v, int G)
{
    for (int m = G >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    return v;
}

// First element of the unit's two chunks; hr = units of the rotated part.
template <int V>
__device__ __forceinline__ void unit_at(int u, int hr, int half, bool inter, int &a, int &b)
{
    if (!inter && u < hr) {
        a = V * u;
        b = half + V * u;
    } else {
        a = inter ? 2 * V * u : 2 * half + 2 * V * (u - hr);
        b = a + V;
    }
}

// cos and sin of the V pairs of unit u.
template <int V>
__device__ __forceinline__ void load_rope(const float *cs, const float *sn, int64_t at,
                                          float (&c)[V], float (&s)[V])
{
    if constexpr (V == 8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 cv = __ldg(reinterpret_cast<const float4 *>(cs + at) + q);
            const float4 sv = __ldg(reinterpret_cast<const float4 *>(sn + at) + q);
            c[4 * q] = cv.x; c[4 * q + 1] = cv.y; c[4 * q + 2] = cv.z; c[4 * q + 3] = cv.w;
            s[4 * q] = sv.x; s[4 * q + 1] = sv.y; s[4 * q + 2] = sv.z; s[4 * q + 3] = sv.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = __ldg(cs + at + i);
            s[i] = __ldg(sn + at + i);
        }
    }
}

// Rotates the V pairs of a unit by (c, s); sgn = -1 rotates back.
template <int V>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float (&c)[V],
                                       const float (&s)[V], bool inter, float sgn)
{
    auto turn = [&](float &u, float &v, float cc, float ss) {
        const float x = u, y = v;
        ss *= sgn;
        u = x * cc - y * ss;
        v = y * cc + x * ss;
    };
    if (V == 1 || !inter) {
#pragma unroll
        for (int i = 0; i < V; ++i) turn(a[i], b[i], c[i], s[i]);
    } else if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
            turn(b[2 * i], b[2 * i + 1], c[V / 2 + i], s[V / 2 + i]);
        }
    }
}

template <int V>
__device__ __forceinline__ void load_gamma(const float *gamma, int at, bool on, float (&g)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = on ? (gamma ? __ldg(gamma + at + i) : 1.f) : 0.f;
}

// What a warp does: tensor, head set, first token.
struct Work {
    int which, set;
    int64_t t;
};
__device__ __forceinline__ bool my_work(const QkGeom &ge, Work &w)
{
    const int64_t gw = int64_t(blockIdx.x) * kQkWarps + (threadIdx.x >> 5);
    const int nb = ge.nb[0] + ge.nb[1];
    const int hb = int(gw % nb);
    w.t = gw / nb;
    w.which = hb >= ge.nb[0];
    w.set = w.which ? hb - ge.nb[0] : hb;
    return w.t < ge.t_step;
}

// Position of token t; false (and a fault) when it is outside the table.
__device__ __forceinline__ bool position(const QkArgs &A, int64_t t, int64_t &p)
{
    p = A.pos ? int64_t(__ldg(A.pos + t)) : t;
    if (A.R == 0 || (p >= 0 && p < A.P)) return true;
    if ((threadIdx.x & 31) == 0) report_fault(A.fault, kFaultPosition);
    return false;
}

template <class T, int V, int K, int HPI>
__global__ void __launch_bounds__(kQkWarps * 32)
    k_qk_fwd(const __grid_constant__ QkArgs A, const __grid_constant__ QkGeom ge)
{
    pdl_wait();
    Work w;
    if (!my_work(ge, w)) return;
    const QkTensor &m = A.m[w.which];
    const int lane = threadIdx.x & 31, G = 1 << ge.lg, l = lane & (G - 1);
    const int ng = 32 >> ge.lg, h0 = w.set * (ng * HPI) + (lane >> ge.lg);
    const int half = A.R / 2, hr = half / V;
    const bool inter = A.interleaved != 0;
    const float inv_d = 1.f / float(A.D);
    int at[K], bt[K];
    bool va[K], vb[K];
    float ga[K][V], gb[K][V];
#pragma unroll
    for (int q = 0; q < K; ++q) {
        unit_at<V>(l + q * G, hr, half, inter, at[q], bt[q]);
        va[q] = at[q] < A.D;
        vb[q] = bt[q] < A.D;
        load_gamma<V>(m.gamma, at[q], va[q], ga[q]);
        load_gamma<V>(m.gamma, bt[q], vb[q], gb[q]);
    }
    for (int64_t t = w.t; t < A.T; t += ge.t_step) {
        Vec<T, V> xa[HPI][K], xb[HPI][K];
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            const int h = h0 + i * ng;
            const T *row = static_cast<const T *>(m.x) + t * m.x_t + h * m.x_h;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                if (h < m.H && va[q]) ld_vec(xa[i][q], row + at[q]); else zero_vec(xa[i][q]);
                if (h < m.H && vb[q]) ld_vec(xb[i][q], row + bt[q]); else zero_vec(xb[i][q]);
            }
        }
        int64_t p;
        const bool ok = position(A, t, p);
        float c[K][V], s[K][V];
#pragma unroll
        for (int q = 0; q < K; ++q)
            if (ok && l + q * G < hr)
                load_rope<V>(A.cs, A.sn, p * half + V * (l + q * G), c[q], s[q]);
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            const int h = h0 + i * ng;
            float ss = 0.f;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                float a[V], b[V];
                widen(xa[i][q], a);
                widen(xb[i][q], b);
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
            }
            ss = group_sum(ss, G);
            const float den = ss * inv_d + A.eps;
            // an all-zero head with eps = 0 gives zeros; an invalid position too
            const float rho = den == 0.f || !ok ? 0.f : rsqrtf(den);
            if (h >= m.H) continue;
            T *row = static_cast<T *>(m.out) + t * m.out_t + h * m.out_h;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                float a[V], b[V];
                widen(xa[i][q], a);
                widen(xb[i][q], b);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a[e] = ok ? a[e] * rho * ga[q][e] : 0.f;
                    b[e] = ok ? b[e] * rho * gb[q][e] : 0.f;
                }
                if (ok && l + q * G < hr) rotate<V>(a, b, c[q], s[q], inter, 1.f);
                Vec<T, V> o;
                narrow(a, o);
                if (va[q]) st_vec(row + at[q], o);
                narrow(b, o);
                if (vb[q]) st_vec(row + bt[q], o);
            }
        }
    }
}

// dgp: [gridDim.x][2][D] partial sums of dgamma, one row per block.
template <class T, int V, int K, int HPI>
__global__ void __launch_bounds__(kQkWarps * 32)
    k_qk_bwd(const __grid_constant__ QkArgs A, const __grid_constant__ QkGeom ge,
             float *__restrict__ dgp)
{
    extern __shared__ float sm[];  // [kQkWarps][D]: a warp's dgamma partial
    __shared__ int owner[kQkWarps];
    pdl_wait();
    Work w;
    const bool active = my_work(ge, w);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = 1 << ge.lg, l = lane & (G - 1);
    const int ng = 32 >> ge.lg;
    const int half = A.R / 2, hr = half / V;
    const bool inter = A.interleaved != 0;
    const float inv_d = 1.f / float(A.D);
    if (lane == 0) owner[warp] = active ? w.which : -1;
    if (active) {
        const QkTensor &m = A.m[w.which];
        const int h0 = w.set * (ng * HPI) + (lane >> ge.lg);
        int at[K], bt[K];
        bool va[K], vb[K];
        float ga[K][V], gb[K][V], da[K][V], db[K][V];
#pragma unroll
        for (int q = 0; q < K; ++q) {
            unit_at<V>(l + q * G, hr, half, inter, at[q], bt[q]);
            va[q] = at[q] < A.D;
            vb[q] = bt[q] < A.D;
            load_gamma<V>(m.gamma, at[q], va[q], ga[q]);
            load_gamma<V>(m.gamma, bt[q], vb[q], gb[q]);
#pragma unroll
            for (int e = 0; e < V; ++e) da[q][e] = db[q][e] = 0.f;
        }
        for (int64_t t = w.t; t < A.T; t += ge.t_step) {
            Vec<T, V> xa[HPI][K], xb[HPI][K], ya[HPI][K], yb[HPI][K];
#pragma unroll
            for (int i = 0; i < HPI; ++i) {
                const int h = h0 + i * ng;
                const T *row = static_cast<const T *>(m.x) + t * m.x_t + h * m.x_h;
                const T *up = static_cast<const T *>(m.up) + t * m.up_t + h * m.up_h;
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    const bool la = h < m.H && va[q], lb = h < m.H && vb[q];
                    if (la) ld_vec(xa[i][q], row + at[q]); else zero_vec(xa[i][q]);
                    if (lb) ld_vec(xb[i][q], row + bt[q]); else zero_vec(xb[i][q]);
                    if (la) ld_vec(ya[i][q], up + at[q]); else zero_vec(ya[i][q]);
                    if (lb) ld_vec(yb[i][q], up + bt[q]); else zero_vec(yb[i][q]);
                }
            }
            int64_t p;
            const bool ok = position(A, t, p);
            float c[K][V], s[K][V];
#pragma unroll
            for (int q = 0; q < K; ++q)
                if (ok && l + q * G < hr)
                    load_rope<V>(A.cs, A.sn, p * half + V * (l + q * G), c[q], s[q]);
#pragma unroll
            for (int i = 0; i < HPI; ++i) {
                const int h = h0 + i * ng;
                float s1 = 0.f, s2 = 0.f;  // sum x^2, sum g x
                float a[K][V], b[K][V], u[K][V], v[K][V];
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    widen(xa[i][q], a[q]);
                    widen(xb[i][q], b[q]);
                    widen(ya[i][q], u[q]);
                    widen(yb[i][q], v[q]);
                    if (ok && l + q * G < hr) rotate<V>(u[q], v[q], c[q], s[q], inter, -1.f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        s1 = fmaf(a[q][e], a[q][e], fmaf(b[q][e], b[q][e], s1));
                        s2 = fmaf(u[q][e] * ga[q][e], a[q][e],
                                  fmaf(v[q][e] * gb[q][e], b[q][e], s2));
                    }
                }
                s1 = group_sum(s1, G);
                s2 = group_sum(s2, G);
                const float den = s1 * inv_d + A.eps;
                const float rho = den == 0.f || !ok ? 0.f : rsqrtf(den);
                const float k2 = s2 * rho * inv_d;  // mean of g xh
                if (h >= m.H) continue;
                T *row = static_cast<T *>(m.out) + t * m.out_t + h * m.out_h;
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    float o1[V], o2[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float xa_ = a[q][e] * rho, xb_ = b[q][e] * rho;
                        o1[e] = ok ? rho * (u[q][e] * ga[q][e] - xa_ * k2) : 0.f;
                        o2[e] = ok ? rho * (v[q][e] * gb[q][e] - xb_ * k2) : 0.f;
                        if (ok) {
                            da[q][e] = fmaf(u[q][e], xa_, da[q][e]);
                            db[q][e] = fmaf(v[q][e], xb_, db[q][e]);
                        }
                    }
                    Vec<T, V> o;
                    narrow(o1, o);
                    if (va[q]) st_vec(row + at[q], o);
                    narrow(o2, o);
                    if (vb[q]) st_vec(row + bt[q], o);
                }
            }
        }
        if (dgp) {
#pragma unroll
            for (int q = 0; q < K; ++q)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    for (int x = 16; x >= G; x >>= 1) {
                        da[q][e] += __shfl_xor_sync(kFull, da[q][e], x);
                        db[q][e] += __shfl_xor_sync(kFull, db[q][e], x);
                    }
                    if (lane < G && va[q]) sm[warp * A.D + at[q] + e] = da[q][e];
                    if (lane < G && vb[q]) sm[warp * A.D + bt[q] + e] = db[q][e];
                }
        }
    }
    if (!dgp) return;
    __syncthreads();
    // the block's partial: its warps in ascending order, per tensor
    for (int i = threadIdx.x; i < 2 * A.D; i += blockDim.x) {
        const int which = i >= A.D, d = which ? i - A.D : i;
        float v = 0.f;
        for (int k = 0; k < kQkWarps; ++k)
            if (owner[k] == which) v += sm[k * A.D + d];
        dgp[int64_t(blockIdx.x) * 2 * A.D + i] = v;
    }
}

// dgamma[d] = sum of the blocks' partials in a fixed order: thread (x, y) of
// a 32 x 32 block adds rows y, y + 32, ... of its column, then the 32 sums
// are added in ascending y.
__global__ void __launch_bounds__(1024)
    k_qk_dgamma(const float *__restrict__ part, int rows, int D, float *__restrict__ dgq,
                float *__restrict__ dgk)
{
    pdl_wait();
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < 2 * D)
        for (int r = threadIdx.y; r < rows; r += 32) s += part[int64_t(r) * 2 * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * D) {
        float t = 0.f;
        for (int g = 0; g < 32; ++g) t += red[g][threadIdx.x];
        float *out = c < D ? dgq : dgk;
        if (out) out[c < D ? c : c - D] = t;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

bool on(const void *p, int64_t st, int64_t sh, int es, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && st * es % bytes == 0 &&
           sh * es % bytes == 0;
}

// Elements of a chunk: the widest form whose rules the call meets.
int qk_vec(const QkArgs &a, int es)
{
    for (int v : {8, 2}) {
        bool ok = a.D % v == 0 && (a.R / 2) % v == 0;
        const int bytes = v == 8 ? 16 : 2 * es;
        for (const QkTensor &m : a.m)
            if (m.H > 0)
                ok = ok && on(m.x, m.x_t, m.x_h, es, bytes) && on(m.out, m.out_t, m.out_h, es, bytes) &&
                     (!m.up || on(m.up, m.up_t, m.up_h, es, bytes));
        if (ok) return v;
    }
    return 1;
}

constexpr int kQkMaxBlocks = kSplitSms * 4;     // forward: four blocks of 8 warps per SM
constexpr int kQkBwdMaxBlocks = kSplitSms * 2;  // backward: two

QkGeom qk_geom(const QkArgs &a, int V, int hpi, int max_blocks, int *blocks)
{
    QkGeom g;
    const int units = (a.D + 2 * V - 1) / (2 * V);
    g.lg = 0;
    while (g.lg < 5 && (1 << g.lg) < units) ++g.lg;
    const int per = (32 >> g.lg) * hpi;
    for (int i = 0; i < 2; ++i) g.nb[i] = (a.m[i].H + per - 1) / per;
    const int64_t nb = g.nb[0] + g.nb[1];
    const int64_t need = (a.T * nb + kQkWarps - 1) / kQkWarps;
    int64_t b = need < max_blocks ? need : max_blocks;
    if (b * kQkWarps < nb) b = (nb + kQkWarps - 1) / kQkWarps;  // one token a pass at least
    *blocks = int(b);
    g.t_step = b * kQkWarps / nb;
    return g;
}

// Enough warps to fill the SMs even with one head (per lane group) a warp?
bool qk_many(const QkArgs &a) { return a.T * (a.m[0].H + a.m[1].H) >= int64_t(kSplitSms) * 64; }

template <class T, int V, int K, int HPI>
cudaError_t run_fwd(const QkArgs &a, cudaStream_t s)
{
    int blocks;
    const QkGeom g = qk_geom(a, V, HPI, kQkMaxBlocks, &blocks);
    MHC_PROF("k_qk_fwd", s);
    return launch_k(k_qk_fwd<T, V, K, HPI>, dim3(unsigned(blocks)), dim3(kQkWarps * 32), 0, s, a, g);
}

template <class T, int V, int K, int HPI>
cudaError_t run_bwd(const QkArgs &a, float *ws, cudaStream_t s)
{
    int blocks;
    const QkGeom g = qk_geom(a, V, HPI, kQkBwdMaxBlocks, &blocks);
    float *part = a.m[0].dgamma || a.m[1].dgamma ? ws : nullptr;
    const size_t smem = part ? size_t(kQkWarps) * a.D * sizeof(float) : 0;
    {
        MHC_PROF("k_qk_bwd", s);
        const cudaError_t e = launch_k(k_qk_bwd<T, V, K, HPI>, dim3(unsigned(blocks)),
                                       dim3(kQkWarps * 32), smem, s, a, g, part);
        if (e != cudaSuccess || !part) return e;
    }
    MHC_PROF("k_qk_dgamma", s);
    return launch_k(k_qk_dgamma, dim3(unsigned((2 * a.D + 31) / 32)), dim3(32, 32), 0, s, part,
                    blocks, a.D, a.m[0].dgamma, a.m[1].dgamma);
}

template <class T>
cudaError_t fwd_of(const QkArgs &a, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        return qk_many(a) ? run_fwd<T, 8, 1, (sizeof(T) == 4 ? 2 : 4)>(a, s)
                          : run_fwd<T, 8, 1, 1>(a, s);
    case 2:
        if (a.D > 128) return run_fwd<T, 2, 4, 1>(a, s);
        return qk_many(a) ? run_fwd<T, 2, 1, 4>(a, s) : run_fwd<T, 2, 1, 1>(a, s);
    default:
        return a.D > 128 ? run_fwd<T, 1, 8, 1>(a, s) : run_fwd<T, 1, 2, 2>(a, s);
    }
}

template <class T>
cudaError_t bwd_of(const QkArgs &a, float *ws, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        return qk_many(a) && sizeof(T) == 2 ? run_bwd<T, 8, 1, 2>(a, ws, s)
                                            : run_bwd<T, 8, 1, 1>(a, ws, s);
    case 2:
        if (a.D > 128) return run_bwd<T, 2, 4, 1>(a, ws, s);
        return qk_many(a) ? run_bwd<T, 2, 1, 4>(a, ws, s) : run_bwd<T, 2, 1, 1>(a, ws, s);
    default:
        return a.D > 128 ? run_bwd<T, 1, 8, 1>(a, ws, s) : run_bwd<T, 1, 2, 2>(a, ws, s);
    }
}

}  // namespace

// One row of partials per block; the backward never has more blocks than
// kQkBwdMaxBlocks, one for every 8 of its T * heads work items, or one token's
// head sets.
size_t qk_bwd_ws_bytes(int64_t T, int64_t heads, int64_t D)
{
    if (T <= 0 || heads <= 0) return 0;
    const int64_t one = (heads + kQkWarps - 1) / kQkWarps;
    const int64_t cap = kQkBwdMaxBlocks > one ? kQkBwdMaxBlocks : one;
    const int64_t need = T > cap * kQkWarps / heads ? cap : (T * heads + kQkWarps - 1) / kQkWarps;
    return ws_align(size_t(need < cap ? need : cap) * 2 * size_t(D) * sizeof(float));
}

cudaError_t launch_qk_fwd(const QkArgs &a, int dtype, cudaStream_t s)
{
    return dtype == 0 ? fwd_of<bf16>(a, s) : dtype == 1 ? fwd_of<fp16>(a, s) : fwd_of<float>(a, s);
}

cudaError_t launch_qk_bwd(const QkArgs &a, int dtype, float *ws, cudaStream_t s)
{
    return dtype == 0 ? bwd_of<bf16>(a, ws, s)
                      : dtype == 1 ? bwd_of<fp16>(a, ws, s) : bwd_of<float>(a, ws, s);
}

}  // namespace mhc
