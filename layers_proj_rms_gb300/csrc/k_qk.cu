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

// V consecutive fp32 values from p (global, read-only) or from shared memory.
template <int V, bool SHARED>
__device__ __forceinline__ void load_f(const float *p, float (&f)[V])
{
    if constexpr (V == 8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 *g = reinterpret_cast<const float4 *>(p) + q;
            const float4 v = SHARED ? *g : __ldg(g);
            f[4 * q] = v.x; f[4 * q + 1] = v.y; f[4 * q + 2] = v.z; f[4 * q + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = SHARED ? p[i] : __ldg(p + i);
    }
}

// What a unit's two chunks are multiplied by: cos for a chunk's own values and
// sin for its partner's, with the signs of the forward rotation.  The partner
// of chunk a is chunk b (half-split pairs), or each value's neighbour
// (interleaved; INTER).
template <int V, bool INTER>
struct Rope {
    typedef typename Elems<V>::E E;
    static constexpr int N = Elems<V>::N, NR = INTER ? 2 * N : N;
    E c[NR], s[NR];
    __device__ __forceinline__ void load(const float *cs, const float *sn, int64_t at)
    {
        float fc[V], fs[V];
        load_f<V, false>(cs + at, fc);
        load_f<V, false>(sn + at, fs);
        if constexpr (V == 1) {
            c[0] = fc[0];
            s[0] = fs[0];
        } else if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                c[i] = f2_make(fc[i], fc[i]);
                s[i] = f2_make(-fs[i], fs[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                c[i] = f2_make(fc[2 * i], fc[2 * i + 1]);
                s[i] = f2_make(fs[2 * i], fs[2 * i + 1]);
            }
        }
    }
    __device__ __forceinline__ E ca(int i) const { return c[i]; }
    __device__ __forceinline__ E cb(int i) const { return INTER ? c[N + i] : c[i]; }
    __device__ __forceinline__ E sa(int i) const { return INTER ? s[i] : e_neg(s[i]); }
    __device__ __forceinline__ E sb(int i) const { return INTER ? s[N + i] : s[i]; }
    // the value that stands beside a's (b's) element i
    static __device__ __forceinline__ E pa(const E (&a)[N], const E (&b)[N], int i)
    {
        return INTER ? e_swap(a[i]) : b[i];
    }
    static __device__ __forceinline__ E pb(const E (&a)[N], const E (&b)[N], int i)
    {
        return INTER ? e_swap(b[i]) : a[i];
    }
};

// The block's copy of both gammas (1 where there is none), rows of Dp floats.
__device__ __forceinline__ int gamma_row(int D) { return (D + 7) & ~7; }
__device__ __forceinline__ void stage_gammas(const QkArgs &A, float *sg)
{
    const int Dp = gamma_row(A.D);
    for (int i = threadIdx.x; i < 2 * Dp; i += blockDim.x) {
        const int which = i >= Dp, d = which ? i - Dp : i;
        const float *g = A.m[which].gamma;
        sg[i] = g && d < A.D ? __ldg(g + d) : 1.f;
    }
    __syncthreads();
}
template <int V>
__device__ __forceinline__ void gamma_e(const float *sg, typename Elems<V>::E (&g)[Elems<V>::N])
{
    float f[V];
    load_f<V, true>(sg, f);
    if constexpr (V == 1) {
        g[0] = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) g[i] = f2_make(f[2 * i], f[2 * i + 1]);
    }
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

// The rows of a token whose position is outside the table: zeros.
template <class T, int V, int K, int HPI>
__device__ __forceinline__ void zero_token(const QkTensor &m, int64_t t, int h0, int ng,
                                           const int (&at)[K], const int (&bt)[K],
                                           const bool (&va)[K], const bool (&vb)[K])
{
    Vec<T, V> z;
    zero_vec(z);
#pragma unroll
    for (int i = 0; i < HPI; ++i) {
        const int h = h0 + i * ng;
        T *row = static_cast<T *>(m.out) + t * m.out_t + h * m.out_h;
#pragma unroll
        for (int q = 0; q < K; ++q) {
            if (h < m.H && va[q]) st_vec(row + at[q], z);
            if (h < m.H && vb[q]) st_vec(row + bt[q], z);
        }
    }
}

// y = rho (x (gamma cos) + partner (gamma sin)): the products with gamma are
// formed once per token and serve the set's heads.  MINB: blocks per SM that
// the registers must leave room for.
template <class T, int V, int K, int HPI, bool INTER, int MINB>
__global__ void __launch_bounds__(kQkWarps * 32, MINB)
    k_qk_fwd(const __grid_constant__ QkArgs A, const __grid_constant__ QkGeom ge)
{
    typedef typename Elems<V>::E E;
    constexpr int N = Elems<V>::N;
    typedef Rope<V, INTER> R;
    extern __shared__ __align__(16) float sg[];
    pdl_wait();
    stage_gammas(A, sg);
    Work w;
    if (!my_work(ge, w)) return;
    const QkTensor &m = A.m[w.which];
    const float *gam = sg + (w.which ? gamma_row(A.D) : 0);
    const int lane = threadIdx.x & 31, G = 1 << ge.lg, l = lane & (G - 1);
    const int ng = 32 >> ge.lg, h0 = w.set * (ng * HPI) + (lane >> ge.lg);
    const int half = A.R / 2, hr = half / V;
    const float inv_d = 1.f / float(A.D);
    int at[K], bt[K];
    bool va[K], vb[K];
#pragma unroll
    for (int q = 0; q < K; ++q) {
        unit_at<V>(l + q * G, hr, half, A.interleaved != 0, at[q], bt[q]);
        va[q] = at[q] < A.D;
        vb[q] = bt[q] < A.D;
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
        if (!position(A, t, p)) {
            zero_token<T, V, K, HPI>(m, t, h0, ng, at, bt, va, vb);
            continue;
        }
        E ca[K][N], cb[K][N], sa[K][N], sb[K][N];
#pragma unroll
        for (int q = 0; q < K; ++q) {
            E ga[N], gb[N];
            gamma_e<V>(gam + (va[q] ? at[q] : 0), ga);
            gamma_e<V>(gam + (vb[q] ? bt[q] : 0), gb);
            if (l + q * G < hr) {
                R r;
                r.load(A.cs, A.sn, p * half + V * (l + q * G));
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    ca[q][e] = e_mul(ga[e], r.ca(e));
                    cb[q][e] = e_mul(gb[e], r.cb(e));
                    sa[q][e] = e_mul(R::pa(ga, gb, e), r.sa(e));
                    sb[q][e] = e_mul(R::pb(ga, gb, e), r.sb(e));
                }
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    ca[q][e] = ga[e];
                    cb[q][e] = gb[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            const int h = h0 + i * ng;
            E a[K][N], b[K][N], ss;
            e_set(ss, 0.f);
#pragma unroll
            for (int q = 0; q < K; ++q) {
                widen_e<T, V>(xa[i][q], a[q]);
                widen_e<T, V>(xb[i][q], b[q]);
#pragma unroll
                for (int e = 0; e < N; ++e) ss = e_fma(a[q][e], a[q][e], e_fma(b[q][e], b[q][e], ss));
            }
            const float den = fmaf(group_sum(e_sum(ss), G), inv_d, A.eps);
            const float rho = den == 0.f ? 0.f : rsqrtf(den);  // an all-zero head, eps = 0: zeros
            if (h >= m.H) continue;
            E rr;
            e_set(rr, rho);
            T *row = static_cast<T *>(m.out) + t * m.out_t + h * m.out_h;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                E ya[N], yb[N];
                if (l + q * G < hr) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        ya[e] = e_mul(rr, e_fma(R::pa(a[q], b[q], e), sa[q][e],
                                                e_mul(a[q][e], ca[q][e])));
                        yb[e] = e_mul(rr, e_fma(R::pb(a[q], b[q], e), sb[q][e],
                                                e_mul(b[q][e], cb[q][e])));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        ya[e] = e_mul(rr, e_mul(a[q][e], ca[q][e]));
                        yb[e] = e_mul(rr, e_mul(b[q][e], cb[q][e]));
                    }
                }
                Vec<T, V> o;
                narrow_e<T, V>(ya, o);
                if (va[q]) st_vec(row + at[q], o);
                narrow_e<T, V>(yb, o);
                if (vb[q]) st_vec(row + bt[q], o);
            }
        }
    }
}

// dgp: [gridDim.x][2][D] partial sums of dgamma, one row per block.
template <class T, int V, int K, int HPI, bool INTER, int MINB>
__global__ void __launch_bounds__(kQkWarps * 32, MINB)
    k_qk_bwd(const __grid_constant__ QkArgs A, const __grid_constant__ QkGeom ge,
             float *__restrict__ dgp)
{
    typedef typename Elems<V>::E E;
    constexpr int N = Elems<V>::N;
    typedef Rope<V, INTER> R;
    extern __shared__ __align__(16) float sm[];  // gammas, then [kQkWarps][D] dgamma partials
    __shared__ int owner[kQkWarps];
    pdl_wait();
    stage_gammas(A, sm);
    float *part = sm + 2 * gamma_row(A.D);
    Work w;
    const bool active = my_work(ge, w);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = 1 << ge.lg, l = lane & (G - 1);
    const int ng = 32 >> ge.lg;
    const int half = A.R / 2, hr = half / V;
    const float inv_d = 1.f / float(A.D);
    if (lane == 0) owner[warp] = active ? w.which : -1;
    if (active) {
        const QkTensor &m = A.m[w.which];
        const float *gam = sm + (w.which ? gamma_row(A.D) : 0);
        const int h0 = w.set * (ng * HPI) + (lane >> ge.lg);
        int at[K], bt[K];
        bool va[K], vb[K];
        E da[K][N], db[K][N];
#pragma unroll
        for (int q = 0; q < K; ++q) {
            unit_at<V>(l + q * G, hr, half, A.interleaved != 0, at[q], bt[q]);
            va[q] = at[q] < A.D;
            vb[q] = bt[q] < A.D;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                e_set(da[q][e], 0.f);
                e_set(db[q][e], 0.f);
            }
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
            if (!position(A, t, p)) {
                zero_token<T, V, K, HPI>(m, t, h0, ng, at, bt, va, vb);
                continue;
            }
            R r[K];
#pragma unroll
            for (int q = 0; q < K; ++q)
                if (l + q * G < hr) r[q].load(A.cs, A.sn, p * half + V * (l + q * G));
#pragma unroll
            for (int i = 0; i < HPI; ++i) {
                const int h = h0 + i * ng;
                E s1, s2;  // sum x^2, sum g x
                e_set(s1, 0.f);
                e_set(s2, 0.f);
                E a[K][N], b[K][N], u[K][N], v[K][N];  // x, then the upstream rotated back
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    E ga[N], gb[N];
                    gamma_e<V>(gam + (va[q] ? at[q] : 0), ga);
                    gamma_e<V>(gam + (vb[q] ? bt[q] : 0), gb);
                    widen_e<T, V>(xa[i][q], a[q]);
                    widen_e<T, V>(xb[i][q], b[q]);
                    widen_e<T, V>(ya[i][q], u[q]);
                    widen_e<T, V>(yb[i][q], v[q]);
                    if (l + q * G < hr) {
                        E ru[N], rv[N];
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            ru[e] = e_fma(R::pa(u[q], v[q], e), e_neg(r[q].sa(e)),
                                          e_mul(u[q][e], r[q].ca(e)));
                            rv[e] = e_fma(R::pb(u[q], v[q], e), e_neg(r[q].sb(e)),
                                          e_mul(v[q][e], r[q].cb(e)));
                        }
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            u[q][e] = ru[e];
                            v[q][e] = rv[e];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        s1 = e_fma(a[q][e], a[q][e], e_fma(b[q][e], b[q][e], s1));
                        s2 = e_fma(e_mul(u[q][e], ga[e]), a[q][e],
                                   e_fma(e_mul(v[q][e], gb[e]), b[q][e], s2));
                    }
                }
                const float den = fmaf(group_sum(e_sum(s1), G), inv_d, A.eps);
                const float rho = den == 0.f ? 0.f : rsqrtf(den);
                const float k2 = group_sum(e_sum(s2), G) * rho * inv_d;  // mean of g xh
                if (h >= m.H) continue;
                E rr, nk;
                e_set(rr, rho);
                e_set(nk, -k2);
                T *row = static_cast<T *>(m.out) + t * m.out_t + h * m.out_h;
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    E ga[N], gb[N], o1[N], o2[N];
                    gamma_e<V>(gam + (va[q] ? at[q] : 0), ga);
                    gamma_e<V>(gam + (vb[q] ? bt[q] : 0), gb);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const E ha = e_mul(a[q][e], rr), hb = e_mul(b[q][e], rr);
                        o1[e] = e_mul(rr, e_fma(ha, nk, e_mul(u[q][e], ga[e])));
                        o2[e] = e_mul(rr, e_fma(hb, nk, e_mul(v[q][e], gb[e])));
                        da[q][e] = e_fma(u[q][e], ha, da[q][e]);
                        db[q][e] = e_fma(v[q][e], hb, db[q][e]);
                    }
                    Vec<T, V> o;
                    narrow_e<T, V>(o1, o);
                    if (va[q]) st_vec(row + at[q], o);
                    narrow_e<T, V>(o2, o);
                    if (vb[q]) st_vec(row + bt[q], o);
                }
            }
        }
        if (dgp) {
#pragma unroll
            for (int q = 0; q < K; ++q) {
                float fa[V], fb[V];
                if constexpr (V == 1) {
                    fa[0] = da[q][0];
                    fb[0] = db[q][0];
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        f2_split(da[q][e], fa[2 * e], fa[2 * e + 1]);
                        f2_split(db[q][e], fb[2 * e], fb[2 * e + 1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    for (int x = 16; x >= G; x >>= 1) {
                        fa[e] += __shfl_xor_sync(kFull, fa[e], x);
                        fb[e] += __shfl_xor_sync(kFull, fb[e], x);
                    }
                    if (lane < G && va[q]) part[warp * A.D + at[q] + e] = fa[e];
                    if (lane < G && vb[q]) part[warp * A.D + bt[q] + e] = fb[e];
                }
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
            if (owner[k] == which) v += part[k * A.D + d];
        dgp[int64_t(blockIdx.x) * 2 * A.D + i] = v;
    }
}

// dgamma[d] = sum of the blocks' partials in a fixed order.  A block has 8
// columns; thread (x, y) adds rows y, y + 128, ... of column x, and the 128
// sums of a column are added by one warp.
__global__ void __launch_bounds__(1024)
    k_qk_dgamma(const float *__restrict__ part, int rows, int D, float *__restrict__ dgq,
                float *__restrict__ dgk)
{
    pdl_wait();
    __shared__ float red[8][128];
    const int x = threadIdx.x & 7, y = threadIdx.x >> 3, c = blockIdx.x * 8 + x;
    float s = 0.f;
    if (c < 2 * D)
#pragma unroll 4
        for (int r = y; r < rows; r += 128) s += __ldg(part + int64_t(r) * 2 * D + c);
    red[x][y] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31, col = threadIdx.x >> 5;
    if (col >= 8) return;
    const float t = warp_sum((red[col][lane] + red[col][lane + 32]) +
                             (red[col][lane + 64] + red[col][lane + 96]));
    const int d = blockIdx.x * 8 + col;
    if (lane == 0 && d < 2 * D) {
        float *out = d < D ? dgq : dgk;
        if (out) out[d < D ? d : d - D] = t;
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

// Blocks of a launch: as many as stay resident, MINB per SM.
constexpr int qk_blocks(int minb) { return kSplitSms * minb; }
constexpr int kQkBwdMaxBlocks = qk_blocks(4);  // what the workspace allows for

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

template <class T, int V, int K, int HPI, int MINB>
cudaError_t run_fwd(const QkArgs &a, cudaStream_t s)
{
    int blocks;
    const QkGeom g = qk_geom(a, V, HPI, qk_blocks(MINB), &blocks);
    const size_t smem = size_t(2) * ((a.D + 7) & ~7) * sizeof(float);
    auto kernel = V > 1 && a.interleaved ? k_qk_fwd<T, V, K, HPI, (V > 1), MINB>
                                         : k_qk_fwd<T, V, K, HPI, false, MINB>;
    MHC_PROF("k_qk_fwd", s);
    return launch_k(kernel, dim3(unsigned(blocks)), dim3(kQkWarps * 32), smem, s, a, g);
}

template <class T, int V, int K, int HPI, int MINB>
cudaError_t run_bwd(const QkArgs &a, float *ws, cudaStream_t s)
{
    static_assert(qk_blocks(MINB) <= kQkBwdMaxBlocks, "the workspace has a row per block");
    int blocks;
    const QkGeom g = qk_geom(a, V, HPI, qk_blocks(MINB), &blocks);
    float *part = a.m[0].dgamma || a.m[1].dgamma ? ws : nullptr;
    const size_t smem = (size_t(2) * ((a.D + 7) & ~7) + (part ? size_t(kQkWarps) * a.D : 0)) *
                        sizeof(float);
    auto kernel = V > 1 && a.interleaved ? k_qk_bwd<T, V, K, HPI, (V > 1), MINB>
                                         : k_qk_bwd<T, V, K, HPI, false, MINB>;
    {
        MHC_PROF("k_qk_bwd", s);
        const cudaError_t e = launch_k(kernel, dim3(unsigned(blocks)), dim3(kQkWarps * 32), smem, s,
                                       a, g, part);
        if (e != cudaSuccess || !part) return e;
    }
    MHC_PROF("k_qk_dgamma", s);
    return launch_k(k_qk_dgamma, dim3(unsigned((2 * a.D + 7) / 8)), dim3(1024), 0, s, part, blocks,
                    a.D, a.m[0].dgamma, a.m[1].dgamma);
}

// Heads per lane group and blocks per SM of the 16-byte forms on long inputs.
// 16384 tokens of 32 + 8 heads of 128, bf16: forward 2, 3 take 56.2 us; 4, 3
// (spills) 59.2; 4, 2 64.3; 1, 4 62.4.  Backward 2, 2 take 95.0; 1, 2 108;
// 1, 3 122.
constexpr int kFwdHeads = 2, kFwdBlocks = 3, kBwdHeads = 2, kBwdBlocks = 2;

template <class T>
cudaError_t fwd_of(const QkArgs &a, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        if (!qk_many(a)) return run_fwd<T, 8, 1, 1, 3>(a, s);
        if constexpr (sizeof(T) == 4) return run_fwd<T, 8, 1, 2, 3>(a, s);
        else return run_fwd<T, 8, 1, kFwdHeads, kFwdBlocks>(a, s);
    case 2:
        if (a.D > 128) return run_fwd<T, 2, 4, 1, 2>(a, s);
        return qk_many(a) ? run_fwd<T, 2, 1, 4, 4>(a, s) : run_fwd<T, 2, 1, 1, 4>(a, s);
    default:
        return a.D > 128 ? run_fwd<T, 1, 8, 1, 2>(a, s) : run_fwd<T, 1, 2, 2, 3>(a, s);
    }
}

template <class T>
cudaError_t bwd_of(const QkArgs &a, float *ws, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        if constexpr (sizeof(T) == 2)
            if (qk_many(a)) return run_bwd<T, 8, 1, kBwdHeads, kBwdBlocks>(a, ws, s);
        return run_bwd<T, 8, 1, 1, 2>(a, ws, s);
    case 2:
        if (a.D > 128) return run_bwd<T, 2, 4, 1, 2>(a, ws, s);
        return qk_many(a) ? run_bwd<T, 2, 1, 4, 3>(a, ws, s) : run_bwd<T, 2, 1, 1, 3>(a, ws, s);
    default:
        return a.D > 128 ? run_bwd<T, 1, 8, 1, 1>(a, ws, s) : run_bwd<T, 1, 2, 2, 2>(a, ws, s);
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
