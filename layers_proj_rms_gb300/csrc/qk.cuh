// Device code that the q/k norm + rotation kernels share: how a head's
// elements lie on lanes, the rotation, gammas, positions, and the work of a warp.
#pragma once

#include "elem.cuh"
#include "launch.h"
#include "qk.h"

namespace mhc {

constexpr int kFaultPosition = 201;  // a position outside the table

constexpr int kQkWarps = 8;  // warps of a block

struct QkGeom {
    int lg;         // log2 of the lanes of a head
    int nb[2];      // head sets of q, k
    int64_t t_step; // tokens advanced per iteration of a warp
};

// Sum over the G lanes of a head (FLG >= 0: G is 2^FLG, known at compile time).
template <int FLG = -1>
__device__ __forceinline__ float group_sum(float v, int G)
{
    if constexpr (FLG >= 0) {
#pragma unroll
        for (int m = (1 << FLG) >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    } else {
        for (int m = G >> 1; m > 0; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    }
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
    if constexpr (V >= 4) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
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
        set(fc, fs);
    }
    __device__ __forceinline__ void set(const float (&fc)[V], const float (&fs)[V])
    {
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

// Forward arithmetic of a unit.  y = rho (x (gamma cos) + partner (gamma sin)):
// the products with gamma are formed once per token and serve all its heads.
template <int V, bool INTER>
struct UnitFwd {
    typedef typename Elems<V>::E E;
    typedef Rope<V, INTER> R;
    static constexpr int N = Elems<V>::N;
    E ca[N], cb[N], sa[N], sb[N];
    __device__ __forceinline__ void fold(const E (&ga)[N], const E (&gb)[N], const R &r)
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            ca[e] = e_mul(ga[e], r.ca(e));
            cb[e] = e_mul(gb[e], r.cb(e));
            sa[e] = e_mul(R::pa(ga, gb, e), r.sa(e));
            sb[e] = e_mul(R::pb(ga, gb, e), r.sb(e));
        }
    }
    __device__ __forceinline__ void still(const E (&ga)[N], const E (&gb)[N])
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            ca[e] = ga[e];
            cb[e] = gb[e];
        }
    }
    __device__ __forceinline__ void apply(const E (&a)[N], const E (&b)[N], E rho, bool turned,
                                          E (&ya)[N], E (&yb)[N]) const
    {
        if (turned) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                ya[e] = e_mul(rho, e_fma(R::pa(a, b, e), sa[e], e_mul(a[e], ca[e])));
                yb[e] = e_mul(rho, e_fma(R::pb(a, b, e), sb[e], e_mul(b[e], cb[e])));
            }
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                ya[e] = e_mul(rho, e_mul(a[e], ca[e]));
                yb[e] = e_mul(rho, e_mul(b[e], cb[e]));
            }
        }
    }
};

// Sum of squares of a unit onto ss.
template <int V>
__device__ __forceinline__ void add_squares(const typename Elems<V>::E (&a)[Elems<V>::N],
                                            const typename Elems<V>::E (&b)[Elems<V>::N],
                                            typename Elems<V>::E &ss)
{
#pragma unroll
    for (int e = 0; e < Elems<V>::N; ++e) ss = e_fma(a[e], a[e], e_fma(b[e], b[e], ss));
}

// 1 / rms of a head; an all-zero head with eps = 0 gives 0
__device__ __forceinline__ float inv_rms(float ss, float inv_d, float eps)
{
    const float den = fmaf(ss, inv_d, eps);
    return den == 0.f ? 0.f : rsqrtf(den);
}

// Backward arithmetic of a unit: the upstream gradient rotated back (u, v),
// its products with gamma, and their sum with x.
template <int V, bool INTER>
struct UnitBwd {
    typedef typename Elems<V>::E E;
    typedef Rope<V, INTER> R;
    static constexpr int N = Elems<V>::N;
    E a[N], b[N], u[N], v[N], ug[N], vg[N];
    __device__ __forceinline__ void turn_back(const R &r)
    {
        E ru[N], rv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            ru[e] = e_fma(R::pa(u, v, e), e_neg(r.sa(e)), e_mul(u[e], r.ca(e)));
            rv[e] = e_fma(R::pb(u, v, e), e_neg(r.sb(e)), e_mul(v[e], r.cb(e)));
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
            u[e] = ru[e];
            v[e] = rv[e];
        }
    }
    __device__ __forceinline__ void sums(const E (&ga)[N], const E (&gb)[N], E &s1, E &s2)
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            ug[e] = e_mul(u[e], ga[e]);
            vg[e] = e_mul(v[e], gb[e]);
            s2 = e_fma(ug[e], a[e], e_fma(vg[e], b[e], s2));
        }
        add_squares<V>(a, b, s1);
    }
    // rho, and minus the mean of g xh; da, db: dgamma so far
    __device__ __forceinline__ void grads(E rho, E nk, E (&o1)[N], E (&o2)[N], E (&da)[N], E (&db)[N]) const
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const E ha = e_mul(a[e], rho), hb = e_mul(b[e], rho);
            o1[e] = e_mul(rho, e_fma(ha, nk, ug[e]));
            o2[e] = e_mul(rho, e_fma(hb, nk, vg[e]));
            da[e] = e_fma(u[e], ha, da[e]);
            db[e] = e_fma(v[e], hb, db[e]);
        }
    }
};

// The warp's dgamma onto lanes 0..G-1 (the groups added in a fixed order) and
// from there to part [D].
template <int V>
__device__ __forceinline__ void put_dgamma(const typename Elems<V>::E (&da)[Elems<V>::N],
                                           const typename Elems<V>::E (&db)[Elems<V>::N], int at,
                                           int bt, bool va, bool vb, int G, float *part)
{
    float fa[V], fb[V];
    if constexpr (V == 1) {
        fa[0] = da[0];
        fb[0] = db[0];
    } else {
#pragma unroll
        for (int e = 0; e < Elems<V>::N; ++e) {
            f2_split(da[e], fa[2 * e], fa[2 * e + 1]);
            f2_split(db[e], fb[2 * e], fb[2 * e + 1]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        for (int x = 16; x >= G; x >>= 1) {
            fa[e] += __shfl_xor_sync(kFull, fa[e], x);
            fb[e] += __shfl_xor_sync(kFull, fb[e], x);
        }
        if (int(threadIdx.x & 31) < G) {
            if (va) part[at + e] = fa[e];
            if (vb) part[bt + e] = fb[e];
        }
    }
}

// The block's dgamma partial [2][D]: its warps' in ascending order, per tensor.
// owner[k]: the tensor of warp k, -1 if it had no work; part: rows of `pitch`.
__device__ __forceinline__ void block_dgamma(const int *owner, const float *part, int pitch, int D,
                                             float *out)
{
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        const int which = i >= D, d = which ? i - D : i;
        float v = 0.f;
        for (int k = 0; k < kQkWarps; ++k)
            if (owner[k] == which) v += part[k * pitch + d];
        out[i] = v;
    }
}

// k_qk_ring.cu: the backward's 16-byte form on long inputs; *blocks rows of
// dgamma partials (part NULL: none).
template <class T>
cudaError_t qk_ring_bwd(const QkArgs &a, float *part, int *blocks, cudaStream_t s);

// Blocks of a launch: as many as stay resident, `per_sm` on each SM.
constexpr int qk_blocks(int per_sm) { return kSplitSms * per_sm; }
constexpr int kQkBwdMaxBlocks = qk_blocks(2);  // rows of partials in the workspace
// log2 of the lanes of a head: K units of two chunks of V elements each.
inline int qk_lanes(int D, int V, int K)
{
    const int units = (D + 2 * V - 1) / (2 * V);
    int lg = 0;
    while (lg < 5 && (K << lg) < units) ++lg;
    return lg;
}
QkGeom qk_geom(const QkArgs &a, int V, int K, int hpi, int max_blocks, int *blocks);

}  // namespace mhc
