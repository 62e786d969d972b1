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
// of 2; V = 1 takes anything (V = 4 was no faster than V = 2).  A lane of a head
// has K units (V = 8: one).  The order of a head's sums is fixed by V, D and R:
// it depends neither on the grid nor on T.
//
// What bounds it: HBM on long inputs, once the instructions are few enough for
// 24 warps an SM to keep it busy: packed fp32 pairs, gamma folded into cos and
// sin once a token, no predicates where a head fills its lanes (FLG).
#include "launch.h"
#include "qk.cuh"

namespace mhc {

namespace {

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

// MINB: blocks per SM that the registers must leave room for.  ALL: every unit is
// rotated (R = D).
template <class T, int V, int K, int HPI, bool INTER, int MINB, int FLG, bool ALL>
__global__ void __launch_bounds__(kQkWarps * 32, MINB)
    k_qk_fwd(const __grid_constant__ QkArgs A, const __grid_constant__ QkGeom ge)
{
    typedef typename Elems<V>::E E;
    constexpr int N = Elems<V>::N;
    extern __shared__ __align__(16) float sg[];
    pdl_wait();
    stage_gammas(A, sg);
    Work w;
    if (!my_work(ge, w)) return;
    const QkTensor &m = A.m[w.which];
    const float *gam = sg + (w.which ? gamma_row(A.D) : 0);
    const int lane = threadIdx.x & 31, G = FLG >= 0 ? 1 << FLG : 1 << ge.lg, l = lane & (G - 1);
    const int ng = 32 / G, h0 = w.set * (ng * HPI) + (lane >> ge.lg);
    const int half = A.R / 2, hr = half / V;
    const float inv_d = 1.f / float(A.D);
    int at[K], bt[K];
    bool va[K], vb[K];
#pragma unroll
    for (int q = 0; q < K; ++q) {
        unit_at<V>(l + q * G, hr, half, A.interleaved != 0, at[q], bt[q]);
        va[q] = FLG >= 0 || at[q] < A.D;
        vb[q] = FLG >= 0 || bt[q] < A.D;
    }
    // this token's rows; a head past the last one reads the last (its result is
    // dropped)
    const T *xrow = static_cast<const T *>(m.x) + w.t * m.x_t;
    T *orow = static_cast<T *>(m.out) + w.t * m.out_t + h0 * m.out_h;
    const int64_t x_step = ge.t_step * m.x_t, o_step = ge.t_step * m.out_t;
    int64_t xh[HPI];
#pragma unroll
    for (int i = 0; i < HPI; ++i) xh[i] = min(h0 + i * ng, m.H - 1) * m.x_h;
    for (int64_t t = w.t; t < A.T; t += ge.t_step, xrow += x_step, orow += o_step) {
        Vec<T, V> xa[HPI][K], xb[HPI][K];
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            const T *row = xrow + xh[i];
#pragma unroll
            for (int q = 0; q < K; ++q) {
                if (va[q]) ld_vec(xa[i][q], row + at[q]); else zero_vec(xa[i][q]);
                if (vb[q]) ld_vec(xb[i][q], row + bt[q]); else zero_vec(xb[i][q]);
            }
        }
        int64_t p;
        if (!position(A, t, p)) {
            zero_token<T, V, K, HPI>(m, t, h0, ng, at, bt, va, vb);
            continue;
        }
        UnitFwd<V, INTER> f[K];
#pragma unroll
        for (int q = 0; q < K; ++q) {
            E ga[N], gb[N];
            gamma_e<V>(gam + (va[q] ? at[q] : 0), ga);
            gamma_e<V>(gam + (vb[q] ? bt[q] : 0), gb);
            if (ALL || l + q * G < hr) {
                Rope<V, INTER> r;
                r.load(A.cs, A.sn, p * half + V * (l + q * G));
                f[q].fold(ga, gb, r);
            } else {
                f[q].still(ga, gb);
            }
        }
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            E a[K][N], b[K][N], ss;
            e_set(ss, 0.f);
#pragma unroll
            for (int q = 0; q < K; ++q) {
                widen_e<T, V>(xa[i][q], a[q]);
                widen_e<T, V>(xb[i][q], b[q]);
                add_squares<V>(a[q], b[q], ss);
            }
            E rho;
            e_set(rho, inv_rms(group_sum<FLG>(e_sum(ss), G), inv_d, A.eps));
            if (h0 + i * ng >= m.H) continue;
            T *row = orow + i * ng * m.out_h;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                E ya[N], yb[N];
                f[q].apply(a[q], b[q], rho, ALL || l + q * G < hr, ya, yb);
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
        const T *xrow = static_cast<const T *>(m.x) + w.t * m.x_t;
        const T *urow = static_cast<const T *>(m.up) + w.t * m.up_t;
        T *orow = static_cast<T *>(m.out) + w.t * m.out_t + h0 * m.out_h;
        const int64_t x_step = ge.t_step * m.x_t, u_step = ge.t_step * m.up_t;
        const int64_t o_step = ge.t_step * m.out_t;
        int64_t xh[HPI], uh[HPI];
#pragma unroll
        for (int i = 0; i < HPI; ++i) {
            const int h = min(h0 + i * ng, m.H - 1);
            xh[i] = h * m.x_h;
            uh[i] = h * m.up_h;
        }
        for (int64_t t = w.t; t < A.T;
             t += ge.t_step, xrow += x_step, urow += u_step, orow += o_step) {
            Vec<T, V> xa[HPI][K], xb[HPI][K], ya[HPI][K], yb[HPI][K];
#pragma unroll
            for (int i = 0; i < HPI; ++i) {
                const T *row = xrow + xh[i], *up = urow + uh[i];
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    if (va[q]) ld_vec(xa[i][q], row + at[q]); else zero_vec(xa[i][q]);
                    if (vb[q]) ld_vec(xb[i][q], row + bt[q]); else zero_vec(xb[i][q]);
                    if (va[q]) ld_vec(ya[i][q], up + at[q]); else zero_vec(ya[i][q]);
                    if (vb[q]) ld_vec(yb[i][q], up + bt[q]); else zero_vec(yb[i][q]);
                }
            }
            int64_t p;
            if (!position(A, t, p)) {
                zero_token<T, V, K, HPI>(m, t, h0, ng, at, bt, va, vb);
                continue;
            }
            Rope<V, INTER> r[K];
#pragma unroll
            for (int q = 0; q < K; ++q)
                if (l + q * G < hr) r[q].load(A.cs, A.sn, p * half + V * (l + q * G));
#pragma unroll
            for (int i = 0; i < HPI; ++i) {
                E s1, s2;  // sum x^2, sum g x
                e_set(s1, 0.f);
                e_set(s2, 0.f);
                UnitBwd<V, INTER> n[K];
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    widen_e<T, V>(xa[i][q], n[q].a);
                    widen_e<T, V>(xb[i][q], n[q].b);
                    widen_e<T, V>(ya[i][q], n[q].u);
                    widen_e<T, V>(yb[i][q], n[q].v);
                    if (l + q * G < hr) n[q].turn_back(r[q]);
                    E ga[N], gb[N];
                    gamma_e<V>(gam + (va[q] ? at[q] : 0), ga);
                    gamma_e<V>(gam + (vb[q] ? bt[q] : 0), gb);
                    n[q].sums(ga, gb, s1, s2);
                }
                const float rho = inv_rms(group_sum(e_sum(s1), G), inv_d, A.eps);
                const float k2 = group_sum(e_sum(s2), G) * rho * inv_d;  // mean of g xh
                if (h0 + i * ng >= m.H) continue;
                E rr, nk;
                e_set(rr, rho);
                e_set(nk, -k2);
                T *row = orow + i * ng * m.out_h;
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    E o1[N], o2[N];
                    n[q].grads(rr, nk, o1, o2, da[q], db[q]);
                    Vec<T, V> o;
                    narrow_e<T, V>(o1, o);
                    if (va[q]) st_vec(row + at[q], o);
                    narrow_e<T, V>(o2, o);
                    if (vb[q]) st_vec(row + bt[q], o);
                }
            }
        }
        if (dgp)
#pragma unroll
            for (int q = 0; q < K; ++q)
                put_dgamma<V>(da[q], db[q], at[q], bt[q], va[q], vb[q], G, part + warp * A.D);
    }
    if (!dgp) return;
    __syncthreads();
    block_dgamma(owner, part, A.D, A.D, dgp + int64_t(blockIdx.x) * 2 * A.D);
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

// Elements of a chunk: the widest form whose rules the call meets.  Nothing
// here goes by T (the token strides count as given, for one token too).
int qk_vec(const QkArgs &a, int es)
{
    for (int v : {8, 2}) {
        const int bytes = v * es < 16 ? v * es : 16;
        if (a.D % v == 0 && (a.R / 2) % v == 0 && a.bits % bytes == 0) return v;
    }
    return 1;
}

// Enough warps to fill the SMs even with one head (per lane group) a warp?
bool qk_many(const QkArgs &a) { return a.T * (a.m[0].H + a.m[1].H) >= int64_t(kSplitSms) * 64; }

bool wants_dgamma(const QkArgs &a) { return a.m[0].dgamma || a.m[1].dgamma; }

cudaError_t sum_dgamma(const QkArgs &a, const float *part, int blocks, cudaStream_t s)
{
    MHC_PROF("k_qk_dgamma", s);
    return launch_k(k_qk_dgamma, dim3(unsigned((2 * a.D + 7) / 8)), dim3(1024), 0, s, part, blocks,
                    a.D, a.m[0].dgamma, a.m[1].dgamma);
}

template <class T, int V, int K, int HPI, int MINB, int FLG = -1, bool ALL = false>
cudaError_t run_fwd(const QkArgs &a, cudaStream_t s)
{
    int blocks;
    const QkGeom g = qk_geom(a, V, K, HPI, qk_blocks(MINB), &blocks);
    const size_t smem = size_t(2) * ((a.D + 7) & ~7) * sizeof(float);
    auto kernel = V > 1 && a.interleaved ? k_qk_fwd<T, V, K, HPI, (V > 1), MINB, FLG, ALL>
                                         : k_qk_fwd<T, V, K, HPI, false, MINB, FLG, ALL>;
    MHC_PROF("k_qk_fwd", s);
    return launch_k(kernel, dim3(unsigned(blocks)), dim3(kQkWarps * 32), smem, s, a, g);
}

template <class T, int V, int K, int HPI, int MINB>
cudaError_t run_bwd(const QkArgs &a, float *ws, cudaStream_t s)
{
    static_assert(qk_blocks(MINB) <= kQkBwdMaxBlocks, "the workspace has a row per block");
    int blocks;
    const QkGeom g = qk_geom(a, V, K, HPI, qk_blocks(MINB), &blocks);
    float *part = wants_dgamma(a) ? ws : nullptr;
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
    return sum_dgamma(a, part, blocks, s);
}

// Heads per lane group and blocks per SM of the 16-byte form on long inputs.
// 16384 tokens of 32 + 8 heads of 128, bf16: 2, 3 take 53.6 us (95% of the
// measured copy bandwidth); 4, 2 55.8; 2, 2 61.4; 1, 3 61.6; 1, 4 (spills) 71.3.
constexpr int kFwdHeads = 2, kFwdPerSm = 3;
// Of the forms with shorter vectors, whose heads take three or four units a
// lane.  2999 tokens of 20 + 20 heads of 80, 20 of them rotated, fp16: 2, 3
// take 12.9 us; 1, 4 13.5; 1, 3 16.7; 2, 2 17.0 (one unit a lane, a whole warp
// a head: 19.8).
constexpr int kNarrowHeads = 2, kNarrowPerSm = 3;

// Whether one head per lane group holds all heads of q and of k (then two would
// only work on heads that are not there).
bool qk_few(const QkArgs &a, int V, int K)
{
    const int ng = 32 >> qk_lanes(a.D, V, K);
    return a.m[0].H <= ng && a.m[1].H <= ng;
}

template <class T>
cudaError_t fwd_of(const QkArgs &a, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        if (!qk_many(a) || qk_few(a, 8, 1)) return run_fwd<T, 8, 1, 1, 3>(a, s);
        if constexpr (sizeof(T) == 2) {
            constexpr int h = kFwdHeads, b = kFwdPerSm;
            const bool all = a.R == a.D;
            switch (a.D) {
            case 64: return all ? run_fwd<T, 8, 1, h, b, 2, true>(a, s) : run_fwd<T, 8, 1, h, b, 2>(a, s);
            case 128: return all ? run_fwd<T, 8, 1, h, b, 3, true>(a, s) : run_fwd<T, 8, 1, h, b, 3>(a, s);
            case 256: return all ? run_fwd<T, 8, 1, h, b, 4, true>(a, s) : run_fwd<T, 8, 1, h, b, 4>(a, s);
            }
        }
        return run_fwd<T, 8, 1, kFwdHeads, kFwdPerSm>(a, s);
    case 2:
        if (a.D <= 64)
            return qk_few(a, 2, 2) ? run_fwd<T, 2, 2, 1, kNarrowPerSm>(a, s)
                                   : run_fwd<T, 2, 2, kNarrowHeads, kNarrowPerSm>(a, s);
        if (a.D <= 96)
            return qk_few(a, 2, 3) ? run_fwd<T, 2, 3, 1, kNarrowPerSm>(a, s)
                                   : run_fwd<T, 2, 3, kNarrowHeads, kNarrowPerSm>(a, s);
        return run_fwd<T, 2, 4, 1, 3>(a, s);
    default:
        return a.D <= 128 ? run_fwd<T, 1, 4, 1, 3>(a, s) : run_fwd<T, 1, 8, 1, 2>(a, s);
    }
}

template <class T>
cudaError_t bwd_of(const QkArgs &a, float *ws, cudaStream_t s)
{
    switch (qk_vec(a, int(sizeof(T)))) {
    case 8:
        if (qk_many(a)) {
            int blocks = 0;
            float *part = wants_dgamma(a) ? ws : nullptr;
            const cudaError_t e = qk_ring_bwd<T>(a, part, &blocks, s);
            return e != cudaSuccess || !part ? e : sum_dgamma(a, part, blocks, s);
        }
        return run_bwd<T, 8, 1, 1, 2>(a, ws, s);
    case 2:
        if (a.D <= 64) return run_bwd<T, 2, 2, 1, 2>(a, ws, s);
        return a.D <= 96 ? run_bwd<T, 2, 3, 1, 2>(a, ws, s) : run_bwd<T, 2, 4, 1, 2>(a, ws, s);
    default:
        return a.D <= 128 ? run_bwd<T, 1, 4, 1, 2>(a, ws, s) : run_bwd<T, 1, 8, 1, 1>(a, ws, s);
    }
}

}  // namespace

QkGeom qk_geom(const QkArgs &a, int V, int K, int hpi, int max_blocks, int *blocks)
{
    QkGeom g;
    g.lg = qk_lanes(a.D, V, K);
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
