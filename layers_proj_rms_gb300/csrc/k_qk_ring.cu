// Backward of q/k norm + rotation on long inputs, 16-byte vectors (the
// definitions and the lanes' units are those of k_qk.cu, and so are the bits of
// every result but dgamma's order of sums).
//
// Two tensors in, one out and dgamma's sums do not leave the registers that
// k_qk.cu needs to have enough bytes on their way (81% of the copy bandwidth).
// Here a warp keeps one tensor and one set of heads and walks over tokens.  Its
// inputs come through a ring of S slots in shared memory that is its own: one
// lane asks for a token's heads, upstream heads and table rows by bulk copies,
// S - 1 tokens ahead, and an mbarrier per slot tells when they are there.  What
// is in flight costs no registers and no instructions of the other lanes, and
// no warp waits for another.  The heads of a set are worked on one after the
// other (a loop, not unrolled), so the registers are those of one head.
#include "qk.cuh"
#include "tc.cuh"

namespace mhc {

namespace {

using tc::smem_u32;

// Heads per lane group, slots of a ring and blocks per SM.  16384 tokens of
// 32 + 8 heads of 128, bf16: 2, 3, 2 take 81.7 us (92% of the measured copy
// bandwidth); 2, 2, 2 83.0; 4, 2, 1 92.7; 1, 3, 3 (half the bytes a copy) 195.
constexpr int kHeads = 2, kSlots = 3, kPerSm = 2;

struct RingGeom {
    QkGeom w;
    int slot;  // bytes of a slot
};

// A warp's life: which heads, where its ring is, and the copies into it.
// FLG >= 0: a head is exactly 2^FLG lanes' units; ALL: and R = D.
template <class T, int HPI, int FLG, bool ALL, int S>
struct Ring {
    const QkArgs &A;
    const QkTensor &m;
    int lane, G, l, ng, h0, nh, half, hr, at, bt, slot;
    bool va, vb;
    char *base;
    uint64_t *bar;

    __device__ __forceinline__ Ring(const QkArgs &A_, const RingGeom &ge, const Work &w, char *base_,
                                    uint64_t *bar_)
        : A(A_), m(A_.m[w.which]), slot(ge.slot), base(base_), bar(bar_)
    {
        lane = threadIdx.x & 31;
        G = FLG >= 0 ? 1 << FLG : 1 << ge.w.lg;
        l = lane & (G - 1);
        ng = 32 / G;
        h0 = w.set * ng * HPI;            // the set's first head
        nh = min(ng * HPI, m.H - h0);     // and how many there are
        half = A.R / 2;
        hr = half / 8;
        unit_at<8>(l, hr, half, A.interleaved != 0, at, bt);
        va = FLG >= 0 || at < A.D;
        vb = FLG >= 0 || bt < A.D;
        if (lane == 0) {
            for (int i = 0; i < S; ++i) tc::mbar_init(bar + i, 1);
            tc::fence_barrier_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool turned() const { return ALL || l < hr; }
    __device__ __forceinline__ bool known(int p) const { return A.R == 0 || (p >= 0 && p < A.P); }
    // the position of token t (past the last one: any); P is below 2^31 when
    // there are positions, and T <= P when there are none
    __device__ __forceinline__ int pos(int64_t t) const
    {
        return t >= A.T ? 0 : A.pos ? __ldg(A.pos + t) : int(t);
    }
    // Bytes of the set's heads of one tensor, and where tensor n lies in a slot.
    __device__ __forceinline__ uint32_t heads_bytes() const { return uint32_t(nh * A.D * int(sizeof(T))); }
    __device__ __forceinline__ char *heads(int s, int n) const
    {
        return base + s * slot + n * ng * HPI * A.D * int(sizeof(T));
    }
    __device__ __forceinline__ char *table(int s, int n) const { return heads(s, 2) + n * half * 4; }

    // Asks for token t (position p) into slot s, whose reads every lane has
    // finished (and made known to the copies by release()).
    __device__ __forceinline__ void fetch(int64_t t, int p, int s) const
    {
        const bool rope = A.R > 0 && known(p);
        if (lane == 0)
            tc::mbar_arrive_expect_tx(bar + s, 2 * heads_bytes() + (rope ? uint32_t(half) * 8 : 0));
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int64_t st = n ? m.up_t : m.x_t, sh = n ? m.up_h : m.x_h;
            const T *row = static_cast<const T *>(n ? m.up : m.x) + t * st + h0 * sh;
            if (sh == A.D) {
                if (lane == n) tc::bulk_load(heads(s, n), row, heads_bytes(), bar + s);
            } else {
                for (int h = lane; h < nh; h += 32)
                    tc::bulk_load(heads(s, n) + h * A.D * int(sizeof(T)), row + h * sh,
                                  uint32_t(A.D * int(sizeof(T))), bar + s);
            }
        }
        if (rope && lane >= 2 && lane < 4)
            tc::bulk_load(table(s, lane - 2), (lane == 2 ? A.cs : A.sn) + int64_t(p) * half,
                          uint32_t(half) * 4, bar + s);
    }
    __device__ __forceinline__ void release() const
    {
        // as tc::mbar_release: every lane's reads before the next copy's writes
        asm volatile("fence.proxy.async.shared::cta;\nfence.acq_rel.cta;" ::: "memory");
        __syncwarp();
    }
    __device__ __forceinline__ void chunk(const char *head, int at_, bool on, Vec<T, 8> &v) const
    {
        if (!on) {
            zero_vec(v);
            return;
        }
        const uint32_t p = smem_u32(head) + uint32_t(at_ * int(sizeof(T)));
#pragma unroll
        for (int i = 0; i < Vec<T, 8>::kWords / 4; ++i) {
            const uint4 u = lds128(p + 16 * i);
            v.w[4 * i] = u.x; v.w[4 * i + 1] = u.y; v.w[4 * i + 2] = u.z; v.w[4 * i + 3] = u.w;
        }
    }
    template <bool INTER>
    __device__ __forceinline__ void rope(int s, Rope<8, INTER> &r) const
    {
        float c[8], sn[8];
        load_f<8, true>(reinterpret_cast<const float *>(table(s, 0)) + 8 * l, c);
        load_f<8, true>(reinterpret_cast<const float *>(table(s, 1)) + 8 * l, sn);
        r.set(c, sn);
    }
    // A token whose position is outside the table: zeros, and a fault.
    __device__ __forceinline__ void refuse(T *orow) const
    {
        if (lane == 0) report_fault(A.fault, kFaultPosition);
        Vec<T, 8> z;
        zero_vec(z);
        for (int h = lane / G; h < nh; h += ng) {
            if (va) st_vec(orow + h * m.out_h + at, z);
            if (vb) st_vec(orow + h * m.out_h + bt, z);
        }
    }
    // work(slot, output rows of the set's heads) for each of the warp's tokens
    template <class F>
    __device__ __forceinline__ void walk(int64_t t, int64_t step, F &&work) const
    {
        int p[S + 1];  // positions of this token and the next ones
#pragma unroll
        for (int i = 0; i <= S; ++i) p[i] = pos(t + i * step);
#pragma unroll
        for (int i = 0; i < S - 1; ++i)
            if (t + i * step < A.T) fetch(t + i * step, p[i], i);
        T *orow = static_cast<T *>(m.out) + t * m.out_t + h0 * m.out_h;
        const int64_t o_step = step * m.out_t;
        int s = 0;
        uint32_t parity = 0;
        for (; t < A.T; t += step, orow += o_step) {
            const int64_t ahead = t + (S - 1) * step;
            if (ahead < A.T) fetch(ahead, p[S - 1], s == 0 ? S - 1 : s - 1);
            const int next = pos(t + (S + 1) * step);
            if (!__all_sync(kFull, tc::mbar_wait(bar + s, parity, A.fault, tc::kFaultTimeoutFull))) {
                // give up, but not before the copies on their way (waited for
                // as long again)
                for (int i = 0; i < S && t + i * step < A.T; ++i) {
                    const int k = (s + i) % S;
                    tc::mbar_wait(bar + k, k < s ? parity ^ 1 : parity, A.fault,
                                  tc::kFaultTimeoutFull);
                }
                return;
            }
            if (known(p[0]))
                work(s, orow);
            else
                refuse(orow);
            release();
#pragma unroll
            for (int i = 0; i < S; ++i) p[i] = p[i + 1];
            p[S] = next;
            if (++s == S) {
                s = 0;
                parity ^= 1;
            }
        }
    }
};

// dgp: [gridDim.x][2][D] partial sums of dgamma, one row per block.
template <class T, int HPI, bool INTER, int FLG, bool ALL, int S, int MINB>
__global__ void __launch_bounds__(kQkWarps * 32, MINB)
    k_qk_ring_bwd(const __grid_constant__ QkArgs A, const __grid_constant__ RingGeom ge,
                  float *__restrict__ dgp)
{
    typedef Elems<8>::E E;
    constexpr int N = Elems<8>::N;
    extern __shared__ __align__(128) float sm[];  // gammas, then the warps' rings
    __shared__ uint64_t bar[kQkWarps][S];
    __shared__ int owner[kQkWarps];
    pdl_wait();
    stage_gammas(A, sm);
    Work w;
    const bool active = my_work(ge.w, w);
    const int warp = threadIdx.x >> 5;
    char *rings = reinterpret_cast<char *>(sm + 2 * gamma_row(A.D));
    if ((threadIdx.x & 31) == 0) owner[warp] = active ? w.which : -1;
    if (active) {
        const Ring<T, HPI, FLG, ALL, S> r(A, ge, w, rings + warp * S * ge.slot, bar[warp]);
        const float *gam = sm + (w.which ? gamma_row(A.D) : 0);
        const float inv_d = 1.f / float(A.D);
        const int64_t out_h = r.m.out_h;
        E da[N], db[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            e_set(da[e], 0.f);
            e_set(db[e], 0.f);
        }
        r.walk(w.t, ge.w.t_step, [&](int s, T *orow) {
            Rope<8, INTER> rope;
            if (r.turned()) r.rope(s, rope);
            const int row = A.D * int(sizeof(T));
            const int up = int(r.heads(s, 1) - r.heads(s, 0));
            const char *head = r.heads(s, 0) + (r.lane / r.G) * row;
            T *out = orow + (r.lane / r.G) * out_h;
#pragma unroll 1
            for (int h = r.lane / r.G; h - r.lane / r.G < r.nh; h += r.ng, head += r.ng * row, out += r.ng * out_h) {
                UnitBwd<8, INTER> n;
                Vec<T, 8> x;
                r.chunk(head, r.at, r.va, x);
                widen_e<T, 8>(x, n.a);
                r.chunk(head, r.bt, r.vb, x);
                widen_e<T, 8>(x, n.b);
                r.chunk(head + up, r.at, r.va, x);
                widen_e<T, 8>(x, n.u);
                r.chunk(head + up, r.bt, r.vb, x);
                widen_e<T, 8>(x, n.v);
                if (r.turned()) n.turn_back(rope);
                E ga[N], gb[N], s1, s2;
                gamma_e<8>(gam + (r.va ? r.at : 0), ga);
                gamma_e<8>(gam + (r.vb ? r.bt : 0), gb);
                e_set(s1, 0.f);
                e_set(s2, 0.f);
                n.sums(ga, gb, s1, s2);
                const float rho = inv_rms(group_sum<FLG>(e_sum(s1), r.G), inv_d, A.eps);
                const float k2 = group_sum<FLG>(e_sum(s2), r.G) * rho * inv_d;  // mean of g xh
                if (h < r.nh) {
                    E rr, nk, o1[N], o2[N];
                    e_set(rr, rho);
                    e_set(nk, -k2);
                    n.grads(rr, nk, o1, o2, da, db);
                    narrow_e<T, 8>(o1, x);
                    if (r.va) st_vec(out + r.at, x);
                    narrow_e<T, 8>(o2, x);
                    if (r.vb) st_vec(out + r.bt, x);
                }
            }
        });
        // the ring's copies have all been waited for: its first slot takes the
        // warp's dgamma
        if (dgp)
            put_dgamma<8>(da, db, r.at, r.bt, r.va, r.vb, r.G, reinterpret_cast<float *>(r.base));
    }
    if (!dgp) return;
    __syncthreads();
    block_dgamma(owner, reinterpret_cast<const float *>(rings), S * ge.slot / 4, A.D,
                 dgp + int64_t(blockIdx.x) * 2 * A.D);
}

// Bytes of a slot: the set's heads of x and of the upstream gradient, a row of
// cos and of sin, and a share of the room for a warp's dgamma.  At most
// 512 * 4 * 2 + 2048 bytes (heads of 512), so eight rings of three fit an SM.
int slot_bytes(const QkArgs &a, int es, int lg, int hpi, int slots)
{
    const int b = (32 >> lg) * hpi * a.D * es * 2 + a.R * 4;
    const int d = (a.D * 4 + slots - 1) / slots;
    return ((b > d ? b : d) + 127) / 128 * 128;
}

size_t ring_smem(const QkArgs &a, int slot, int slots)
{
    return size_t(2) * ((a.D + 7) & ~7) * sizeof(float) + size_t(kQkWarps) * slots * slot;
}

template <class T, int HPI, int S, int MINB, int FLG = -1, bool ALL = false>
cudaError_t run_bwd(const QkArgs &a, float *part, int *blocks, cudaStream_t s)
{
    static_assert(qk_blocks(MINB) <= kQkBwdMaxBlocks, "the workspace has a row per block");
    RingGeom g;
    g.w = qk_geom(a, 8, 1, HPI, qk_blocks(MINB), blocks);
    g.slot = slot_bytes(a, sizeof(T), g.w.lg, HPI, S);
    const size_t smem = ring_smem(a, g.slot, S);
    auto kernel = a.interleaved ? k_qk_ring_bwd<T, HPI, true, FLG, ALL, S, MINB>
                                : k_qk_ring_bwd<T, HPI, false, FLG, ALL, S, MINB>;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), int(smem));
    if (e != cudaSuccess) return e;
    MHC_PROF("k_qk_ring_bwd", s);
    return launch_k(kernel, dim3(unsigned(*blocks)), dim3(kQkWarps * 32), smem, s, a, g, part);
}

}  // namespace

template <class T>
cudaError_t qk_ring_bwd(const QkArgs &a, float *part, int *blocks, cudaStream_t s)
{
    constexpr int heads = sizeof(T) == 4 ? kHeads / 2 : kHeads;  // as many bytes
    if constexpr (sizeof(T) == 2) {
        constexpr int h = heads, n = kSlots, b = kPerSm;
        const bool all = a.R == a.D;
        switch (a.D) {
        case 64:
            return all ? run_bwd<T, h, n, b, 2, true>(a, part, blocks, s)
                       : run_bwd<T, h, n, b, 2>(a, part, blocks, s);
        case 128:
            return all ? run_bwd<T, h, n, b, 3, true>(a, part, blocks, s)
                       : run_bwd<T, h, n, b, 3>(a, part, blocks, s);
        case 256:
            return all ? run_bwd<T, h, n, b, 4, true>(a, part, blocks, s)
                       : run_bwd<T, h, n, b, 4>(a, part, blocks, s);
        }
    }
    return run_bwd<T, heads, kSlots, kPerSm>(a, part, blocks, s);
}

template cudaError_t qk_ring_bwd<bf16>(const QkArgs &, float *, int *, cudaStream_t);
template cudaError_t qk_ring_bwd<fp16>(const QkArgs &, float *, int *, cudaStream_t);
template cudaError_t qk_ring_bwd<float>(const QkArgs &, float *, int *, cudaStream_t);

}  // namespace mhc
