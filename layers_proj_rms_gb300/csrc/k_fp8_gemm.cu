// Products of 8-bit floating-point matrices whose scales are given for blocks
// of 128 along the reduced dimension, grouped by experts:
//
//   rows:     out[r][n] = sum_kb sa[kb][r] sb[e][kb][n/128] P_kb[r][n],
//             P_kb[r][n] = sum_{k in block kb} a[r][k] b[e][n][k],
//             e the expert whose segment of the sorted rows holds r;
//   weights:  out[e][m][n] = sum_rb sa[rb][m] sb[rb][n] P_rb[m][n], the sum
//             over the blocks of 128 rows of expert e's segment (both operands
//             stored along the rows).
//
// P_kb is a tensor-core product (tcgen05.mma kind::f8f6f4, products exact,
// fp32 sums) into one of two TMEM accumulators; while the tensor cores work on
// the next block, the epilogue warps read it back, scale it and add it to fp32
// registers; the long sum is rounded to nearest, once a block.  Of the rows the
// two scales are one factor, or two one after the other where that factor would
// be no normal number (a row of zeros has the least scale: 7001 rows of 61 experts in
// segments of 16, e5m2, then take 137.5 us, not 135).  Of the weights P is multiplied by
// sa, then by sb, which neither overflows nor loses bits between for sa in [2^-94, 2^88]
// (a look at each block's scales there costs 7%: 838 us of 781).
//
// What bounds it: an MMA of 128 x 256 x 32 reads 12 KB of shared memory and its
// TMA loads write as much, 855 cycles a block of 128 where the products are 512; the
// epilogue's instructions run beside that (in pairs of fp32: 968 us of 1008, for
// weights 777 of 930; figures here are of runs of 20 calls: held at work for seconds the
// GPU is at its power limit, 1355 W and 1770 MHz of 2070, and 970 us are 1062).  Tiles
// of 128 x 256 move 1.5 times the products per byte of 128 x 128 (65536 rows of 64
// experts, K 4096, 4096 columns: 968 us of 1221) and are taken where enough of them
// fill the SMs; the rule and its measurements stand at wide_sooner().  Two CTAs that
// share a tile of 256 x 256, each with half of B (cta_group::2, 32 KB in and out for
// the same products), were 1037 us of 978, 787 of 783 for weights: the waits across
// the pair take more than the feed gains, so there are no pairs.
//
// A CTA is persistent, one an SM: a warp that brings the operands (TMA), two that
// issue the MMAs of the even and the odd blocks, one that brings the scales
// (cp.async) and waits for the products, and eight epilogue warps, with 256 columns
// sixteen, each 32 rows x 64 columns.  (The scales by the operands' warp: 1089 us
// of 1081, 963 of 926 with weights; its own loop is what feeds the MMAs.)  Results
// leave through a 4 KB box of shared memory a warp (32 rows x 128 bytes) by TMA
// store, so the next tile's blocks do not wait for them; a box that the segment's
// end cuts is copied row by row.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

namespace mhc {

namespace {

constexpr int BM = 128, BK = 128;

// Fault codes of bad offsets in device memory.
enum : int { kFaultOffsets = 205, kFaultOffsetsAlign = 206 };

// Tiles of 128 x BN.
template <int BN_>
struct GemmCfg {
    static constexpr int BN = BN_;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 128 ? 5 : 3;
    static constexpr bool SPLIT = BN == 256;  // registers go to the epilogue
    static constexpr int SC = 6;     // blocks whose scales are there or in flight
    static constexpr int AHEAD = 4;  // of them in flight at most; two are being read
    static constexpr int SC_FLOATS = BM + BN;
    static constexpr int COLS = 64;  // of an epilogue warp
    static constexpr int GROUPS = BN / COLS;  // of four epilogue warps
    static constexpr int EPI_WARPS = 4 * GROUPS;
    static constexpr int BOX = 32 * 128;
    static constexpr int THREADS = 32 * (4 + EPI_WARPS);
    static constexpr int TMEM_COLS = 2 * BN;
    // shared memory: stages, output boxes, scales, segments' starts and first tiles, barriers
    static constexpr int OFF_OUT = STAGES * STAGE;
    static constexpr int OFF_SC = OFF_OUT + EPI_WARPS * BOX;
    static constexpr int OFF_SEG = OFF_SC + SC * SC_FLOATS * 4;
    static constexpr int OFF_TILE = OFF_SEG + 1040 * 4;
    static constexpr int OFF_BAR = OFF_TILE + 1040 * 4;
    static constexpr int SMEM = OFF_BAR + 256 + 1024 /*align*/;
    static_assert(SMEM <= 232448, "shared memory");
};

struct GemmP {
    const float *sa, *sb;
    const int32_t *offsets;
    int64_t out_rows;    // rows: R; weights: M
    int64_t N;
    int G, R;            // segments, sorted rows
    int nkb;             // rows: blocks of K
    int mt, nt;          // tiles of M (weights) and N
    uint32_t idesc;
    void *out;
    int *fault;
};

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Named barriers: block i's products are there (a group of epilogue warps and the
// warp that waits for them), block i's accumulator is read (all epilogue warps and
// the MMA warp); i even or odd.
__device__ __forceinline__ int bar_ready(int group, int b) { return 1 + 2 * group + b; }
__device__ __forceinline__ int bar_read(int b) { return 9 + b; }
__device__ __forceinline__ void bar_arrive(int id, int count)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// TMA loads by shared-memory addresses
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *m, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z,
                                        uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void store_2d(const CUtensorMap *m, uint32_t src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap *m, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
// Instruction descriptor of kind::f8f6f4, K-major A and B in 8 bits (0 e4m3,
// 1 e5m2), fp32 accumulator, shape M x N.
constexpr uint32_t idesc_f8_f32(int fa, int fb, int M, int N)
{
    return (1u << 4) | (uint32_t(fa) << 7) | (uint32_t(fb) << 10) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

// 16 consecutive TMEM columns.  The registers hold them once tmem_wait() is
// through; what uses them also uses a value that passes through that wait, so it
// cannot be moved before it.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(taddr));
}
// 16 TMEM lanes x 16 columns as fragments: v[4 j + 2 i + c] is lane 8 i + lane / 4,
// column 8 j + 2 (lane % 4) + c.
__device__ __forceinline__ void tmem_ld16x16(uint32_t taddr, float (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
// a += v s, for pairs
__device__ __forceinline__ void fma_pair(float *a, f32x2 v, f32x2 s)
{
    f2_split(f2_fma(v, s, f2_make(a[0], a[1])), a[0], a[1]);
}
__device__ __forceinline__ void tmem_wait(float &through)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(through)::"memory");
}
__device__ __forceinline__ void tmem_wait(float &through, float &too)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(through), "+f"(too)::"memory");
}

// One output tile: where its operands and results stand.
struct Tile {
    int e;         // segment
    int row0;      // rows: first sorted row; weights: first row of M
    int row_end;   // one past the last row that is stored
    int n0;
    int kb0, nkb;  // first block of the reduced dimension and their number
};

// Tiles of an expert go down the rows first, in groups of 16 row tiles: the
// CTAs that run at one time then share both operands' tiles in L2.
template <class P, bool W>
__device__ __forceinline__ Tile tile_of(const GemmP &p, const int *seg, const int *first, int t)
{
    Tile x;
    int local, mt;
    if (W) {
        mt = p.mt;
        x.e = t / (mt * p.nt);
        local = t - x.e * mt * p.nt;
    } else {
        int lo = 0, hi = p.G;  // the last e with first[e] * nt <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] * p.nt <= t)
                lo = mid;
            else
                hi = mid;
        }
        x.e = lo;
        local = t - first[lo] * p.nt;
        mt = first[lo + 1] - first[lo];
    }
    const int g = local / (16 * p.nt), rem = local - g * 16 * p.nt;
    const int ms = min(16, mt - 16 * g);
    const int m = 16 * g + rem % ms;
    x.n0 = rem / ms * P::BN;
    if (W) {
        x.row0 = m * BM;
        x.row_end = int(p.out_rows);
        x.kb0 = seg[x.e] / BK;
        x.nkb = (seg[x.e + 1] - seg[x.e] + BK - 1) / BK;
    } else {
        x.row0 = seg[x.e] + m * BM;
        x.row_end = seg[x.e + 1];
        x.kb0 = 0;
        x.nkb = p.nkb;
    }
    return x;
}

// Its number of blocks alone.
template <bool W>
__device__ __forceinline__ int blocks_of(const GemmP &p, const int *seg, int t)
{
    if (!W) return p.nkb;
    const int e = t / (p.mt * p.nt);
    return (seg[e + 1] - seg[e] + BK - 1) / BK;
}

// The scales of a CTA's blocks, one block after the other, by a warp: a lane's
// pointers and what of them is inside, stepped from block to block.
template <class P, bool W>
struct Cursor {
    static constexpr int NC = W ? P::BN / 128 : 1;  // copies of column scales
    const float *row, *col;  // the lane's first row scale, its first column scale
    int64_t row_step, col_step;
    uint32_t in;   // bits 0-3: rows j*32 + lane; 4: all rows, 16 bytes a lane; 8..: columns
    int t, tstep, ntiles, left;  // tile; blocks of it that are left, 0 at the end

    __device__ __forceinline__ Cursor(const GemmP &p, const int *seg, const int *first, int t0,
                                      int step, int nt, int lane)
        : row(nullptr), col(nullptr), row_step(0), col_step(0), in(0), t(t0 - step), tstep(step),
          ntiles(nt), left(1)
    {
        next(p, seg, first, lane);
    }
    __device__ __forceinline__ void next(const GemmP &p, const int *seg, const int *first, int lane)
    {
        row += row_step;
        col += col_step;
        if (--left) return;
        do {
            t += tstep;
            if (t >= ntiles) return;
            const Tile x = tile_of<P, W>(p, seg, first, t);
            left = x.nkb;
            const int64_t r0 = int64_t(x.kb0) * p.out_rows + x.row0;
            // all 128 rows by 16 bytes a lane, where they and the step are so aligned
            const bool wide = x.row0 + BM <= x.row_end && ((r0 | p.out_rows) & 3) == 0;
            in = wide ? 16u : 0u;
#pragma unroll
            for (int j = 0; j < BM / 32; ++j)
                if (x.row0 + j * 32 + lane < x.row_end) in |= 1u << j;
            row = p.sa + r0 + (wide ? 4 * lane : lane);
            row_step = p.out_rows;
            if (W) {
                // N is a multiple of 8: four columns are in or out together
                col = p.sb + int64_t(x.kb0) * p.N + x.n0 + 4 * lane;
                col_step = p.N;
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (x.n0 + j * 128 + 4 * lane < p.N) in |= 256u << j;
            } else {
                const int nbs = int((p.N + 127) / 128), nb = x.n0 / 128 + lane;
                col = p.sb + int64_t(x.e) * p.nkb * nbs + nb;
                col_step = nbs;
                if (lane < P::BN / 128 && nb < nbs) in |= 256u;
            }
        } while (left == 0);
    }
    // brings the block's scales to dst (BM row scales, then the columns'); one group
    __device__ __forceinline__ void load(const GemmP &p, uint32_t dst) const
    {
        const int lane = threadIdx.x & 31;
        if (in & 16u) {
            tc::cp_async16(dst + lane * 16, row, 16);
        } else {
#pragma unroll
            for (int j = 0; j < BM / 32; ++j)
                tc::cp_async4(dst + (j * 32 + lane) * 4, in >> j & 1 ? row + j * 32 : p.sa,
                              in >> j & 1 ? 4 : 0);
        }
        if (W) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const bool on = in >> (8 + j) & 1;
                tc::cp_async16(dst + (BM + j * 128 + 4 * lane) * 4, on ? col + j * 128 : p.sb, on ? 16 : 0);
            }
        } else if (lane < P::BN / 128) {
            tc::cp_async4(dst + (BM + lane) * 4, in & 256u ? col : p.sb, in & 256u ? 4 : 0);
        }
        tc::cp_async_commit();
    }
};

template <class P, bool W, class O>
__global__ void __launch_bounds__(P::THREADS, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
               const __grid_constant__ CUtensorMap tmo, const GemmP p)
{
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(smem + P::OFF_SC);
    int *seg = reinterpret_cast<int *>(smem + P::OFF_SEG);
    int *first = reinterpret_cast<int *>(smem + P::OFF_TILE);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + P::OFF_BAR);
    uint64_t *empty = full + P::STAGES;
    uint64_t *acc_full = empty + P::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *collected = abort_flag + 1;  // [2] even, odd blocks: one past the last one read

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < P::STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) tc::mbar_init(&acc_full[b], 1);
        *abort_flag = 0;
        collected[0] = collected[1] = 0;
        tc::fence_barrier_init();
        tc::tma_prefetch_desc(&tma);
        tc::tma_prefetch_desc(&tmb);
        tc::tma_prefetch_desc(&tmo);
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, P::TMEM_COLS);
    // The segments: offsets that go back, leave the rows or (weights) stand off
    // the blocks are moved to the nearest that do not, and reported.
    for (int e = threadIdx.x; e <= p.G; e += P::THREADS)
        seg[e] = p.offsets ? __ldg(p.offsets + e) : (e ? p.R : 0);
    __syncthreads();
    if (warp == 0) {
        int carry = 0, base = 0;
        for (int e0 = 0; e0 <= p.G; e0 += 32) {
            const int e = e0 + lane;
            const int raw = e <= p.G ? seg[e] : 0;
            int v = min(max(raw, 0), p.R);
            if (W && v % BK && v != p.R) v -= v % BK;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kFull, v, d);
                if (lane >= d) v = max(v, o);
            }
            v = max(v, carry);
            if (e <= p.G) {
                seg[e] = v;
                if (v != raw && blockIdx.x == 0)
                    report_fault(p.fault, W && raw >= 0 && raw <= p.R && raw % BK ? kFaultOffsetsAlign
                                                                                 : kFaultOffsets);
            }
            // row tiles of segment e - 1 before v
            int prev = __shfl_up_sync(kFull, v, 1);
            if (lane == 0) prev = e0 == 0 ? v : carry;
            int n = e <= p.G && e > 0 ? (v - prev + BM - 1) / BM : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(kFull, n, d);
                if (lane >= d) n += o;
            }
            n += base;
            if (e <= p.G) first[e] = n;
            base = __shfl_sync(kFull, n, 31);
            carry = __shfl_sync(kFull, v, 31);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = W ? p.G * p.mt * p.nt : first[p.G] * p.nt;
    const int t0 = blockIdx.x, tstep = gridDim.x;

    // With 256 columns registers go from the four issuing warps to the epilogue, which
    // holds the sums: 128 * 64 + 512 * 104 = 640 * 96, what the block was launched with.
    if (warp < 4) {
        if constexpr (P::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // These loops run beside the epilogue's warps, at five cycles and more an
        // instruction: a hundred instructions a block would be the products' time, so
        // what changes from block to block is stepped, not computed.
        if (warp == 0) {
            if (lane == 0) {
                int st = 0, left = 0;  // stage; loads that nothing has waited for
                uint32_t ph = 1;       // a barrier's phase before its first counts as complete
                const uint32_t smem0 = tc::smem_u32(smem), bar0 = tc::smem_u32(full);
                bool ok = true;
                for (int t = t0; t < ntiles && ok; t += tstep) {
                    const Tile x = tile_of<P, W>(p, seg, first, t);
                    int k = x.kb0 * BK;
                    for (int kb = 0; kb < x.nkb; ++kb, k += BK) {
                        ok = tc::mbar_wait(&empty[st], ph, p.fault, tc::kFaultTimeoutEmpty);
                        if (!ok) break;
                        const uint32_t a = smem0 + st * P::STAGE, bar = bar0 + st * 8;
                        tc::mbar_arrive_expect_tx(&full[st], P::STAGE);
                        load_2d(a, &tma, k, x.row0, bar);
                        if (W)
                            load_2d(a + P::A_BYTES, &tmb, k, x.n0, bar);
                        else
                            load_3d(a + P::A_BYTES, &tmb, k, x.n0, x.e, bar);
                        left = min(left + 1, P::STAGES);
                        if (++st == P::STAGES) {
                            st = 0;
                            ph ^= 1;
                        }
                    }
                }
                // Do not leave while copies into this CTA's shared memory, MMAs that read it or
                // their arrivals are in flight: what was issued is consumed.  After a fault that
                // does not come; the copies then get the time that they may take.
                for (; left > 0 && ok; --left) {
                    // the oldest of the loads left: `left` stages back
                    const int o = st - left;
                    ok = tc::mbar_wait(&empty[o < 0 ? o + P::STAGES : o], o < 0 ? ph : ph ^ 1, p.fault,
                                       tc::kFaultTimeoutMisc);
                }
                if (!ok) {
                    *abort_flag = 1;
                    const long long c0 = clock64();
                    while (clock64() - c0 < 1000000) {
                    }
                }
            }
            __syncwarp();
        } else if (warp != 2) {
            // Two warps issue the MMAs of the even and the odd blocks, each with its accumulator:
            // while one's run the other goes through its waits, 100 cycles and more each beside
            // the tensor cores' own traffic (one warp alone spent 640 of 1420 cycles a block
            // on them).  After a fault they only keep the barriers going.
            const int b = warp >> 1;
            const uint64_t da0 = tc::desc_kmajor_sw128(tc::smem_u32(smem));
            const uint64_t db0 = tc::desc_kmajor_sw128(tc::smem_u32(smem) + P::A_BYTES);
            const uint32_t d0 = tmem + b * P::BN;
            int st = b, done = 0;       // stage; blocks of this warp so far
            int gone = 0;               // those that are read
            uint32_t ph = 0;            // phase of the stage's barrier
            bool ok = true;
            auto collect = [&]() {  // this warp's oldest block: accumulator and scales are read
                tc::named_bar_sync(bar_read(b), 32 * (P::EPI_WARPS + 1));
                if (lane == 0) collected[b] = ++gone;
            };
            int par = b;  // the first block of the next tile that is this warp's
            for (int t = t0; t < ntiles; t += tstep) {
                const int nkb = blocks_of<W>(p, seg, t);
                int kb = par;
                for (; kb < nkb; kb += 2, ++done) {
                    if (done) collect();
                    if (lane == 0 && ok) {
                        ok = tc::mbar_wait(&full[st], ph, p.fault, tc::kFaultTimeoutFull);
                        if (!ok) *abort_flag = 1;
                    }
                    if (lane == 0 && ok) {
                        tc::tc_fence_after();
                        const uint64_t da = da0 + st * (P::STAGE >> 4), db = db0 + st * (P::STAGE >> 4);
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            mma_f8(d0, da + 2 * kk, db + 2 * kk, p.idesc, kk > 0);
                        tc::mma_commit(&empty[st]);
                        tc::mma_commit(&acc_full[b]);
                    }
                    st += 2;
                    if (st >= P::STAGES) {
                        st -= P::STAGES;
                        ph ^= 1;
                    }
                    __syncwarp();
                }
                par = kb - nkb;
            }
            if (done) collect();
        } else {
            // Brings each block's scales, AHEAD blocks before they are read, and waits for the
            // products and the scales for the epilogue: one warp at the barriers in shared
            // memory, which the tensor cores keep busy, not sixteen.
            Cursor<P, W> c(p, seg, first, t0, tstep, ntiles, lane);
            const uint32_t ring = tc::smem_u32(scales);
            uint32_t slot = 0;
            int ahead = 0;  // blocks whose scales are brought and not yet passed on
            int i = 0;
            bool ok = true;
            for (;;) {
                while (ahead < P::AHEAD && c.left) {
                    c.load(p, ring + slot);
                    slot = slot == (P::SC - 1) * P::SC_FLOATS * 4 ? 0 : slot + P::SC_FLOATS * 4;
                    ++ahead;
                    c.next(p, seg, first, lane);
                }
                if (ahead == 0) break;
                if (ahead == P::AHEAD)
                    asm volatile("cp.async.wait_group %0;" ::"n"(P::AHEAD - 1) : "memory");
                else
                    tc::cp_async_wait_all();
                const int b = i & 1;
                if (ok && !tc::mbar_wait(&acc_full[b], (i >> 1) & 1, p.fault, tc::kFaultTimeoutAcc)) {
                    ok = false;
                    *abort_flag = 1;
                }
                // after a fault the epilogue runs on, block by block
                for (const long long c0 = clock64();
                     !ok && collected[b] < (i >> 1) && clock64() - c0 < tc::kWaitCycles;) {
                }
                tc::tc_fence_after();
                tc::tc_fence_before();
                __syncwarp();
#pragma unroll
                for (int h = 0; h < P::GROUPS; ++h) bar_arrive(bar_ready(h, b), 160);
                ++i;
                --ahead;
            }
        }
    } else {
        if constexpr (P::SPLIT) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int q = warp & 3, h = (warp - 4) >> 2;
        const int g = lane >> 2, tig = lane & 3;
        const uint32_t trow = tmem + (uint32_t(q * 32) << 16) + h * P::COLS;
        const uint32_t box = tc::smem_u32(smem + P::OFF_OUT + (warp - 4) * P::BOX);
        O *out = static_cast<O *>(p.out);
        const uint32_t sc0 = tc::smem_u32(scales);
        uint32_t slot = 0;
        int b = 0;
        for (int t = t0; t < ntiles; t += tstep) {
            const Tile x = tile_of<P, W>(p, seg, first, t);
            // rows: acc[c], row q*32 + lane, column c;  weights: acc[8 n + v], fragment v
            // (tmem_ld16x16) of rows 16 (n % 2), columns 16 (n / 2)
            float acc[P::COLS];
#pragma unroll
            for (int j = 0; j < P::COLS; ++j) acc[j] = 0.f;
            for (int kb = 0; kb < x.nkb; ++kb, b ^= 1) {
                tc::named_bar_sync(bar_ready(h, b), 160);
                tc::tc_fence_after();
                const uint32_t sc = sc0 + slot;
                slot = slot == (P::SC - 1) * P::SC_FLOATS * 4 ? 0 : slot + P::SC_FLOATS * 4;
                float r[4];          // weights: of the lane's rows; rows: what d is multiplied by
                bool apart = false;  // rows: by r[1] before, somewhere in the warp
                float d[W ? 8 : 16];
                if constexpr (!W) tmem_ld16(trow + b * P::BN, d);
                if (W) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[j] = lds32f(sc + (q * 32 + 8 * j + g) * 4);
                } else {
                    const float ra = lds32f(sc + (q * 32 + lane) * 4);
                    const float rb = lds32f(sc + (BM + h * P::COLS / 128) * 4);
                    r[0] = ra * rb;
                    r[1] = 1.f;
                    const bool mine = f8_apart(ra, rb);
                    apart = __any_sync(kFull, mine);
                    if (mine) {
                        r[0] = fabsf(ra) > fabsf(rb) ? rb : ra;
                        r[1] = fabsf(ra) > fabsf(rb) ? ra : rb;
                    }
                }
                const uint32_t d0 = trow + b * P::BN;
                // the accumulator goes back as soon as its last columns are in registers
                auto release = [&]() {
                    tc::tc_fence_before();
                    bar_arrive(bar_read(b), 32 * (P::EPI_WARPS + 1));
                };
                if constexpr (W) {
                    constexpr int NL = P::COLS / 8;  // loads of 16 lanes x 16 columns
                    f32x2 c[2];
#pragma unroll
                    for (int n = 0; n < NL; ++n) {
                        if (n % 2 == 0) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const uint2 u = lds64(
                                    sc + (BM + h * P::COLS + (n / 2) * 16 + 8 * j + 2 * tig) * 4);
                                c[j] = f2_make(__uint_as_float(u.x), __uint_as_float(u.y));
                            }
                        }
                        float &r0 = r[2 * (n & 1)], &r1 = r[2 * (n & 1) + 1];
                        tmem_ld16x16(d0 + (n / 2) * 16 + (uint32_t(n & 1) << 20), d);
                        tmem_wait(r0, r1);
                        if (n + 1 == NL) release();
                        float *ac = acc + 8 * n;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            fma_pair(ac + 4 * j, f2_mul(f2_make(d[4 * j], d[4 * j + 1]), f2_make(r0, r0)), c[j]);
                            fma_pair(ac + 4 * j + 2, f2_mul(f2_make(d[4 * j + 2], d[4 * j + 3]), f2_make(r1, r1)),
                                     c[j]);
                        }
                    }
                } else {
                    auto add = [&](auto twice) {
#pragma unroll
                        for (int c = 0; c < P::COLS / 16; ++c) {
                            if (c) tmem_ld16(d0 + c * 16, d);
                            tmem_wait(r[0]);
                            if (c + 1 == P::COLS / 16) release();
                            if constexpr (decltype(twice)::value) {
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    if constexpr (P::SPLIT) {  // (pairs of registers would be spilled)
                                        d[j] *= r[1];
                                        d[j + 1] *= r[1];
                                    } else {
                                        const f32x2 v = f2_mul(f2_make(d[j], d[j + 1]), f2_make(r[1], r[1]));
                                        f2_split(v, d[j], d[j + 1]);
                                    }
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; j += 2)
                                fma_pair(acc + c * 16 + j, f2_make(d[j], d[j + 1]), f2_make(r[0], r[0]));
                        }
                    };
                    if (apart)
                        add(std::true_type());
                    else
                        add(std::false_type());
                }
            }
            if (*abort_flag) continue;
            // rounded once, 128 bytes of each of the warp's 32 rows at a time
            constexpr int VN = 16 / int(sizeof(O)), CH = 8 * VN;
            const int wrow = x.row0 + q * 32, col0 = x.n0 + h * P::COLS;
            const bool whole = W ? wrow < x.row_end : wrow + 32 <= x.row_end;
            if (wrow >= x.row_end) continue;
#pragma unroll
            for (int c = 0; c < P::COLS / CH; ++c) {
                if (col0 + c * CH >= p.N) break;
                if (lane == 0) tc::bulk_wait_read_all();
                __syncwarp();
                if constexpr (!W) {
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        float f[VN];
#pragma unroll
                        for (int j = 0; j < VN; ++j) f[j] = acc[c * CH + v * VN + j];
                        Vec<O, VN> o;
                        narrow<O, VN>(f, o);
                        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                         box + lane * 128 + ((v ^ (lane & 7)) * 16)),
                                     "r"(o.w[0]), "r"(o.w[1]), "r"(o.w[2]), "r"(o.w[3])
                                     : "memory");
                    }
                } else {
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi)
#pragma unroll
                        for (int jj = 0; jj < CH / 8; ++jj)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int cc = c * CH + 8 * jj;  // columns cc + 2 tig, + 1
                                const float *v = acc + 8 * (2 * (cc / 16) + hi) + 4 * (cc % 16 / 8) + 2 * k;
                                const int row = 16 * hi + 8 * k + g;
                                const int byte = (8 * jj + 2 * tig) * int(sizeof(O));
                                const uint32_t to = box + row * 128 + (((byte >> 4) ^ g) << 4) + (byte & 15);
                                if constexpr (sizeof(O) == 4)
                                    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(to), "f"(v[0]),
                                                 "f"(v[1])
                                                 : "memory");
                                else
                                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(to),
                                                 "r"(round2(v[0], v[1], static_cast<const O *>(nullptr)))
                                                 : "memory");
                            }
                }
                if (whole) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (W)
                            store_3d(&tmo, box, col0 + c * CH, wrow, x.e);
                        else
                            store_2d(&tmo, box, col0 + c * CH, wrow);
                        tc::bulk_commit_group();
                    }
                } else {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = j * 4 + (lane >> 3), v = lane & 7;
                        const uint4 u = lds128(box + r * 128 + ((v ^ (r & 7)) * 16));
                        const int64_t col = col0 + c * CH + v * VN;
                        if (wrow + r < x.row_end && col < p.N)
                            st_stream(out + int64_t(wrow + r) * p.N + col, u);
                    }
                }
            }
        }
        // the rows of no segment
        if (!W && !*abort_flag) {
            const int64_t n0 = int64_t(seg[0]) * p.N, n1 = int64_t(seg[p.G]) * p.N;
            constexpr int VN = 16 / int(sizeof(O));
            const int64_t all = (int64_t(p.R) * p.N - n1 + n0) / VN;
            const int64_t step = int64_t(gridDim.x) * (32 * P::EPI_WARPS);
            for (int64_t v = int64_t(blockIdx.x) * (32 * P::EPI_WARPS) + threadIdx.x - 128; v < all;
                 v += step) {
                const int64_t el = v * VN < n0 ? v * VN : v * VN - n0 + n1;
                st_stream(out + el, make_uint4(0, 0, 0, 0));
            }
        }
        if (lane == 0) tc::bulk_wait_all();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, P::TMEM_COLS);
}

template <class P, bool W, class O>
cudaError_t run(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &to, const GemmP &p,
                int64_t tiles, cudaStream_t s)
{
    auto *kernel = k_fp8_gemm<P, W, O>;
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), P::SMEM);
    if (e != cudaSuccess) return e;
    MHC_PROF(W ? "k_fp8_wgrad" : "k_fp8_gemm", s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(num_sms(), std::max<int64_t>(tiles, 1))));
    cfg.blockDim = dim3(P::THREADS);
    cfg.dynamicSmemBytes = P::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, ta, tb, to, p);
}

template <class P, bool W>
cudaError_t by_type(const CUtensorMap &ta, const CUtensorMap &tb, const CUtensorMap &to,
                    const GemmP &p, int64_t tiles, int out_dtype, cudaStream_t s)
{
    if (out_dtype == 0) return run<P, W, bf16>(ta, tb, to, p, tiles, s);
    if (out_dtype == 1) return run<P, W, fp16>(ta, tb, to, p, tiles, s);
    return run<P, W, float>(ta, tb, to, p, tiles, s);
}

typedef GemmCfg<128> Narrow;
typedef GemmCfg<256> Wide;

template <class P>
cudaError_t gemm_rows(const Fp8GemmArgs &a, int out_dtype, cudaStream_t s)
{
    GemmP p = {};
    p.sa = a.sa;
    p.sb = a.sb;
    p.offsets = a.offsets;
    p.out_rows = a.R;
    p.N = a.N;
    p.G = int(a.G);
    p.R = int(a.R);
    p.nkb = int(fp8_blocks(a.K));
    p.nt = int((a.N + P::BN - 1) / P::BN);
    p.idesc = idesc_f8_f32(a.fa, a.fb, BM, P::BN);
    p.out = a.out;
    p.fault = a.fault;
    CUtensorMap ta, tb, to;
    const uint64_t es = out_dtype == 2 ? 4 : 2;
    const uint64_t da[2] = {uint64_t(a.K), uint64_t(a.R)}, ra[1] = {uint64_t(a.K)};
    const uint64_t db[3] = {uint64_t(a.K), uint64_t(a.N), uint64_t(a.G)};
    const uint64_t rb[2] = {uint64_t(a.K), uint64_t(a.K) * uint64_t(a.N)};
    const uint64_t dn[2] = {uint64_t(a.N), uint64_t(a.R)}, rn[1] = {uint64_t(a.N) * es};
    const uint32_t ba[2] = {BK, BM}, bb[3] = {BK, P::BN, 1}, bo[2] = {uint32_t(128 / es), 32};
    if (!tmap_u8(&ta, a.a, 2, da, ra, ba) || !tmap_u8(&tb, a.b, 3, db, rb, bb) ||
        !tmap_out(&to, a.out, out_dtype, 2, dn, rn, bo))
        return cudaErrorInvalidValue;
    // a bound on the tiles: every segment may end inside one
    const int64_t tiles = (a.R / BM + std::min(a.G, a.R)) * p.nt;
    return by_type<P, false>(ta, tb, to, p, tiles, out_dtype, s);
}

template <class P>
cudaError_t gemm_weights(const Fp8WgradArgs &a, int out_dtype, cudaStream_t s)
{
    GemmP p = {};
    p.sa = a.sa;
    p.sb = a.sb;
    p.offsets = a.offsets;
    p.out_rows = a.M;
    p.N = a.N;
    p.G = int(a.G);
    p.R = int(a.R);
    p.mt = int((a.M + BM - 1) / BM);
    p.nt = int((a.N + P::BN - 1) / P::BN);
    p.idesc = idesc_f8_f32(a.fa, a.fb, BM, P::BN);
    p.out = a.out;
    p.fault = a.fault;
    CUtensorMap ta, tb, to;
    const uint64_t es = out_dtype == 2 ? 4 : 2;
    const uint64_t da[2] = {uint64_t(a.R), uint64_t(a.M)}, db[2] = {uint64_t(a.R), uint64_t(a.N)};
    const uint64_t r[1] = {uint64_t(a.R)};
    const uint64_t dn[3] = {uint64_t(a.N), uint64_t(a.M), uint64_t(a.G)};
    const uint64_t rn[2] = {uint64_t(a.N) * es, uint64_t(a.N) * uint64_t(a.M) * es};
    const uint32_t ba[2] = {BK, BM}, bb[2] = {BK, P::BN}, bo[3] = {uint32_t(128 / es), 32, 1};
    if (!tmap_u8(&ta, a.a, 2, da, r, ba) || !tmap_u8(&tb, a.b, 2, db, r, bb) ||
        !tmap_out(&to, a.out, out_dtype, 3, dn, rn, bo))
        return cudaErrorInvalidValue;
    return by_type<P, true>(ta, tb, to, p, a.G * p.mt * p.nt, out_dtype, s);
}

// Whether tiles of 128 x 256 are done sooner, from the numbers of row tiles and
// columns: by rounds of one tile an SM, where a narrow tile takes 0.64 of a wide
// one's time (65536 rows of 64 experts, 4096 x 4096: 1221 us of 968; 65536 rows of 8,
// K 2048, 384 columns: 70 of 69; one segment of 512 rows, 2816 columns, less than a
// round either way: 14 of 20; weights 1024 x 1024 from 8192 rows, likewise: 27 of 38;
// 61 experts' weights 1000 x 1328: 39.5 of 34.3; 128 columns, half of a wide tile
// empty: 58 of 76).
bool wide_sooner(int64_t row_tiles, int64_t N)
{
    const int64_t sms = num_sms();
    const int64_t narrow = (row_tiles * ((N + 127) / 128) + sms - 1) / sms;
    const int64_t wide = (row_tiles * ((N + 255) / 256) + sms - 1) / sms;
    return 25 * wide <= 16 * narrow;
}

}  // namespace

// Where the weights' way through HBM counts the wide tile's gain is small: with fewer
// than 160 rows a segment it must not leave half of its last tile empty (7001 rows of
// 61 experts, 1328 columns: narrow 134 us, wide 138; 8192 rows of 64, 2816 columns: 168
// and 152; 4096 rows: 136 and 131), and with fewer than 64 narrow tiles, which have more
// stages, are the faster (296 rows of 60: 119 and 121.5).
cudaError_t launch_fp8_gemm(const Fp8GemmArgs &a, int out_dtype, cudaStream_t s)
{
    const bool rows = a.R >= 160 * a.G || (a.R >= 64 * a.G && (a.N + 127) / 128 % 2 == 0);
    const bool wide = rows && wide_sooner(a.R / BM + std::min(a.G, a.R), a.N);
    return wide ? gemm_rows<Wide>(a, out_dtype, s) : gemm_rows<Narrow>(a, out_dtype, s);
}

cudaError_t launch_fp8_wgrad(const Fp8WgradArgs &a, int out_dtype, cudaStream_t s)
{
    return wide_sooner(a.G * ((a.M + BM - 1) / BM), a.N) ? gemm_weights<Wide>(a, out_dtype, s)
                                                        : gemm_weights<Narrow>(a, out_dtype, s);
}

}  // namespace mhc
