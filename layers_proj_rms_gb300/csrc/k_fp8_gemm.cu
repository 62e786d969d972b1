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
// registers, so scales of any value are exact to fp32 and the long sum is
// rounded to nearest, once a block.
//
// A CTA is persistent, one an SM: a TMA producer, the MMA issuer, a warp that
// brings the scales (cp.async, as deep as the tiles' ring), a spare warp and
// eight epilogue warps, each 32 rows x half the columns.
#include <cuda_fp16.h>

#include <algorithm>

#include "elem.cuh"
#include "fp8.h"
#include "launch.h"
#include "tc.cuh"
#include "tmap.h"

namespace mhc {

namespace {

constexpr int BM = 128, BK = 128;

// Fault codes of bad offsets in device memory.
enum : int { kFaultOffsets = 205, kFaultOffsetsAlign = 206 };

template <int BN_>
struct GemmCfg {
    static constexpr int BN = BN_;
    static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK, STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr int SC = 5;  // blocks whose scales are in flight
    static constexpr int SC_FLOATS = BM + BN;
    static constexpr int EPI_WARPS = 8;
    static constexpr int HALF = BN / 2;  // columns of an epilogue warp
    static constexpr int OUT_BYTES = EPI_WARPS * 32 * 64;
    static constexpr int THREADS = 32 * (4 + EPI_WARPS);
    static constexpr int TMEM_COLS = 2 * BN;
    // shared memory: stages, output staging, scales, segments' starts and first tiles, barriers
    static constexpr int OFF_OUT = STAGES * STAGE;
    static constexpr int OFF_SC = OFF_OUT + OUT_BYTES;
    static constexpr int OFF_SEG = OFF_SC + SC * SC_FLOATS * 4;
    static constexpr int OFF_TILE = OFF_SEG + 1040 * 4;
    static constexpr int OFF_BAR = OFF_TILE + 1040 * 4;
    static constexpr int SMEM = OFF_BAR + 512 + 1024 /*align*/;
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

// Instruction descriptor of kind::f8f6f4, K-major A and B in 8 bits (0 e4m3,
// 1 e5m2), fp32 accumulator, shape M x N.
constexpr uint32_t idesc_f8_f32(int fa, int fb, int M, int N)
{
    return (1u << 4) | (uint32_t(fa) << 7) | (uint32_t(fb) << 10) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

// Arrives on `bar` when this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(bar))
                 : "memory");
}

// 32 consecutive TMEM columns, as 16 pairs.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t taddr, f32x2 (&v)[16])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = f2_make(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
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

template <class P, bool W, class O>
__global__ void __launch_bounds__(P::THREADS, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
               const GemmP p)
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
    uint64_t *sc_full = empty + P::STAGES;
    uint64_t *sc_empty = sc_full + P::SC;
    uint64_t *acc_full = sc_empty + P::SC;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *done = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < P::STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < P::SC; ++s) {
            tc::mbar_init(&sc_full[s], 32);
            tc::mbar_init(&sc_empty[s], P::EPI_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&acc_full[b], 1);
            tc::mbar_init(&acc_empty[b], P::EPI_WARPS);
        }
        tc::mbar_init(done, 1);
        *abort_flag = 0;
        tc::fence_barrier_init();
        tc::tma_prefetch_desc(&tma);
        tc::tma_prefetch_desc(&tmb);
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
    // rows before the first segment belong to none
    const int row_first = seg[0], row_last = seg[p.G];

    // Registers go from the four issuing warps to the epilogue, which holds the
    // sums: 128 * 56 + 256 * 224 = 384 * 168, what the block was launched with.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (int t = blockIdx.x; t < ntiles && !*abort_flag; t += gridDim.x) {
                const Tile x = tile_of<P, W>(p, seg, first, t);
                for (int kb = 0; kb < x.nkb; ++kb, ++i) {
                    const int s = i % P::STAGES;
                    if (*abort_flag ||
                        (i >= P::STAGES && !tc::mbar_wait(&empty[s], ((i / P::STAGES) & 1) ^ 1,
                                                          p.fault, tc::kFaultTimeoutEmpty))) {
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t *st = smem + s * P::STAGE;
                    const int k = (x.kb0 + kb) * BK;
                    tc::mbar_arrive_expect_tx(&full[s], P::STAGE);
                    tc::tma_load_2d(st, &tma, k, x.row0, &full[s]);
                    if (W)
                        tc::tma_load_2d(st + P::A_BYTES, &tmb, k, x.n0, &full[s]);
                    else
                        tc::tma_load_3d(st + P::A_BYTES, &tmb, k, x.n0, x.e, &full[s]);
                }
            }
            // do not leave while copies into this CTA's shared memory are in flight
            for (int j = max(0, i - P::STAGES); j < i; ++j)
                tc::mbar_wait(&full[j % P::STAGES], (j / P::STAGES) & 1, p.fault,
                              tc::kFaultTimeoutMisc);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int i = 0;
            for (int t = blockIdx.x; t < ntiles && !*abort_flag; t += gridDim.x) {
                const Tile x = tile_of<P, W>(p, seg, first, t);
                for (int kb = 0; kb < x.nkb; ++kb, ++i) {
                    const int s = i % P::STAGES, b = i & 1;
                    if (*abort_flag ||
                        !tc::mbar_wait(&full[s], (i / P::STAGES) & 1, p.fault,
                                       tc::kFaultTimeoutFull) ||
                        (i >= 2 && !tc::mbar_wait(&acc_empty[b], ((i >> 1) & 1) ^ 1, p.fault,
                                                  tc::kFaultTimeoutAcc))) {
                        *abort_flag = 1;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t a = tc::smem_u32(smem + s * P::STAGE);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        mma_f8(tmem + b * P::BN, tc::desc_kmajor_sw128(a + kk * 32),
                               tc::desc_kmajor_sw128(a + P::A_BYTES + kk * 32), p.idesc, kk > 0);
                    tc::mma_commit(&empty[s]);
                    tc::mma_commit(&acc_full[b]);
                }
            }
            // the MMAs in flight end before TMEM and shared memory go
            tc::mma_commit(done);
            tc::mbar_wait(done, 0, p.fault, tc::kFaultTimeoutMisc);
        }
        __syncwarp();
    } else if (warp == 2) {
        int i = 0;
        for (int t = blockIdx.x; t < ntiles && !*abort_flag; t += gridDim.x) {
            const Tile x = tile_of<P, W>(p, seg, first, t);
            for (int kb = 0; kb < x.nkb; ++kb, ++i) {
                const int s = i % P::SC;
                if (*abort_flag || (i >= P::SC && !tc::mbar_wait(&sc_empty[s], ((i / P::SC) & 1) ^ 1,
                                                                 p.fault, tc::kFaultTimeoutEmpty))) {
                    *abort_flag = 1;
                    break;
                }
                const uint32_t dst = tc::smem_u32(scales + s * P::SC_FLOATS);
                const int64_t blk = x.kb0 + kb;
                const float *ra = p.sa + blk * p.out_rows + x.row0;
#pragma unroll
                for (int j = 0; j < BM / 32; ++j) {
                    const int r = j * 32 + lane;
                    const bool in = x.row0 + r < x.row_end;
                    tc::cp_async4(dst + r * 4, in ? ra + r : p.sa, in ? 4 : 0);
                }
                if (W) {
                    const float *cb = p.sb + blk * p.N + x.n0;
#pragma unroll
                    for (int j = 0; j < P::BN / 32; ++j) {
                        const int c = j * 32 + lane;
                        const bool in = x.n0 + c < p.N;
                        tc::cp_async4(dst + (BM + c) * 4, in ? cb + c : p.sb, in ? 4 : 0);
                    }
                } else if (lane < (P::BN + 127) / 128) {
                    const int nbs = int((p.N + 127) / 128), nb = x.n0 / 128 + lane;
                    const bool in = nb < nbs;
                    const float *cb = p.sb + (int64_t(x.e) * p.nkb + kb) * nbs + nb;
                    tc::cp_async4(dst + (BM + lane) * 4, in ? cb : p.sb, in ? 4 : 0);
                }
                cp_async_arrive(&sc_full[s]);
            }
        }
        tc::cp_async_wait_all();
        __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t trow = tmem + (uint32_t(q * 32) << 16) + h * P::HALF;
        const uint32_t stage_out = tc::smem_u32(smem + P::OFF_OUT + (warp - 4) * 2048);
        O *out = static_cast<O *>(p.out);
        int i = 0;
        for (int t = blockIdx.x; t < ntiles; t += gridDim.x) {
            const Tile x = tile_of<P, W>(p, seg, first, t);
            f32x2 acc[P::HALF / 2];
#pragma unroll
            for (int j = 0; j < P::HALF / 2; ++j) acc[j] = 0;
            bool ok = true;
            for (int kb = 0; kb < x.nkb; ++kb, ++i) {
                const int s = i % P::SC, b = i & 1;
                if (*abort_flag ||
                    !tc::mbar_wait(&sc_full[s], (i / P::SC) & 1, p.fault, tc::kFaultTimeoutFull) ||
                    !tc::mbar_wait(&acc_full[b], (i >> 1) & 1, p.fault, tc::kFaultTimeoutAcc)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                tc::tc_fence_after();
                const uint32_t sc = tc::smem_u32(scales + s * P::SC_FLOATS);
                float r = lds32f(sc + (q * 32 + lane) * 4);
                if (!W) r *= lds32f(sc + (BM + h * P::HALF / 128) * 4);
                const f32x2 r2 = f2_make(r, r);
#pragma unroll
                for (int c = 0; c < P::HALF / 32; ++c) {
                    f32x2 d[16];
                    tmem_ld32_wait(trow + b * P::BN + c * 32, d);
                    if (W) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint4 v = lds128(sc + (BM + h * P::HALF + c * 32 + j * 4) * 4);
                            const f32x2 s0 = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
                            const f32x2 s1 = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
                            acc[c * 16 + 2 * j] =
                                f2_fma(d[2 * j], f2_mul(r2, s0), acc[c * 16 + 2 * j]);
                            acc[c * 16 + 2 * j + 1] =
                                f2_fma(d[2 * j + 1], f2_mul(r2, s1), acc[c * 16 + 2 * j + 1]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[c * 16 + j] = f2_fma(d[j], r2, acc[c * 16 + j]);
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&acc_empty[b]);
                    tc::mbar_arrive(&sc_empty[s]);
                }
            }
            if (!ok) break;
            // rounded once, through shared memory in pieces of 64 bytes a row:
            // whole sectors leave (a row a lane would write 16 bytes of each)
            constexpr int VN = 16 / int(sizeof(O)), CH = 4 * VN;
            const int64_t row_base = W ? int64_t(x.e) * p.out_rows : 0;
#pragma unroll
            for (int c = 0; c < P::HALF / CH; ++c) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float f[VN];
#pragma unroll
                    for (int j = 0; j < VN / 2; ++j)
                        f2_split(acc[(c * CH + v * VN) / 2 + j], f[2 * j], f[2 * j + 1]);
                    Vec<O, VN> o;
                    narrow<O, VN>(f, o);
                    const uint32_t at = stage_out + lane * 64 + ((v ^ ((lane >> 1) & 3)) * 16);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(o.w[0]),
                                 "r"(o.w[1]), "r"(o.w[2]), "r"(o.w[3])
                                 : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = j * 8 + (lane >> 2), v = lane & 3;
                    const uint4 u = lds128(stage_out + r * 64 + ((v ^ ((r >> 1) & 3)) * 16));
                    const int row = x.row0 + q * 32 + r;
                    const int64_t col = x.n0 + h * P::HALF + c * CH + v * VN;
                    if (row < x.row_end && col < p.N)
                        st_stream(out + (row_base + row) * p.N + col, u);
                }
                __syncwarp();
            }
        }
        // the rows of no segment
        if (!W && !*abort_flag) {
            const int64_t n0 = int64_t(row_first) * p.N, n1 = int64_t(row_last) * p.N;
            constexpr int VN = 16 / int(sizeof(O));
            const int64_t all = (int64_t(p.R) * p.N - n1 + n0) / VN;
            const int64_t step = int64_t(gridDim.x) * (32 * P::EPI_WARPS);
            for (int64_t v = int64_t(blockIdx.x) * (32 * P::EPI_WARPS) + threadIdx.x - 128; v < all;
                 v += step) {
                const int64_t el = v * VN < n0 ? v * VN : v * VN - n0 + n1;
                st_stream(out + el, make_uint4(0, 0, 0, 0));
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, P::TMEM_COLS);
}

template <class P, bool W, class O>
cudaError_t run(const CUtensorMap &ta, const CUtensorMap &tb, const GemmP &p, int64_t tiles,
                cudaStream_t s)
{
    auto *kernel = k_fp8_gemm<P, W, O>;
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), P::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t sms = num_sms();
    MHC_PROF(W ? "k_fp8_wgrad" : "k_fp8_gemm", s);
    return launch_k(kernel, dim3(unsigned(std::min(sms, std::max<int64_t>(tiles, 1)))),
                    dim3(P::THREADS), P::SMEM, s, ta, tb, p);
}

template <class P, bool W>
cudaError_t by_type(const CUtensorMap &ta, const CUtensorMap &tb, const GemmP &p, int64_t tiles,
                    int out_dtype, cudaStream_t s)
{
    if (out_dtype == 0) return run<P, W, bf16>(ta, tb, p, tiles, s);
    if (out_dtype == 1) return run<P, W, fp16>(ta, tb, p, tiles, s);
    return run<P, W, float>(ta, tb, p, tiles, s);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs &a, int out_dtype, cudaStream_t s)
{
    typedef GemmCfg<256> P;
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
    CUtensorMap ta, tb;
    const uint64_t da[2] = {uint64_t(a.K), uint64_t(a.R)}, ra[1] = {uint64_t(a.K)};
    const uint64_t db[3] = {uint64_t(a.K), uint64_t(a.N), uint64_t(a.G)};
    const uint64_t rb[2] = {uint64_t(a.K), uint64_t(a.K) * uint64_t(a.N)};
    const uint32_t ba[2] = {BK, BM}, bb[3] = {BK, P::BN, 1};
    if (!tmap_u8(&ta, a.a, 2, da, ra, ba) || !tmap_u8(&tb, a.b, 3, db, rb, bb))
        return cudaErrorInvalidValue;
    // a bound on the tiles: every segment may end inside one
    const int64_t tiles = (a.R / BM + std::min(a.G, a.R)) * p.nt;
    return by_type<P, false>(ta, tb, p, tiles, out_dtype, s);
}

cudaError_t launch_fp8_wgrad(const Fp8WgradArgs &a, int out_dtype, cudaStream_t s)
{
    typedef GemmCfg<256> P;
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
    CUtensorMap ta, tb;
    const uint64_t da[2] = {uint64_t(a.R), uint64_t(a.M)}, db[2] = {uint64_t(a.R), uint64_t(a.N)};
    const uint64_t r[1] = {uint64_t(a.R)};
    const uint32_t ba[2] = {BK, BM}, bb[2] = {BK, P::BN};
    if (!tmap_u8(&ta, a.a, 2, da, r, ba) || !tmap_u8(&tb, a.b, 2, db, r, bb))
        return cudaErrorInvalidValue;
    return by_type<P, true>(ta, tb, p, a.G * p.mt * p.nt, out_dtype, s);
}

}  // namespace mhc
