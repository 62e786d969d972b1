// The whole experts' layer for a few tokens, in two launches and a short one:
//
//   up:    h[t,j] = silu(W1g[e] x[t]) * (W1u[e] x[t]),  e = ids[t][j]
//   down:  y[t,j] = W2[e] h[t,j]
//   sum:   f[t] = sum_j w[t][j] y[t,j]
//
// Few tokens read far more weights than anything else, so the weights go by once
// and straight into registers: a warp's piece is 128 bytes of 32 weight rows,
// 16 bytes a lane and load, in the order of a tensor-core operand's words (the
// product does not care about the order of k as long as both operands have the
// same), the tokens are the other operand's 8 columns.  mma.sync, not tcgen05:
// there are 8 columns, the tensor cores are far from busy, and operands that stay
// in registers need no trip through shared memory.
//
// Work: (segment, tile) in order of the experts, a segment up to 8 slots of one
// expert (16 at a time took longer wherever it was tried, 308 us for 257 with 16
// slots an expert: the second 8 find the weights in L2, the rows of 16 have no room in L1),
// a tile 32 weight rows (16 of gate and the same 16 of up); a
// block, one an SM, takes a contiguous share of it.  One to 16 warps split a
// tile's k in pieces and join through shared memory in a fixed order (split_of).  The next
// piece is always in flight: 16 warps x 4 KB an SM.
//
// h stands in the workspace in fp32.  16-bit weights: x as it is; h is split where it is
// read into terms of the type: three of bf16, which hold all of its 24 bits, or, of
// fp16, two of the values times a power of two that brings the largest of the 32 that a
// column has in a step to [2^14, 2^15), undone in the fp32 sums: off by 2^-23 of the
// value or 2^-40 of that largest (unscaled terms overflow at 65504 and are
// subnormal below 1e-4).  The splitting, the third term and the sums that each piece has
// for itself take 199 us for 190 at 13 tokens of 60 experts, 4096 x 1408.  8-bit weights:
// x and h are quantised by blocks of 128, as mhc_fp8_quant does, when a segment's rows
// are brought to shared memory; each block's product is scaled into fp32 sums, by a row's
// scale above 2^88 or below 2^-94 with care (f8_scaled).
//
// A slot's row of y is written once and a token's slots are added up in their
// order, so nothing depends on which block did what.  (The last block at a tile of
// columns adding them up, found by counts, took longer: the counts' round trips at
// every tile, and nearly all of the sums in the one block with the last segment.)
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "launch.h"

namespace mhc {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRows = 32;                 // weight rows of a tile
constexpr int TOK = 8;                    // slots of a segment: the tensor cores' columns
constexpr int kPitch = 36;                // floats of a token's partial sums: no bank conflicts
constexpr int kMaxSlots = kMoeFewTokens * 32, kMaxExperts = 1024;
constexpr int kMaxSegments = kMaxExperts + kMaxSlots / TOK;
constexpr int kPiece = 128;               // bytes of k a warp takes at once
enum : int { kFaultExpert = 202 };

struct FewP {
    const void *x;        // [T, C]
    const int32_t *ids;
    const float *w;
    const void *wt;       // weights [E, rows, K]
    const float *s;       // their scales [E, blocks of K, blocks of rows], or NULL
    int64_t K, rows;      // reduced length; weight rows of an expert
    int T, k, E;
    int ntiles;           // tiles of an expert
    int wk;               // warps that split a tile's k
    float *h;             // [T*k, F]
    float *y;             // [T*k, C]
    int64_t F, C;
    int *fault;
};

struct E4m3 { uint8_t v; };

// d = a b + c, c = d or zeros; 16-bit operands of type W
#define MHC_MMA(type)                                                                               \
    if (FIRST)                                                                                      \
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." type ".f32 {%0,%1,%2,%3}, "           \
                     "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"                                   \
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                               \
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));             \
    else                                                                                            \
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." type ".f32 {%0,%1,%2,%3}, "           \
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                                       \
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                               \
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
template <class W, bool FIRST>
__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<W, bf16>::value) {
        MHC_MMA("bf16.bf16");
    } else {
        MHC_MMA("f16.f16");
    }
}
#undef MHC_MMA

// Four e4m3 values as two pairs of fp16, which hold them exactly.  Volatile: kept
// for a second use, the conversions of a piece would take 64 registers.
__device__ __forceinline__ uint2 widen_e4m3(uint32_t w)
{
    uint2 v;
    asm volatile("{\n"
        ".reg .b16 lo, hi;\n"
        "mov.b32 {lo, hi}, %2;\n"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n"
        "}\n"
        : "=r"(v.x), "=r"(v.y)
        : "r"(w));
    return v;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// h in terms of the weights' type: 8 consecutive values v of one of the 8 columns (the four
// lanes of a quad hold 32), whose terms' sum is v times the power of two whose inverse is
// returned.  An infinity is its first term alone (inf - inf would make it a NaN); a step that
// holds one is rare.
constexpr float kLargest = 3.4028235e38f;  // of fp32

__device__ __forceinline__ float largest8(const float (&v)[8])
{
    return fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                 fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
}
__device__ __forceinline__ f32x2 rest2(f32x2 v, float lo, float hi)  // v - (lo, hi)
{
    return f2_fma(f2_make(lo, hi), f2_make(-1.f, -1.f), v);
}
__device__ __forceinline__ float cut16(float v)
{
    return __uint_as_float(__float_as_uint(v) & 0xffff0000u);
}
__device__ __forceinline__ uint32_t tops(float lo, float hi)
{
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
template <bool INFINITE>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[3][4], int i)
{
    // cut, not rounded: what is left is exact and fits
    t[0][i] = tops(x, y);
    f32x2 r = rest2(f2_make(x, y), cut16(x), cut16(y));
    if constexpr (INFINITE) {
        const float a = fabsf(x) > kLargest ? 0.f : x - cut16(x);
        r = f2_make(a, fabsf(y) > kLargest ? 0.f : y - cut16(y));
    }
    f2_split(r, x, y);
    t[1][i] = tops(x, y);
    f2_split(rest2(r, cut16(x), cut16(y)), x, y);
    t[2][i] = tops(x, y);
}
__device__ __forceinline__ float split8(const float (&v)[8], uint32_t (&t)[3][4], const bf16 *)
{
    if (__any_sync(kFull, largest8(v) > kLargest)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) split2<true>(v[2 * i], v[2 * i + 1], t, i);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) split2<false>(v[2 * i], v[2 * i + 1], t, i);
    }
    return 1.f;
}
__device__ __forceinline__ float split8(const float (&v)[8], uint32_t (&t)[2][4], const fp16 *)
{
    const fp16 *type = nullptr;
    float m = largest8(v);
    const bool infinite = __any_sync(kFull, m > kLargest);
    if (infinite) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]) > kLargest ? 0.f : fabsf(v[i]));
    }
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
    const uint32_t e = max(__float_as_uint(m) >> 23, 15u);
    const float up = __uint_as_float((268u - e) << 23);  // 2^(141 - e)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 s = f2_mul(f2_make(v[2 * i], v[2 * i + 1]), f2_make(up, up));
        float x, y, x0, y0;
        f2_split(s, x, y);
        t[0][i] = round2(x, y, type);
        widen2(t[0][i], x0, y0, type);
        f2_split(rest2(s, x0, y0), x, y);
        if (infinite) {
            x = fabsf(x0) > kLargest ? 0.f : x;
            y = fabsf(y0) > kLargest ? 0.f : y;
        }
        t[1][i] = round2(x, y, type);
    }
    return __uint_as_float((e - 14u) << 23);
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// 16 bytes that are read once, or zeros: a predicated load, which nothing waits for
// before its values are used (a choice of values would).
__device__ __forceinline__ uint4 ld_or_zero(const void *p, bool in)
{
    uint4 v;
    asm volatile(
        "{\n"
        ".reg .pred q;\n"
        "setp.ne.b32 q, %5, 0;\n"
        "mov.b32 %0, 0;\n"
        "mov.b32 %1, 0;\n"
        "mov.b32 %2, 0;\n"
        "mov.b32 %3, 0;\n"
        "@q ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
        "}\n"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(int(in)));
    return v;
}

// A warp's piece in flight: for each of two 64-byte steps the 16 bytes of rows
// g, g + 8, g + 16, g + 24 (g = lane / 4), and the scales of the two row groups.
template <bool EIGHT>
struct Piece {
    uint4 a[2][4];
    float s[EIGHT ? 2 : 1];
};

// W: bf16, fp16 or E4m3; X: the activations.
template <class W, class X, bool DOWN>
__global__ void __launch_bounds__(kThreads, 1) k_moe_few(const FewP p)
{
    constexpr bool EIGHT = sizeof(W) == 1;
    extern __shared__ __align__(16) uint8_t smem[];
    // slots in order of their experts, the experts' first slots and first segments, the
    // segments' experts
    uint16_t *slots = reinterpret_cast<uint16_t *>(smem);
    int *first = reinterpret_cast<int *>(smem + kMaxSlots * 2);
    int *fseg = first + kMaxExperts + 4;
    uint16_t *expert = reinterpret_cast<uint16_t *>(fseg + kMaxExperts + 4);
    float *red = reinterpret_cast<float *>(expert + kMaxSegments);  // [2][warps][TOK][kPitch]
    uint8_t *xs = reinterpret_cast<uint8_t *>(red + 2 * kWarps * TOK * kPitch);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int n = p.T * p.k, E = p.E;

    // The next launch's blocks may come as this one's leave (each fills an SM).  down
    // begins with ids and weights: all of up's blocks are past their wait then, so what
    // came before up is done; only h is its work.
    if (!DOWN) pdl_wait();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Every block sorts the slots by their experts, in the same order.  (A thread an expert
    // that looks at all slots, twice: 188 us of 132 with 1024 slots of 64 experts, 2048 x 768.)
    int *ids = reinterpret_cast<int *>(red), *count = ids + kMaxSlots;  // red is not in use yet
    int *sums = count + kMaxExperts;
    for (int e = tid; e < E; e += kThreads) count[e] = 0;
    for (int i = tid; i < n; i += kThreads) {
        int e = __ldg(p.ids + i);
        if (e < -1 || e >= E) {
            if (blockIdx.x == 0 && !DOWN) report_fault(p.fault, kFaultExpert);
            e = -1;
        }
        ids[i] = e;
    }
    __syncthreads();
    if (warp == 0) {  // a slot's place among its expert's, above the id's bits: 32 slots a step
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane, e = i < n ? ids[i] : -1;
            const uint32_t same = __match_any_sync(kFull, e);
            const int before = e >= 0 ? count[e] : 0, at = __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e >= 0) {
                ids[i] = e | (before + at) << 10;
                if (at == 0) count[e] = before + __popc(same);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    {
        // two experts a thread; numbers of slots below, of segments above bit 16
        static_assert(kMaxExperts == 2 * kThreads && kMaxExperts <= 1 << 10, "experts");
        static_assert(kMaxSegments < 1 << 15 && kMaxSlots < 1 << 16, "two numbers in a word");
        const int e = 2 * tid, c0 = e < E ? count[e] : 0, c1 = e + 1 < E ? count[e + 1] : 0;
        const int a0 = c0 | (c0 + TOK - 1) / TOK << 16, a1 = c1 | (c1 + TOK - 1) / TOK << 16;
        int v = a0 + a1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(kFull, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) sums[warp] = v;
        __syncthreads();
        v += int(__reduce_add_sync(kFull, lane < warp ? unsigned(sums[lane]) : 0u)) - a0 - a1;
        for (int j = 0; j < 2; ++j) {
            if (e + j <= E) {
                first[e + j] = v & 0xffff;
                fseg[e + j] = v >> 16;
            }
            const int c = j ? a1 : a0;
            for (int q = 0; q < c >> 16; ++q) expert[(v >> 16) + q] = uint16_t(e + j);
            v += c;
        }
        if (tid == kThreads - 1 && E == kMaxExperts) {
            first[E] = v & 0xffff;
            fseg[E] = v >> 16;
        }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int v = ids[i];
        if (v >= 0) slots[first[v & 1023] + (v >> 10)] = uint16_t(i);
    }
    __syncthreads();
    const int nseg = fseg[E];

    const int WK = p.wk, NG = kWarps / WK;
    const int gi = warp / WK, wk = warp % WK;
    const int gtid = tid - gi * WK * 32, gsize = WK * 32;
    auto group_sync = [&]() {  // the warps of a tile; 8 such groups at most have more than one
        if (WK == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + gi), "r"(gsize) : "memory");
    };
    const int64_t Kb = p.K * int64_t(sizeof(W));  // bytes of a weight row
    const int np = int((Kb + kPiece - 1) / kPiece);
    const int nkb = int((p.K + kFp8Block - 1) / kFp8Block);
    const int nrb = int((p.rows + kFp8Block - 1) / kFp8Block);
    const int xpitch = nkb * kFp8Block + 64;
    float *sx = reinterpret_cast<float *>(xs + (EIGHT ? TOK * xpitch : 0));  // [nkb][TOK]
    const uint8_t *wt = static_cast<const uint8_t *>(p.wt);

    static_assert(kMaxSegments * (kMoeFewMaxK / 16) < 1 << 30, "tiles");
    const int total = nseg * p.ntiles;
    const int t_begin = int(int64_t(total) * blockIdx.x / gridDim.x);
    const int t_end = int(int64_t(total) * (blockIdx.x + 1) / gridDim.x);
    bool waited = !DOWN;
    int parity = 0;

    for (int t0 = t_begin; t0 < t_end;) {
        const int seg = t0 / p.ntiles;
        const int t1 = min(t_end, (seg + 1) * p.ntiles);
        const int e = expert[seg];
        const int s0 = first[e] + (seg - fseg[e]) * TOK;
        const int ns = min(TOK, first[e + 1] - s0);
        const uint8_t *we = wt + int64_t(e) * p.rows * Kb;

        auto row_of = [&](int tile, int m) {  // first weight row of row group m
            return DOWN ? int64_t(tile) * kRows + m * 16 : m * p.F + int64_t(tile) * 16;
        };
        // this warp's pieces: wk, wk + WK, ... of tiles gi, gi + NG, ...; where the next one
        // stands is stepped, as an instruction costs a warp beside 15 others five cycles
        const int tile0 = t0 - seg * p.ntiles, tile1 = t1 - seg * p.ntiles;
        int ltile = tile0 + gi, lpiece = wk;
        const uint8_t *la[2];  // row g of the row groups, this lane's bytes of the piece
        const float *ls[2];    // the row groups' scales of the piece
        const int64_t row8 = 8 * Kb;
        auto seek = [&]() {  // to the first piece of ltile
            lpiece = wk;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                int64_t r = row_of(ltile, m);
                if (DOWN) r = min(r, p.rows - 16);  // a last tile of 16 rows
                la[m] = we + (r + g) * Kb + wk * kPiece + tig * 16;
                if constexpr (EIGHT) ls[m] = p.s + (int64_t(e) * nkb + wk) * nrb + r / kFp8Block;
            }
        };
        auto load = [&](Piece<EIGHT> &b) {  // the next piece
            if ((lpiece + 1) * kPiece <= Kb) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        b.a[st][2 * m] = ld_stream(la[m] + st * 64);
                        b.a[st][2 * m + 1] = ld_stream(la[m] + row8 + st * 64);
                    }
            } else {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const bool in = lpiece * kPiece + tig * 16 + st * 64 < Kb;
                        b.a[st][2 * m] = ld_or_zero(la[m] + st * 64, in);
                        b.a[st][2 * m + 1] = ld_or_zero(la[m] + row8 + st * 64, in);
                    }
            }
            if constexpr (EIGHT) {
                b.s[0] = __ldg(ls[0]);
                b.s[1] = __ldg(ls[1]);
            }
            lpiece += WK;
            if (lpiece < np) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    la[m] += WK * kPiece;
                    if constexpr (EIGHT) ls[m] += WK * nrb;
                }
            } else {
                ltile += NG;
                seek();
            }
        };
        Piece<EIGHT> b0, b1;
        int tile = ltile, piece = wk;
        seek();
        if (tile < tile1) load(b0);
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        bool far = false;  // whether a scale of the segment's rows is one that needs care
        if constexpr (EIGHT) {
            // the segment's rows, quantised, to shared memory
            __syncthreads();
            for (int i = warp; i < ns * nkb; i += kWarps) {
                const int t = i / nkb, kb = i - t * nkb, slot = slots[s0 + t];
                const int64_t k0 = int64_t(kb) * kFp8Block + lane * 4;
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (k0 < p.K) {
                    if constexpr (DOWN) {
                        const float4 u =
                            __ldcg(reinterpret_cast<const float4 *>(p.h + int64_t(slot) * p.K + k0));
                        v[0] = u.x;
                        v[1] = u.y;
                        v[2] = u.z;
                        v[3] = u.w;
                    } else {
                        Vec<X, 4> u;
                        ld_vec<X, 4>(u, static_cast<const X *>(p.x) + int64_t(slot / p.k) * p.K + k0);
                        widen<X, 4>(u, v);
                    }
                }
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) m = max(m, f8_mag(v[j]));
                m = __reduce_max_sync(kFull, m);
                const bool zeros = m == 0;
                m = max(m, kLeastBits);
                const float up = f8_up<0>(m);
                *reinterpret_cast<uint32_t *>(xs + t * xpitch + kb * kFp8Block + lane * 4) =
                    f8_cvt4<0>(v[0] * up, v[1] * up, v[2] * up, v[3] * up);
                const float scale = f8_scale<0>(m);
                far |= f8_far(scale) && !zeros;
                if (lane == 0) sx[kb * TOK + t] = scale;
            }
            far = __syncthreads_or(far);
        }
        // columns of the operand without a slot repeat the first: nobody reads their sums
        const int bt = g < ns ? g : 0, bslot = slots[s0 + bt];
        const uint8_t *bx;   // 16 bits: x
        const float *bh;     // and h
        uint32_t bs = 0;     // 8 bits: the row in shared memory
        if constexpr (EIGHT) {
            bs = uint32_t(__cvta_generic_to_shared(xs + bt * xpitch + tig * 16));
        } else if constexpr (DOWN) {
            bh = p.h + bslot * p.K + tig * 8;
        } else {
            bx = static_cast<const uint8_t *>(p.x) + int64_t(bslot / p.k) * Kb + tig * 16;
        }
        float acc[2][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = 0.f;
        };
        auto add = [&](const float (&part)[2][4], float q0, float q1) {  // times the columns' scales
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                acc[m][0] = fmaf(part[m][0], q0, acc[m][0]);
                acc[m][1] = fmaf(part[m][1], q1, acc[m][1]);
                acc[m][2] = fmaf(part[m][2], q0, acc[m][2]);
                acc[m][3] = fmaf(part[m][3], q1, acc[m][3]);
            }
        };
        auto compute = [&](const Piece<EIGHT> &b, int pc) {
            const int off = pc * kPiece;
            if constexpr (EIGHT) {
                // The weights and the rows as fp16 (exactly): the tensor cores' form for warps
                // of e4m3 is that conversion again for each of its operands.
                float part[2][4];
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const uint4 x = lds128(bs + off + st * 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 y = widen_e4m3(word(x, i));
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint2 u = widen_e4m3(word(b.a[st][2 * m], i));
                            const uint2 v = widen_e4m3(word(b.a[st][2 * m + 1], i));
                            if (st == 0 && i == 0)
                                mma8<fp16, true>(part[m], u.x, v.x, u.y, v.y, y.x, y.y);
                            else
                                mma8<fp16, false>(part[m], u.x, v.x, u.y, v.y, y.x, y.y);
                        }
                    }
                }
                const float2 q = *reinterpret_cast<const float2 *>(sx + pc * TOK + 2 * tig);
                auto scaled = [&](auto care) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float r = j & 1 ? q.y : q.x;
                            // by the column's own scale: the others keep their bits
                            if (decltype(care)::value && f8_far(r))
                                acc[m][j] += f8_scaled(part[m][j], r, b.s[m]);
                            else
                                acc[m][j] = fmaf(part[m][j] * r, b.s[m], acc[m][j]);
                        }
                };
                if (far)
                    scaled(std::true_type());
                else
                    scaled(std::false_type());
            } else {
                // A piece's products have sums of their own, added with rounding to nearest: the tensor
                // cores cut what they add to: along 16384 a bias of 6e-6 in fp16, 9e-7 in bf16.
                if constexpr (DOWN) {
                    constexpr bool SCALED = std::is_same<W, fp16>::value;
                    constexpr int TERMS = SCALED ? 2 : 3;
                    float4 h[2][2];  // both steps' values on their way together
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        h[st][0] = h[st][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (off + st * 64 + tig * 16 < Kb) {
                            const float *at = bh + (off >> 1) + st * 32;
                            h[st][0] = *reinterpret_cast<const float4 *>(at);
                            h[st][1] = *reinterpret_cast<const float4 *>(at + 4);
                        }
                    }
                    float part[2][4];
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        const float4 lo = h[st][0], hi = h[st][1];
                        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        uint32_t x[TERMS][4];
                        const float down = split8(v, x, static_cast<const W *>(nullptr));
#pragma unroll
                        for (int q = TERMS - 1; q >= 0; --q)  // the least term first
#pragma unroll
                            for (int i = 0; i < 4; i += 2)
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    const uint4 &u = b.a[st][2 * m], &w = b.a[st][2 * m + 1];
                                    const uint32_t a0 = word(u, i), a1 = word(w, i);
                                    const uint32_t a2 = word(u, i + 1), a3 = word(w, i + 1);
                                    if ((SCALED || st == 0) && q == TERMS - 1 && i == 0)
                                        mma8<W, true>(part[m], a0, a1, a2, a3, x[q][i], x[q][i + 1]);
                                    else
                                        mma8<W, false>(part[m], a0, a1, a2, a3, x[q][i], x[q][i + 1]);
                                }
                        if constexpr (SCALED)  // of columns 2 tig and 2 tig + 1
                            add(part, __shfl_sync(kFull, down, 8 * tig),
                                __shfl_sync(kFull, down, 8 * tig + 4));
                    }
                    if constexpr (!SCALED) add(part, 1.f, 1.f);
                } else {
                    uint4 x[2];
#pragma unroll
                    for (int st = 0; st < 2; ++st) {
                        x[st] = zero4();
                        if (off + st * 64 + tig * 16 < Kb)
                            x[st] = *reinterpret_cast<const uint4 *>(bx + off + st * 64);
                    }
                    float part[2][4];
#pragma unroll
                    for (int st = 0; st < 2; ++st)
#pragma unroll
                        for (int i = 0; i < 4; i += 2)
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const uint4 &u = b.a[st][2 * m], &w = b.a[st][2 * m + 1];
                                const uint32_t a0 = word(u, i), a1 = word(w, i);
                                const uint32_t a2 = word(u, i + 1), a3 = word(w, i + 1);
                                const uint32_t b0 = word(x[st], i), b1 = word(x[st], i + 1);
                                if (st == 0 && i == 0)
                                    mma8<W, true>(part[m], a0, a1, a2, a3, b0, b1);
                                else
                                    mma8<W, false>(part[m], a0, a1, a2, a3, b0, b1);
                            }
                    add(part, 1.f, 1.f);
                }
            }
        };
        auto finish = [&](int tl) {
            float *mine = red + (parity * kWarps + warp) * TOK * kPitch;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mine[(2 * tig + (j & 1)) * kPitch + m * 16 + g + (j >> 1) * 8] = acc[m][j];
            group_sync();
            const float *all = red + (parity * kWarps + gi * WK) * TOK * kPitch;
            parity ^= 1;
            if constexpr (!DOWN) {
                for (int o = gtid; o < ns * 16; o += gsize) {
                    const int r = o & 15, t = o >> 4;
                    float gate = 0.f, up = 0.f;
                    for (int w = 0; w < WK; ++w) {
                        gate += all[(w * TOK + t) * kPitch + r];
                        up += all[(w * TOK + t) * kPitch + 16 + r];
                    }
                    const float h = silu(gate, sigm(gate)) * up;
                    p.h[int64_t(slots[s0 + t]) * p.F + int64_t(tl) * 16 + r] = h;
                }
            } else {
                for (int o = gtid; o < ns * 32; o += gsize) {
                    const int r = o & 31, t = o >> 5;
                    const int64_t row = int64_t(tl) * kRows + r;
                    if (row >= p.C) continue;
                    float y = 0.f;
                    for (int w = 0; w < WK; ++w) y += all[(w * TOK + t) * kPitch + r];
                    p.y[int64_t(slots[s0 + t]) * p.C + row] = y;
                }
            }
        };
        clear();
        // one piece is computed while the next is on its way
        auto step = [&](Piece<EIGHT> &now, Piece<EIGHT> &next) {
            const int nt = ltile, npc = lpiece;
            if (nt < tile1) load(next);
            compute(now, piece);
            if (nt != tile) {
                finish(tile);
                clear();
            }
            tile = nt;
            piece = npc;
        };
        while (tile < tile1) {
            step(b0, b1);
            if (tile >= tile1) break;
            step(b1, b0);
        }
        t0 = t1;
    }
    if (!waited) pdl_wait();
}

// f[t] = sum over the token's slots, in their order, of w y; 8 columns a thread.
template <class X>
__global__ void __launch_bounds__(128) k_moe_few_sum(const float *__restrict__ y,
                                                     const int32_t *__restrict__ ids,
                                                     const float *__restrict__ w, int T, int k, int E,
                                                     int64_t C, X *__restrict__ f)
{
    const int64_t i = int64_t(blockIdx.x) * 128 + threadIdx.x, per = C / 8;
    const int t = int(i / per);
    const int64_t c = (i - t * per) * 8;
    pdl_wait();
    if (t >= T) return;
    float sum[8] = {};
    constexpr int U = 8;  // slots whose loads are in flight together
    for (int j0 = 0; j0 < k; j0 += U) {
        float m[U], v[U][8];
        bool in[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            in[j] = j0 + j < k;
            if (!in[j]) continue;
            const int slot = t * k + j0 + j, e = __ldg(ids + slot);
            const float *row = y + int64_t(slot) * C + c;  // of a slot without an expert: not used
            *reinterpret_cast<float4 *>(&v[j][0]) = __ldcg(reinterpret_cast<const float4 *>(row));
            *reinterpret_cast<float4 *>(&v[j][4]) = __ldcg(reinterpret_cast<const float4 *>(row + 4));
            m[j] = __ldg(w + slot);
            in[j] = e >= 0 && e < E;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
            for (int q = 0; q < 8; ++q) sum[q] = in[j] ? fmaf(m[j], v[j][q], sum[q]) : sum[q];
    }
    Vec<X, 8> o;
    narrow<X, 8>(sum, o);
    st_vec<X, 8>(f + t * C + c, o);
}

size_t few_smem(bool eight, int64_t K)
{
    const int64_t nkb = fp8_blocks(K);
    int64_t b = kMaxSlots * 2 + (kMaxExperts + 4) * 2 * 4 + kMaxSegments * 2 + 2 * kWarps * TOK * kPitch * 4;
    if (eight) b += TOK * (nkb * kFp8Block + 64) + nkb * TOK * 4;
    return size_t(b);
}

// How many of a block's 16 warps split a tile's k.  More of them finish a tile
// sooner but join more often, which costs a warp about two pieces' time; fewer
// leave warps without a tile where a block has few.  So the least of tiles in
// turn x (pieces of a warp + 2), for as many segments as the slots can make; but
// four at least, whose pieces are 512 bytes in a row.  With one, two, four, eight and 16:
// 13 tokens, 60 experts, 4096 x 1408, 16 bits: 266, 220, 199, 192, 215 us (four are taken,
// 3% from the best); one token, 64 experts, 7168 x 2048, 8 bits: 84, 69, 68, 71, 75 (four),
// 16 bits: 147, 125, 122, 127, 130 (four); 64 tokens, 8 experts, 4096 x 14336, 16 bits: 865,
// 840, 843, 871, 929 (four); one token, 8 experts, 1024 x 512, 8 bits: 14.7, 12.2, 10.6,
// 10.2, 10.2 (eight up, four down: 10.2).
// The number sets the order of a row's sums: it goes by kSplitSms, not by the device, and in
// batch-invariant mode, where it must not go by the number of slots, by k alone.
int split_of(int64_t K, int bytes, int64_t tiles)
{
    const int64_t np = (K * bytes + kPiece - 1) / kPiece;
    const double per_block = double(tiles) / kSplitSms;
    int best = int(std::min<int64_t>(np, 4));
    best = best == 3 ? 2 : best;
    if (batch_invariant()) return best;
    double least = 1e30;
    for (int w = best; w <= kWarps && w <= np; w *= 2) {
        const double turns = per_block * w / kWarps;
        const double cost = (turns < 1 ? 1 : turns) * double((np + w - 1) / w + 2);
        if (cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

template <class W, class X, bool DOWN>
cudaError_t launch_one(const FewP &p, cudaStream_t s)
{
    auto *kernel = k_moe_few<W, X, DOWN>;
    const size_t smem = few_smem(sizeof(W) == 1, p.K);
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), int(smem));
    if (e != cudaSuccess) return e;
    MHC_PROF(DOWN ? "k_moe_few_down" : "k_moe_few_up", s);
    return launch_k(kernel, dim3(unsigned(num_sms())), dim3(kThreads), smem, s, p);
}

template <class W, class X>
cudaError_t both(FewP &p, const MoeFewArgs &a, cudaStream_t s)
{
    p.wt = a.w1;
    p.s = a.s1;
    p.K = a.C;
    p.rows = 2 * a.F;
    p.ntiles = int(a.F / 16);
    const int64_t segments = std::min<int64_t>(a.E, a.T * a.k);
    p.wk = split_of(p.K, sizeof(W), segments * p.ntiles);
    cudaError_t e = launch_one<W, X, false>(p, s);
    if (e != cudaSuccess) return e;
    p.wt = a.w2;
    p.s = a.s2;
    p.K = a.F;
    p.rows = a.C;
    p.ntiles = int((a.C + kRows - 1) / kRows);
    p.wk = split_of(p.K, sizeof(W), segments * p.ntiles);
    e = launch_one<W, X, true>(p, s);
    if (e != cudaSuccess) return e;
    const int64_t n = a.T * (a.C / 8);
    MHC_PROF("k_moe_few_sum", s);
    return launch_k(k_moe_few_sum<X>, dim3(unsigned((n + 127) / 128)), dim3(128), 0, s,
                    static_cast<const float *>(p.y), p.ids, p.w, p.T, p.k, p.E, p.C,
                    static_cast<X *>(a.f));
}

}  // namespace

size_t moe_few_ws_bytes(int64_t T, int k, int64_t CF)
{
    return ws_align(size_t(T) * size_t(k) * size_t(CF) * 4) + 256;  // h and y
}

cudaError_t launch_moe_few(const MoeFewArgs &a, int dtype, int eight, cudaStream_t s)
{
    FewP p = {};
    p.x = a.x;
    p.ids = a.ids;
    p.w = a.w;
    p.T = int(a.T);
    p.k = a.k;
    p.E = a.E;
    p.F = a.F;
    p.C = a.C;
    p.fault = a.fault;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const size_t n = size_t(a.T) * size_t(a.k);
    p.h = reinterpret_cast<float *>(ws);
    p.y = reinterpret_cast<float *>(ws + n * size_t(a.F) * 4);
    if (eight) return dtype == 0 ? both<E4m3, bf16>(p, a, s) : both<E4m3, fp16>(p, a, s);
    return dtype == 0 ? both<bf16, bf16>(p, a, s) : both<fp16, fp16>(p, a, s);
}

}  // namespace mhc
