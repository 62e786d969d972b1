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
// there are 8 or 16 columns, the tensor cores are far from busy, and operands
// that stay in registers need no trip through shared memory.
//
// Work: (segment, tile) in order of the experts, a segment up to 8 or 16 slots
// of one expert, a tile 32 weight rows (16 of gate and the same 16 of up); a
// block, one an SM, takes a contiguous share of it.  One to 16 warps split a
// tile's k in pieces and join through shared memory in a fixed order (split_of).  The next
// piece is always in flight: 16 warps x 4 KB an SM.
//
// 16-bit weights: x as it is; h as two terms of the type (its rounding and the
// rest), so nothing is lost between the products.  8-bit weights: x and h are
// quantised by blocks of 128, as mhc_fp8_quant does, when a segment's rows are
// brought to shared memory; each block's product is scaled into fp32 sums.
//
// A slot's row of y is written once and a token's slots are added up in their
// order, so nothing depends on which block did what.  (The last block at a tile of
// columns adding them up, found by counts, took longer: the counts' round trips at
// every tile, and nearly all of the sums in the one block with the last segment.)
#include <algorithm>

#include "elem.cuh"
#include "fp8.cuh"
#include "fp8.h"
#include "launch.h"

namespace mhc {

namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRows = 32;                 // weight rows of a tile
constexpr int kPitch = 36;                // floats of a token's partial sums: no bank conflicts
constexpr int kMaxSlots = kMoeFewTokens * 32;
constexpr int kPiece = 128;               // bytes of k a warp takes at once
enum : int { kFaultExpert = 202 };

struct FewP {
    const void *x;        // up: [T, C] rows; down: h
    const int32_t *ids;
    const float *w;
    const void *wt;       // weights [E, rows, K]
    const float *s;       // their scales [E, blocks of K, blocks of rows], or NULL
    int64_t K, rows;      // reduced length; weight rows of an expert
    int T, k, E;
    int ntiles;           // tiles of an expert
    int wk;               // warps that split a tile's k
    void *h;              // [T*k, F] fp32, or two terms of the type
    float *y;             // [T*k, C]
    int64_t F, C;
    int *fault;
};

struct E4m3 { uint8_t v; };

template <class W>
__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma8<bf16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma8<fp16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma8<E4m3>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// A warp's piece in flight: for each of two 64-byte steps the 16 bytes of rows
// g, g + 8, g + 16, g + 24 (g = lane / 4), and the scales of the two row groups.
template <bool EIGHT>
struct Piece {
    uint4 a[2][4];
    float s[EIGHT ? 2 : 1];
};

// W: bf16, fp16 or E4m3; X: the activations.
template <class W, class X, int NT, bool DOWN>
__global__ void __launch_bounds__(kThreads, 1) k_moe_few(const FewP p)
{
    constexpr bool EIGHT = sizeof(W) == 1;
    constexpr int TOK = 8 * NT;
    extern __shared__ __align__(16) uint8_t smem[];
    // slots in order of their experts, the experts' first slots and first segments
    uint16_t *slots = reinterpret_cast<uint16_t *>(smem);
    int *first = reinterpret_cast<int *>(smem + kMaxSlots * 2);
    int *fseg = first + 1028;
    float *red = reinterpret_cast<float *>(fseg + 1028);  // [2][warps][TOK][kPitch]
    uint8_t *xs = reinterpret_cast<uint8_t *>(red + 2 * kWarps * TOK * kPitch);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, tig = lane & 3;
    const int n = p.T * p.k, E = p.E;

    // What the ids say was there before the first launch began; only h is its work.
    if (!DOWN) pdl_wait();
    int *ids = reinterpret_cast<int *>(red);  // not in use yet
    for (int i = tid; i < n; i += kThreads) {
        int e = __ldg(p.ids + i);
        if (e < -1 || e >= E) {
            if (blockIdx.x == 0 && !DOWN) report_fault(p.fault, kFaultExpert);
            e = -1;
        }
        ids[i] = e;
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        int c = 0;
        for (int i = 0; i < n; ++i) c += ids[i] == e;
        first[e + 1] = c;
        fseg[e + 1] = (c + TOK - 1) / TOK;
    }
    if (tid == 0) first[0] = fseg[0] = 0;
    __syncthreads();
    if (warp == 0) {
        int a = 0, b = 0;
        for (int e0 = 1; e0 <= E; e0 += 32) {
            const int e = e0 + lane;
            int u = e <= E ? first[e] : 0, v = e <= E ? fseg[e] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int ou = __shfl_up_sync(kFull, u, d), ov = __shfl_up_sync(kFull, v, d);
                if (lane >= d) {
                    u += ou;
                    v += ov;
                }
            }
            if (e <= E) {
                first[e] = u + a;
                fseg[e] = v + b;
            }
            a += __shfl_sync(kFull, u, 31);
            b += __shfl_sync(kFull, v, 31);
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
        int at = first[e];
        if (first[e + 1] > at)
            for (int i = 0; i < n; ++i)
                if (ids[i] == e) slots[at++] = uint16_t(i);
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

    const int64_t total = int64_t(nseg) * p.ntiles;
    const int64_t t_begin = total * blockIdx.x / gridDim.x;
    const int64_t t_end = total * (blockIdx.x + 1) / gridDim.x;
    bool waited = !DOWN;
    int parity = 0;

    for (int64_t t0 = t_begin; t0 < t_end;) {
        const int seg = int(t0 / p.ntiles);
        const int64_t t1 = min(t_end, int64_t(seg + 1) * p.ntiles);
        int lo = 0, hi = E;  // the last e with fseg[e] <= seg: an expert with slots
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (fseg[mid] <= seg)
                lo = mid;
            else
                hi = mid;
        }
        const int e = lo;
        const int s0 = first[e] + (seg - fseg[e]) * TOK;
        const int ns = min(TOK, first[e + 1] - s0);
        const uint8_t *we = wt + int64_t(e) * p.rows * Kb;

        auto row_of = [&](int tile, int m) {  // first weight row of row group m
            return DOWN ? int64_t(tile) * kRows + m * 16 : m * p.F + int64_t(tile) * 16;
        };
        auto load = [&](Piece<EIGHT> &b, int tile, int piece) {
            const int64_t off = int64_t(piece) * kPiece + tig * 16;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                int64_t r = row_of(tile, m);
                if (DOWN) r = min(r, p.rows - 16);  // a last tile of 16 rows
                const uint8_t *a = we + (r + g) * Kb + off;
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const bool in = off + st * 64 < Kb;
                    b.a[st][2 * m] = in ? ld_stream(a + st * 64) : zero4();
                    b.a[st][2 * m + 1] = in ? ld_stream(a + 8 * Kb + st * 64) : zero4();
                }
                if constexpr (EIGHT)
                    b.s[m] = __ldg(p.s + (int64_t(e) * nkb + piece) * nrb + r / kFp8Block);
            }
        };
        // this warp's pieces: wk, wk + WK, ... of tiles gi, gi + NG, ...
        const int tile0 = int(t0 - int64_t(seg) * p.ntiles), tile1 = int(t1 - int64_t(seg) * p.ntiles);
        Piece<EIGHT> b0, b1;
        int tile = tile0 + gi, piece = wk;
        if (tile < tile1) load(b0, tile, piece);
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        if constexpr (EIGHT) {
            // the segment's rows, quantised, to shared memory
            __syncthreads();
            for (int i = warp; i < ns * nkb; i += kWarps) {
                const int t = i / nkb, kb = i - t * nkb, slot = slots[s0 + t];
                const int64_t k0 = int64_t(kb) * kFp8Block + lane * 4;
                float v[4] = {0.f, 0.f, 0.f, 0.f};
                if (k0 < p.K) {
                    if constexpr (DOWN) {
                        const float4 u = __ldcg(reinterpret_cast<const float4 *>(
                            static_cast<const float *>(p.h) + int64_t(slot) * p.K + k0));
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
                uint32_t m = kLeastBits;
#pragma unroll
                for (int j = 0; j < 4; ++j) m = max(m, f8_mag(v[j]));
                m = __reduce_max_sync(kFull, m);
                const float up = f8_up<0>(m);
                *reinterpret_cast<uint32_t *>(xs + t * xpitch + kb * kFp8Block + lane * 4) =
                    f8_cvt4<0>(v[0] * up, v[1] * up, v[2] * up, v[3] * up);
                if (lane == 0) sx[kb * TOK + t] = f8_scale<0>(m);
            }
            __syncthreads();
        }
        // columns of the operand without a slot repeat the first: nobody reads their sums
        const uint8_t *bx[NT][DOWN && !EIGHT ? 2 : 1];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const int t = c * 8 + g < ns ? c * 8 + g : 0, slot = slots[s0 + t];
            if constexpr (EIGHT) {
                bx[c][0] = xs + t * xpitch + tig * 16;
            } else if constexpr (DOWN) {
                const uint8_t *hh = static_cast<const uint8_t *>(p.h);
                bx[c][0] = hh + slot * Kb + tig * 16;
                bx[c][1] = hh + (int64_t(n) + slot) * Kb + tig * 16;
            } else {
                bx[c][0] = static_cast<const uint8_t *>(p.x) + int64_t(slot / p.k) * Kb + tig * 16;
            }
        }
        float acc[2][NT][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][c][j] = 0.f;
        };
        auto compute = [&](const Piece<EIGHT> &b, int pc) {
            const int64_t off = int64_t(pc) * kPiece;
            if constexpr (EIGHT) {
                float part[2][NT][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[m][c][j] = 0.f;
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        if (c * 8 >= ns) continue;
                        const uint4 x = *reinterpret_cast<const uint4 *>(bx[c][0] + off + st * 64);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint4 u = b.a[st][2 * m], v = b.a[st][2 * m + 1];
                            mma8<W>(part[m][c], u.x, v.x, u.y, v.y, x.x, x.y);
                            mma8<W>(part[m][c], u.z, v.z, u.w, v.w, x.z, x.w);
                        }
                    }
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    if (c * 8 >= ns) continue;
                    const float2 q = *reinterpret_cast<const float2 *>(sx + pc * TOK + c * 8 + 2 * tig);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const float q0 = q.x * b.s[m], q1 = q.y * b.s[m];
                        acc[m][c][0] = fmaf(part[m][c][0], q0, acc[m][c][0]);
                        acc[m][c][1] = fmaf(part[m][c][1], q1, acc[m][c][1]);
                        acc[m][c][2] = fmaf(part[m][c][2], q0, acc[m][c][2]);
                        acc[m][c][3] = fmaf(part[m][c][3], q1, acc[m][c][3]);
                    }
                }
            } else {
                constexpr int TERMS = DOWN ? 2 : 1;
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const bool in = off + st * 64 + tig * 16 < Kb;
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        if (c * 8 >= ns) continue;
#pragma unroll
                        for (int q = 0; q < TERMS; ++q) {
                            uint4 x = zero4();
                            if (in) x = *reinterpret_cast<const uint4 *>(bx[c][q] + off + st * 64);
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const uint4 u = b.a[st][2 * m], v = b.a[st][2 * m + 1];
                                mma8<W>(acc[m][c], u.x, v.x, u.y, v.y, x.x, x.y);
                                mma8<W>(acc[m][c], u.z, v.z, u.w, v.w, x.z, x.w);
                            }
                        }
                    }
                }
            }
        };
        auto finish = [&](int tl) {
            float *mine = red + (parity * kWarps + warp) * TOK * kPitch;
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mine[(c * 8 + 2 * tig + (j & 1)) * kPitch + m * 16 + g + (j >> 1) * 8] =
                            acc[m][c][j];
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
                    const int slot = slots[s0 + t];
                    const int64_t at = int64_t(slot) * p.F + int64_t(tl) * 16 + r;
                    if constexpr (EIGHT) {
                        static_cast<float *>(p.h)[at] = h;
                    } else {
                        X *hh = static_cast<X *>(p.h);
                        const X top = X(h);
                        const float rest = h - float(top);
                        hh[at] = top;
                        hh[int64_t(n) * p.F + at] = X(isfinite(rest) ? rest : 0.f);
                    }
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
            int nt = tile, npc = piece + WK;
            if (npc >= np) {
                npc = wk;
                nt = tile + NG;
            }
            if (nt < tile1) load(next, nt, npc);
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
    for (int j = 0; j < k; ++j) {
        const int slot = t * k + j, e = __ldg(ids + slot);
        if (e < 0 || e >= E) continue;
        const float *row = y + int64_t(slot) * C + c;
        const float4 a = *reinterpret_cast<const float4 *>(row), b = *reinterpret_cast<const float4 *>(row + 4);
        const float m = __ldg(w + slot), v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = fmaf(m, v[q], sum[q]);
    }
    Vec<X, 8> o;
    narrow<X, 8>(sum, o);
    st_vec<X, 8>(f + t * C + c, o);
}

size_t few_smem(int NT, bool eight, int64_t K)
{
    const int64_t nkb = fp8_blocks(K), tok = 8 * NT;
    int64_t b = kMaxSlots * 2 + 1028 * 2 * 4 + 2 * kWarps * tok * kPitch * 4;
    if (eight) b += tok * (nkb * kFp8Block + 64) + nkb * tok * 4;
    return size_t(b);
}
constexpr size_t kSmemMax = 232448;

// How many of a block's 16 warps split a tile's k.  More of them finish a tile
// sooner but join more often, which costs a warp about two pieces' time; fewer
// leave warps without a tile where a block has few.  So the least of tiles in
// turn x (pieces of a warp + 2), for as many segments as the slots can make; but
// four at least, whose pieces are 512 bytes in a row (13 tokens, 4096 x 1408, 60
// experts, 16 bits: 315 us with one, 269 with two, 226 with four, 219 with eight).
int split_of(int64_t K, int bytes, int64_t tiles)
{
    const int64_t np = (K * bytes + kPiece - 1) / kPiece;
    const double per_block = double(tiles) / num_sms();
    int best = int(std::min<int64_t>(np, 4));
    best = best == 3 ? 2 : best;
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

template <class W, class X, int NT, bool DOWN>
cudaError_t launch_one(const FewP &p, cudaStream_t s)
{
    auto *kernel = k_moe_few<W, X, NT, DOWN>;
    const size_t smem = few_smem(NT, sizeof(W) == 1, p.K);
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel), int(smem));
    if (e != cudaSuccess) return e;
    MHC_PROF(DOWN ? "k_moe_few_down" : "k_moe_few_up", s);
    return launch_k(kernel, dim3(unsigned(num_sms())), dim3(kThreads), smem, s, p);
}

template <class W, class X, bool DOWN>
cudaError_t by_columns(const FewP &p, cudaStream_t s)
{
    // 16 columns where an expert may have more than 8 slots and they fit
    if (p.T > 8 && few_smem(2, sizeof(W) == 1, p.K) <= kSmemMax)
        return launch_one<W, X, 2, DOWN>(p, s);
    return launch_one<W, X, 1, DOWN>(p, s);
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
    cudaError_t e = by_columns<W, X, false>(p, s);
    if (e != cudaSuccess) return e;
    p.wt = a.w2;
    p.s = a.s2;
    p.K = a.F;
    p.rows = a.C;
    p.ntiles = int((a.C + kRows - 1) / kRows);
    p.wk = split_of(p.K, sizeof(W), segments * p.ntiles);
    e = by_columns<W, X, true>(p, s);
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
    p.h = ws;
    p.y = reinterpret_cast<float *>(ws + n * size_t(a.F) * 4);
    if (eight) return dtype == 0 ? both<E4m3, bf16>(p, a, s) : both<E4m3, fp16>(p, a, s);
    return dtype == 0 ? both<bf16, bf16>(p, a, s) : both<fp16, fp16>(p, a, s);
}

}  // namespace mhc
