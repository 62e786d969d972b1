// Stable counting sort of token slots by expert.
//
// ids [N] (N = T * k) names the expert of every slot, -1 a dropped slot.
// Expert e's rows are [offsets[e], offsets[e] + counts[e]), in ascending slot
// order, and offsets[e + 1] - offsets[e] is counts[e] rounded up to `align`.
// row_of [N] is a slot's row (-1: dropped), slot_of [R] a row's slot (-1:
// padding, or past the last segment).
//
// One launch of one thread-block cluster, or of several that each sort a share
// of the slots and count the others' for themselves, so that no cluster waits
// for another.  The slots are cut into contiguous segments, one per warp.  Each
// warp counts its segment's experts in shared memory: ballots group the equal
// ids of 32 slots, and the group's lowest lane adds its size, so the order is
// never open (other shares are only counted, where it does not matter).
// What a slot found there before it is its rank in the segment.  The counts of
// a block's warps are scanned per expert, the blocks' totals exchanged through
// distributed shared memory, and one scan over the experts gives the offsets:
// a slot's row is its segment's base + its rank, stable by construction.
// Segments of up to 256 slots stay in registers; longer ones are walked twice.
//
// What bounds it: latency (a training step's 131072 slots are 0.5 MB); far beyond
// that, that each cluster counts all the slots of the others (1 M slots: 33 us).
#include <cooperative_groups.h>

#include "launch.h"
#include "moe.h"

namespace cg = cooperative_groups;

namespace mhc {

constexpr int kFaultExpert = 202;  // an expert id outside [-1, E)

namespace {

// Warps of a block: 8 for a few slots and experts (fewer to synchronise: 148
// slots of 60 experts), else 32.
constexpr int kFewWarps = 8, kSortWarps = 32;

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(kFull, v); }

struct SortArgs {
    const int32_t *ids;
    int32_t *counts, *offsets, *row_of, *slot_of;
    int64_t N, R, seg;  // seg: slots of a warp, a multiple of 32
    int E, align;
    int *fault;
};

// ids of one tile of a warp's segment: TILE x 32 slots from b on
constexpr int kTile = 8;  // at most

template <int TILE>
__device__ __forceinline__ void load_tile(const SortArgs &A, int64_t b, int64_t s1, int lane,
                                          int (&e)[TILE])
{
#pragma unroll
    for (int q = 0; q < TILE; ++q) {
        const int64_t i = b + 32 * q + lane;
        e[q] = i < s1 ? __ldg(A.ids + i) : -1;
    }
#pragma unroll
    for (int q = 0; q < TILE; ++q)
        if (e[q] < -1 || e[q] >= A.E) {
            report_fault(A.fault, kFaultExpert);
            e[q] = -1;
        }
}

// All ones where bit b of e is set, else 0.
__device__ __forceinline__ unsigned bit_mask(int e, int b)
{
    unsigned m;
    asm("bfe.s32 %0, %1, %2, 1;" : "=r"(m) : "r"(e), "r"(b));
    return m;
}

// Ranks of a tile's slots among the segment's slots of the same expert; mine
// holds how many there were before, and is brought up to date.  The lanes of
// equal ids are found by a ballot per bit of the id.
template <int TILE>
__device__ __forceinline__ void rank_tile(const int (&e)[TILE], int bits, int *mine, int lane,
                                          int (&rank)[TILE])
{
    const unsigned below = (1u << lane) - 1u;
    unsigned same[TILE];
#pragma unroll
    for (int q = 0; q < TILE; ++q) {
        same[q] = __ballot_sync(kFull, e[q] >= 0);  // a dropped slot's is not used
    }
#pragma unroll
    for (int b = 0; b < 10; ++b) {  // E <= 1024
        if (b >= bits) break;
#pragma unroll
        for (int q = 0; q < TILE; ++q) {
            const unsigned m = __ballot_sync(kFull, e[q] & (1 << b));
            same[q] &= ~(m ^ bit_mask(e[q], b));
        }
    }
#pragma unroll
    for (int q = 0; q < TILE; ++q) {
        rank[q] = e[q] >= 0 ? mine[e[q]] + __popc(same[q] & below) : 0;
        __syncwarp();
        if (e[q] >= 0 && (same[q] & below) == 0) mine[e[q]] += __popc(same[q]);
        __syncwarp();
    }
}

// Counts the experts of slots [lo, hi) into cnt (shared memory): thread i of n.
// lo is a multiple of 4.  Sums of ones: no order matters.
__device__ __forceinline__ void count_range(const SortArgs &A, int64_t lo, int64_t hi, int64_t i,
                                            int64_t n, int *cnt)
{
    auto add = [&](int e) {
        if (e >= 0 && e < A.E) atomicAdd(cnt + e, 1);
    };
    const int4 *ids = reinterpret_cast<const int4 *>(A.ids);
#pragma unroll 4
    for (int64_t q = lo / 4 + i; q < hi / 4; q += n) {
        const int4 v = __ldg(ids + q);
        add(v.x);
        add(v.y);
        add(v.z);
        add(v.w);
    }
    if (lo < hi && i < hi % 4) add(__ldg(A.ids + hi / 4 * 4 + i));
}

// slot_of = -1 everywhere: thread i of n
__device__ __forceinline__ void fill_unused(int32_t *slot_of, int64_t R, int64_t i, int64_t n)
{
    const int4 none = make_int4(-1, -1, -1, -1);
    for (int64_t r = i; r < R / 4; r += n) reinterpret_cast<int4 *>(slot_of)[r] = none;
    if (i < R % 4) slot_of[R / 4 * 4 + i] = -1;
}

// ONE: every segment is one tile (of TILE x 32 slots).  W: warps of a block;
// E <= 32 W.  MANY: several clusters, each with a share of the slots; a cluster
// counts the others' slots for itself, so no cluster waits for another.
template <bool ONE, bool MANY, int W, int TILE>
__global__ void __launch_bounds__(32 * W) k_moe_sort(const SortArgs A)
{
    extern __shared__ int sm[];
    const int E = A.E;
    int *hist = sm;                       // [warps][E], then exclusive over warps
    int *total = hist + W * E;            // [E] this block's counts (read by the cluster)
    int *base = total + E;                // [E] row of this block's first slot of e
    int *off = base + E;                  // [E + 1] padded offsets
    int *count = off + E + 1;             // [E] counts over all blocks
    int *loc = count + E;                 // [E] this block's slots of lower experts
    int *pre = loc + E;                   // [E] MANY: counted of the shares before,
    int *post = pre + E;                  // [E] and after the cluster's
    int *sorted = post + E;               // [32 W TILE] ONE: the block's slots by expert
    __shared__ int wsum[2][W];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster.block_rank()), nb = int(cluster.num_blocks());
    const int64_t block = MANY ? int64_t(blockIdx.x) : rank;  // of all blocks
    const int64_t blocks = MANY ? int64_t(gridDim.x) : nb;
    const int64_t gw = block * W + warp;
    const int64_t s0 = gw * A.seg < A.N ? gw * A.seg : A.N;
    const int64_t s1 = s0 + A.seg < A.N ? s0 + A.seg : A.N;
    int *mine = hist + warp * E;
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    if (MANY) {
        for (int e = tid; e < E; e += 32 * W) pre[e] = post[e] = 0;
        __syncthreads();
    }
    __syncwarp();
    pdl_wait();

    const int bits = 32 - __clz(E - 1);  // of an id; 0 where E = 1
    int e[TILE], rk[TILE];
    if (ONE) load_tile(A, s0, s1, lane, e);
    if (MANY) {
        const int64_t share = int64_t(nb) * W * A.seg, from = (block - rank) / nb * share;
        const int64_t me = int64_t(rank) * (32 * W) + tid, n = int64_t(nb) * (32 * W);
        count_range(A, 0, from < A.N ? from : A.N, me, n, pre);
        count_range(A, from + share < A.N ? from + share : A.N, A.N, me, n, post);
    }
    // first -1 everywhere (the slots' rows follow after the cluster's barriers):
    // on few slots this takes 0.3 to 1.4 us less than clearing the padding alone
    if (ONE && !MANY) fill_unused(A.slot_of, A.R, int64_t(rank) * (32 * W) + tid, int64_t(nb) * (32 * W));
    for (int64_t b = s0; b < s1; b += 32 * TILE) {
        if (!ONE) load_tile(A, b, s1, lane, e);
        rank_tile(e, bits, mine, lane, rk);
    }
    __syncthreads();
    for (int x = tid; x < E; x += 32 * W) {
        int c[W], s = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) c[w] = hist[w * E + x];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            hist[w * E + x] = s;
            s += c[w];
        }
        total[x] = s;
    }
    cluster.sync();
    // E <= 32 * W: thread x owns expert x
    int all = 0, before = 0;
    if (tid < E)
#pragma unroll 8
        for (int b = 0; b < nb; ++b) {
            const int c = cluster.map_shared_rank(total, b)[tid];
            before += b < rank ? c : 0;
            all += c;
            if (MANY) {
                const int q = cluster.map_shared_rank(pre, b)[tid];
                before += q;
                all += q + cluster.map_shared_rank(post, b)[tid];
            }
        }
    // padded < 2^31: the caller has checked R
    const int padded = (all + A.align - 1) / A.align * A.align;
    int incl = padded, here = tid < E ? total[tid] : 0, incl_here = here;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, d), w = __shfl_up_sync(kFull, incl_here, d);
        if (lane >= d) {
            incl += v;
            incl_here += w;
        }
    }
    if (lane == 31) {
        wsum[0][warp] = incl;
        wsum[1][warp] = incl_here;
    }
    __syncthreads();
    const int start = warp_sum_int(lane < warp ? wsum[0][lane] : 0) + incl - padded;
    const int mine_from = warp_sum_int(lane < warp ? wsum[1][lane] : 0) + incl_here - here;
    if (tid < E) {
        off[tid] = start;
        base[tid] = start + before;
        count[tid] = all;
        if (tid == E - 1) off[E] = start + padded;
        loc[tid] = mine_from;
        if (block == 0) {
            A.counts[tid] = all;
            A.offsets[tid] = start;
            if (tid == E - 1) A.offsets[E] = start + padded;
        }
    }
    // also: nobody leaves while its totals are still being read
    cluster.sync();

    if constexpr (ONE) {
        // rows in slot order; slots by expert into shared memory, from where
        // neighbours of a segment leave together (straight to memory, each of
        // 32 lanes to a line of its own, they took 5 us of 131072 slots' 14.6)
        const int64_t block0 = block * W * A.seg;
#pragma unroll
        for (int q = 0; q < TILE; ++q) {
            const int64_t i = s0 + 32 * q + lane;
            if (i < s1) {
                const int x = e[q], r = x < 0 ? 0 : mine[x] + rk[q];
                A.row_of[i] = x < 0 ? -1 : base[x] + r;
                if (x >= 0) sorted[loc[x] + r] = int(i - block0) << 10 | x;
            }
        }
        __syncthreads();
        const int n = loc[E - 1] + total[E - 1];
        for (int i = tid; i < n; i += 32 * W) {
            const int x = sorted[i] & 1023;
            A.slot_of[base[x] + i - loc[x]] = int(block0) + (sorted[i] >> 10);
        }
    } else {
        for (int64_t b = s0; b < s1; b += 32 * TILE) {
            load_tile(A, b, s1, lane, e);
            rank_tile(e, bits, mine, lane, rk);
#pragma unroll
            for (int q = 0; q < TILE; ++q) {
                const int64_t i = b + 32 * q + lane;
                if (i < s1) {
                    const int row = e[q] < 0 ? -1 : base[e[q]] + rk[q];
                    A.row_of[i] = row;
                    if (row >= 0) A.slot_of[row] = int(i);
                }
            }
        }
    }
    if constexpr (!ONE || MANY) {
        // padding of the segments, eight lanes to an expert, then the rows past
        // the last one
        for (int64_t x = gw * 4 + lane / 8; x < E; x += blocks * W * 4)
            for (int r = off[x] + count[x] + lane % 8; r < off[x + 1]; r += 8) A.slot_of[r] = -1;
        for (int64_t r = off[E] + block * (32 * W) + tid; r < A.R; r += blocks * (32 * W))
            A.slot_of[r] = -1;
    }
}

size_t sort_smem(int E, bool one, int warps)
{
    return (size_t(warps + 7) * E + 1 + (one ? warps * 32 * kTile : 0)) * sizeof(int);
}

// The form for segments of `seg` slots (ONE only where a segment fits its tile).
// One cluster's are never longer than 64.
typedef void (*SortKernel)(SortArgs);
SortKernel sort_kernel(bool many, int w, int64_t seg, bool *one)
{
    *one = seg <= 32 * kTile;
    if (!*one) return k_moe_sort<false, true, kSortWarps, kTile>;
    if (many)
        return seg <= 32   ? k_moe_sort<true, true, kSortWarps, 1>
               : seg <= 64 ? k_moe_sort<true, true, kSortWarps, 2>
                           : k_moe_sort<true, true, kSortWarps, kTile>;
    if (w == kFewWarps) return k_moe_sort<true, false, kFewWarps, 1>;
    return seg <= 32 ? k_moe_sort<true, false, kSortWarps, 1> : k_moe_sort<true, false, kSortWarps, 2>;
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t *ids, int64_t N, int E, int align, int64_t R,
                            int32_t *counts, int32_t *offsets, int32_t *row_of,
                            int32_t *slot_of, int *fault, cudaStream_t s)
{
    SortArgs a{ids, counts, offsets, row_of, slot_of, N, R, 0, E, align, fault};
    // Up to 32768 slots: one cluster, 1024 slots a block (4096 slots: 4.6 us; up
    // to 4096 a block: 6.4) and at most 16 blocks.  More: clusters of four with
    // 4096 slots each, at most 32 (131072 slots of 256 experts: 9.1 us; one cluster
    // of 16 13.3, eight of 16, not all resident at once, 16.0, sixteen of 8 13.6;
    // 32768 slots: 7.0, one cluster 6.2).
    const bool many = N > 32768;
    int nb = 1, p = 1;
    if (many) {
        nb = 4;
        while (p < 32 && int64_t(p) * 4096 < N) ++p;
    } else {
        while (nb < 16 && int64_t(nb) * 1024 < N) nb *= 2;
    }
    const int w = N <= kFewWarps * 32 && E <= kFewWarps * 32 ? kFewWarps : kSortWarps;
    const int64_t warps = int64_t(p) * nb * w;
    a.seg = (N + warps * 32 - 1) / (warps * 32) * 32;
    bool one;
    const SortKernel kernel = sort_kernel(many, w, a.seg, &one);
    if (!many && (a.seg > 64 || (w == kFewWarps && a.seg > 32))) return cudaErrorInvalidValue;
    const size_t smem = sort_smem(E, one, w);
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel),
                                   int(sort_smem(32 * w, one, w)));
    if (e == cudaSuccess && nb > 8)
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p * nb));
    cfg.blockDim = dim3(unsigned(32 * w));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(nb);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    MHC_PROF("k_moe_sort", s);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mhc
