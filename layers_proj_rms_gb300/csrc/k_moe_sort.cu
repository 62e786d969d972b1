// Stable counting sort of token slots by expert.
//
// ids [N] (N = T * k) names the expert of every slot, -1 a dropped slot.
// Expert e's rows are [offsets[e], offsets[e] + counts[e]), in ascending slot
// order, and offsets[e + 1] - offsets[e] is counts[e] rounded up to `align`.
// row_of [N] is a slot's row (-1: dropped), slot_of [R] a row's slot (-1:
// padding, or past the last segment).
//
// One launch of one thread-block cluster.  The slots are cut into contiguous
// segments, one per warp of the cluster.  Each warp counts its segment's
// experts in shared memory: match_any groups the equal ids of 32 slots, and
// the group's lowest lane adds its size, so no atomics and no order left open.
// What a slot found there before it is its rank in the segment.  The counts of
// a block's warps are scanned per expert, the blocks' totals exchanged through
// distributed shared memory, and one scan over the experts gives the offsets:
// a slot's row is its segment's base + its rank, stable by construction.
// Segments of up to 256 slots stay in registers; longer ones are walked twice.
//
// What bounds it: latency (a training step's 131072 slots are 0.5 MB).
#include <cooperative_groups.h>

#include "launch.h"
#include "moe.h"

namespace cg = cooperative_groups;

namespace mhc {

constexpr int kFaultExpert = 202;  // an expert id outside [-1, E)

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(kFull, v); }

struct SortArgs {
    const int32_t *ids;
    int32_t *counts, *offsets, *row_of, *slot_of;
    int64_t N, R, seg;  // seg: slots of a warp, a multiple of 32
    int E, align;
    int *fault;
};

// ids of one tile of a warp's segment: kTile x 32 slots from b on
constexpr int kTile = 8;

__device__ __forceinline__ void load_tile(const SortArgs &A, int64_t b, int64_t s1, int lane,
                                          int (&e)[kTile])
{
#pragma unroll
    for (int q = 0; q < kTile; ++q) {
        const int64_t i = b + 32 * q + lane;
        e[q] = i < s1 ? __ldg(A.ids + i) : -1;
    }
#pragma unroll
    for (int q = 0; q < kTile; ++q)
        if (e[q] < -1 || e[q] >= A.E) {
            report_fault(A.fault, kFaultExpert);
            e[q] = -1;
        }
}

// Ranks of a tile's slots among the segment's slots of the same expert; mine
// holds how many there were before, and is brought up to date.
__device__ __forceinline__ void rank_tile(const int (&e)[kTile], int *mine, int lane, int (&rank)[kTile])
{
    const unsigned below = (1u << lane) - 1u;
    unsigned same[kTile];
#pragma unroll
    for (int q = 0; q < kTile; ++q) same[q] = __match_any_sync(kFull, e[q]);
#pragma unroll
    for (int q = 0; q < kTile; ++q) {
        rank[q] = e[q] >= 0 ? mine[e[q]] + __popc(same[q] & below) : 0;
        __syncwarp();
        if (e[q] >= 0 && (same[q] & below) == 0) mine[e[q]] += __popc(same[q]);
        __syncwarp();
    }
}

// ONE: every segment is one tile
template <bool ONE>
__global__ void __launch_bounds__(kSortThreads) k_moe_sort(const SortArgs A)
{
    extern __shared__ int sm[];
    const int E = A.E;
    int *hist = sm;                       // [warps][E], then exclusive over warps, plus base
    int *total = hist + kSortWarps * E;   // [E] this block's counts (read by the cluster)
    int *base = total + E;                // [E] row of this block's first slot of e
    int *off = base + E;                  // [E + 1] padded offsets
    int *count = off + E + 1;             // [E] counts over all blocks
    __shared__ int wsum[kSortWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster.block_rank()), nb = int(cluster.num_blocks());
    const int64_t gw = int64_t(rank) * kSortWarps + warp;
    const int64_t s0 = gw * A.seg < A.N ? gw * A.seg : A.N;
    const int64_t s1 = s0 + A.seg < A.N ? s0 + A.seg : A.N;
    int *mine = hist + warp * E;
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    pdl_wait();

    int e[kTile], rk[kTile];
    for (int64_t b = s0; b < s1; b += 32 * kTile) {
        load_tile(A, b, s1, lane, e);
        rank_tile(e, mine, lane, rk);
    }
    __syncthreads();
    for (int x = tid; x < E; x += kSortThreads) {
        int c[kSortWarps], s = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * E + x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            hist[w * E + x] = s;
            s += c[w];
        }
        total[x] = s;
    }
    cluster.sync();
    // E <= kSortThreads: thread x owns expert x
    int all = 0, before = 0;
    if (tid < E)
#pragma unroll 8
        for (int b = 0; b < nb; ++b) {
            const int c = cluster.map_shared_rank(total, b)[tid];
            before += b < rank ? c : 0;
            all += c;
        }
    // padded < 2^31: the caller has checked R
    const int padded = (all + A.align - 1) / A.align * A.align;
    int incl = padded;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    const int before_warps = warp_sum_int(lane < warp ? wsum[lane] : 0);
    const int start = before_warps + incl - padded;
    if (tid < E) {
        off[tid] = start;
        base[tid] = start + before;
        count[tid] = all;
        if (tid == E - 1) off[E] = start + padded;
        if (rank == 0) {
            A.counts[tid] = all;
            A.offsets[tid] = start;
            if (tid == E - 1) A.offsets[E] = start + padded;
        }
    }
    // also: nobody leaves while its totals are still being read
    cluster.sync();

    for (int64_t b = s0; b < s1; b += 32 * kTile) {
        if (!ONE) {
            load_tile(A, b, s1, lane, e);
            rank_tile(e, mine, lane, rk);
        }
#pragma unroll
        for (int q = 0; q < kTile; ++q) {
            const int64_t i = b + 32 * q + lane;
            if (i < s1) {
                const int row = e[q] < 0 ? -1 : base[e[q]] + rk[q] + (ONE ? mine[e[q]] : 0);
                A.row_of[i] = row;
                if (row >= 0) A.slot_of[row] = int(i);
            }
        }
    }
    // padding of the segments, then the rows past the last one
    for (int e = int(gw); e < E; e += nb * kSortWarps)
        for (int r = off[e] + count[e] + lane; r < off[e + 1]; r += 32) A.slot_of[r] = -1;
    for (int64_t r = off[E] + int64_t(rank) * kSortThreads + tid; r < A.R;
         r += int64_t(nb) * kSortThreads)
        A.slot_of[r] = -1;
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t *ids, int64_t N, int E, int align, int64_t R,
                            int32_t *counts, int32_t *offsets, int32_t *row_of,
                            int32_t *slot_of, int *fault, cudaStream_t s)
{
    SortArgs a{ids, counts, offsets, row_of, slot_of, N, R, 0, E, align, fault};
    // blocks: up to 2048 slots each (two of eight lookups a lane), 16 at most
    int nb = 1;
    while (nb < 16 && int64_t(nb) * 2048 < N) nb *= 2;
    const int64_t warps = int64_t(nb) * kSortWarps;
    a.seg = (N + warps * 32 - 1) / (warps * 32) * 32;
    const bool one = a.seg <= 32 * kTile;
    void (*kernel)(SortArgs) = one ? k_moe_sort<true> : k_moe_sort<false>;
    const size_t smem = (size_t(kSortWarps + 4) * E + 1) * sizeof(int);
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kernel),
                                   int((size_t(kSortWarps + 4) * kMoeMaxExperts + 1) * sizeof(int)));
    if (e == cudaSuccess && nb > 8)
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(nb));
    cfg.blockDim = dim3(kSortThreads);
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
