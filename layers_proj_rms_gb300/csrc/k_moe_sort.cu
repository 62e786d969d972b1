// Stable counting sort of token slots by expert.
//
// ids [N] (N = T * k) names the expert of every slot, -1 a dropped slot.
// Expert e's rows are [offsets[e], offsets[e] + counts[e]), in ascending slot
// order, and offsets[e + 1] - offsets[e] is counts[e] rounded up to `align`.
// row_of [N] is a slot's row (-1: dropped), slot_of [R] a row's slot (-1:
// padding, or past the last segment).
//
// One launch of one thread-block cluster.  The slots are cut into contiguous
// segments, one per warp of the cluster.  First pass: each warp counts its
// segment's experts in shared memory (match_any groups equal ids of 32 slots,
// the group's lowest lane adds its size: no atomics, no order left open).
// The counts of a block's warps are scanned per expert; the blocks' totals
// are exchanged through distributed shared memory; one block scan over the
// experts gives the offsets.  Second pass: the same walk gives each slot its
// rank, so a row is base + rank and the order is stable by construction.
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

struct SortArgs {
    const int32_t *ids;
    int32_t *counts, *offsets, *row_of, *slot_of;
    int64_t N, R, seg;  // seg: slots of a warp, a multiple of 32
    int E, align;
    int *fault;
};

__global__ void __launch_bounds__(kSortThreads) k_moe_sort(const SortArgs A)
{
    extern __shared__ int sm[];
    const int E = A.E;
    int *hist = sm;                       // [warps][E], then exclusive over warps
    int *total = hist + kSortWarps * E;   // [E] this block's counts (read by the cluster)
    int *base = total + E;                // [E] row of this block's first slot of e
    int *off = base + E;                  // [E + 1] padded offsets
    int *count = off + E + 1;             // [E] counts over all blocks
    __shared__ int wsum[kSortWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster.block_rank()), nb = int(cluster.num_blocks());
    for (int i = tid; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait();

    const int64_t gw = int64_t(rank) * kSortWarps + warp;
    const int64_t s0 = gw * A.seg < A.N ? gw * A.seg : A.N;
    const int64_t s1 = s0 + A.seg < A.N ? s0 + A.seg : A.N;
    int *mine = hist + warp * E;
    const unsigned below = (1u << lane) - 1u;
    auto expert = [&](int64_t i) {
        int e = i < s1 ? __ldg(A.ids + i) : -1;
        if (e < -1 || e >= E) {
            report_fault(A.fault, kFaultExpert);
            e = -1;
        }
        return e;
    };
    for (int64_t b = s0; b < s1; b += 32) {
        const int e = expert(b + lane);
        const unsigned same = __match_any_sync(kFull, e);
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) {
        int s = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = s;
            s += c;
        }
        total[e] = s;
    }
    cluster.sync();
    // E <= kSortThreads: thread e owns expert e
    int all = 0, before = 0;
    if (tid < E)
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
    int start = incl - padded;
    for (int w = 0; w < warp; ++w) start += wsum[w];
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

    for (int64_t b = s0; b < s1; b += 32) {
        const int64_t i = b + lane;
        const int e = expert(i);
        const unsigned same = __match_any_sync(kFull, e);
        int row = -1;
        if (e >= 0) row = base[e] + mine[e] + __popc(same & below);
        __syncwarp();
        if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
        __syncwarp();
        if (i < s1) {
            A.row_of[i] = row;
            if (row >= 0) A.slot_of[row] = int(i);
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
    int nb = 1;  // blocks: about 2048 slots each, at most the portable cluster
    while (nb < 8 && int64_t(nb) * 2048 < N) nb *= 2;
    const int64_t warps = int64_t(nb) * kSortWarps;
    a.seg = (N + warps * 32 - 1) / (warps * 32) * 32;
    const size_t smem = (size_t(kSortWarps + 4) * E + 1) * sizeof(int);
    cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(k_moe_sort),
                                   int((size_t(kSortWarps + 4) * kMoeMaxExperts + 1) * sizeof(int)));
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
    return cudaLaunchKernelEx(&cfg, k_moe_sort, a);
}

}  // namespace mhc
