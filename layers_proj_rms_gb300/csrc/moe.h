// Launchers of the mixture-of-experts operators (k_moe_sort.cu, k_moe_rows.cu,
// k_moe_router.cu).  dtype: 0 bf16, 1 fp16, 2 fp32.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mhc {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxK = 32;

// Rows that T * k sorted slots can take: each expert that has a slot pads its
// last tile of `align` rows.
inline int64_t moe_rows(int64_t T, int k, int E, int align)
{
    const int64_t n = T * k;
    return n + (n < E ? n : E) * int64_t(align - 1);
}

cudaError_t launch_moe_router_fwd(const void *logits, int dtype, int64_t T, int E, int k,
                                  int score, int renorm, float scale, int32_t *ids, float *w,
                                  cudaStream_t s);
cudaError_t launch_moe_router_bwd(const float *dw, const void *logits, int dtype,
                                  const int32_t *ids, int64_t T, int E, int k, int score,
                                  int renorm, float scale, void *dlogits, int *fault,
                                  cudaStream_t s);
cudaError_t launch_moe_sort(const int32_t *ids, int64_t N, int E, int align, int64_t R,
                            int32_t *counts, int32_t *offsets, int32_t *row_of,
                            int32_t *slot_of, int *fault, cudaStream_t s);
cudaError_t launch_moe_dispatch_fwd(const void *x, int dtype, const int32_t *row_of,
                                    const int32_t *slot_of, int64_t T, int k, int64_t R,
                                    int64_t C, void *xs, int *fault, cudaStream_t s);
// f[t] = sum_j w[t][j] ys[row_of[t][j]]; w NULL: unweighted
cudaError_t launch_moe_combine_fwd(const void *ys, int dtype, const float *w,
                                   const int32_t *row_of, int64_t T, int k, int64_t R, int64_t C,
                                   void *f, int *fault, cudaStream_t s);
cudaError_t launch_moe_combine_bwd(const void *df, const void *ys, int dtype, const float *w,
                                   const int32_t *row_of, const int32_t *slot_of, int64_t T,
                                   int k, int64_t R, int64_t C, void *dys, float *dw, int *fault,
                                   cudaStream_t s);

}  // namespace mhc
