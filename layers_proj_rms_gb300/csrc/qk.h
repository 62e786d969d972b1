// Arguments and launchers of the q/k norm + rotation kernels (k_qk.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mhc {

// One of the two tensors (q, k): [T, H, D] with its own token and head
// strides in elements; head elements are contiguous.  x is the input; up is
// the upstream gradient (backward); out the output or the input's gradient.
struct QkTensor {
    const void *x, *up;
    void *out;
    int64_t x_t, x_h, up_t, up_h, out_t, out_h;
    const float *gamma;  // [D] or NULL
    float *dgamma;       // [D] or NULL (backward)
    int H;
};

struct QkArgs {
    QkTensor m[2];  // q, k
    const float *cs, *sn;  // [P, R/2]
    const int32_t *pos;    // [T] or NULL: pos = t
    int64_t T, P;
    int D, R;
    int interleaved;
    uint64_t bits;  // the pointers and the strides in bytes, as given, or-ed (their alignment)
    float eps;
    int *fault;
};

size_t qk_bwd_ws_bytes(int64_t T, int64_t heads, int64_t D);
cudaError_t launch_qk_fwd(const QkArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_qk_bwd(const QkArgs &a, int dtype, float *ws, cudaStream_t s);

}  // namespace mhc
