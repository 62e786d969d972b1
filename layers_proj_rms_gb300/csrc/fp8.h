// Launchers of the 8-bit floating-point operators (k_fp8_quant.cu,
// k_fp8_gemm.cu) and of the experts' layer for a few tokens (k_moe_few.cu).
// dtype: 0 bf16, 1 fp16, 2 fp32; format: 0 e4m3, 1 e5m2.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mhc {

// Elements that share a scale along the reduced dimension (and along both
// dimensions of a tile).
constexpr int kFp8Block = 128;

inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// What is quantised: the rows themselves, silu(gate) up of rows [gate | up],
// or the gradient of that.
enum Fp8Source { kFp8Plain = 0, kFp8Swiglu = 1, kFp8SwigluGrad = 2 };

struct Fp8QuantArgs {
    const void *x;    // [G, R, C] (plain), [R, 2F]
    const void *da;   // [R, F]
    void *y;          // the values in the activations' type, or NULL
    uint8_t *q, *qt;  // [G, R, C], [G, C, R], or NULL
    float *s, *st;    // their scales
    int64_t G, R, C;  // C: columns of the result
    int64_t F;        // swiglu: columns of gate
    int tiles;        // one scale a tile of 128 x 128
    unsigned nrb, ncb;  // blocks of R and C; G times them is below 2^31
};

cudaError_t launch_fp8_quant(const Fp8QuantArgs &a, int source, int dtype, int format,
                             cudaStream_t s);

// out [R, N] = a b[e]^T over the rows of segment e, e < G; rows past the last
// segment are zeroed.  offsets NULL: one segment of all R rows (G = 1).
struct Fp8GemmArgs {
    const uint8_t *a, *b;  // [R, K], [G, N, K]
    const float *sa, *sb;  // [blocks of K, R], [G, blocks of K, blocks of N]
    const int32_t *offsets;
    int64_t G, R, N, K;
    int fa, fb;  // formats
    void *out;
    int *fault;
};
cudaError_t launch_fp8_gemm(const Fp8GemmArgs &a, int out_dtype, cudaStream_t s);

// out [G, M, N] = a[:, segment e] b[:, segment e]^T
struct Fp8WgradArgs {
    const uint8_t *a, *b;  // [M, R], [N, R]
    const float *sa, *sb;  // [blocks of R, M], [blocks of R, N]
    const int32_t *offsets;
    int64_t G, R, M, N;
    int fa, fb;
    void *out;
    int *fault;
};
cudaError_t launch_fp8_wgrad(const Fp8WgradArgs &a, int out_dtype, cudaStream_t s);

// The experts' layer for T tokens of k slots.
struct MoeFewArgs {
    const void *x;  // [T, C]
    const int32_t *ids;
    const float *w;
    const void *w1, *w2;    // [E, 2F, C], [E, C, F]: 16 bits, or e4m3 with scales
    const float *s1, *s2;   // [E, blocks of C, blocks of 2F], [E, blocks of F, blocks of C]
    int64_t T, C, F;
    int k, E;
    void *f;  // [T, C]
    void *ws;
    int *fault;
};
constexpr int kMoeFewTokens = 128;
size_t moe_few_ws_bytes(int64_t T, int k, int64_t CF);  // CF = C + F
constexpr int kMoeFewMaxK = 16384;  // C and F
cudaError_t launch_moe_few(const MoeFewArgs &a, int dtype, int eight, cudaStream_t s);

}  // namespace mhc
