// tern_q8.h -- host-side launchers of the root-mean-square norm and of the 8-bit
// activations: their conversion and their product with ternary weights.  Every
// launcher assumes that its arguments were validated by tern_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tern {

constexpr int64_t kNormMaxK = 65536;   // a row is one workgroup's

struct NormArgs {
    const void *X;      // [M,K]
    int x_dtype;        // 0 = fp16, 1 = bf16, 2 = fp32
    const void *R;      // [M,K] residual, or null
    int r_dtype;
    const void *W;      // [K] weights, or null: ones
    int w_dtype;
    void *H;            // [M,K] in r_dtype: the sum, with R only
    void *Y;            // [M,K] normed values, or null
    int y_dtype;
    int8_t *Q;          // [M,K] codes, or null
    float *S;           // their scales: [M], or [M,K/128] where grouped is not 0
    int grouped;
    int normalize;      // 0: the codes of x itself
    int64_t M, K;
    float eps;
    hipStream_t stream;
};

hipError_t launch_norm(const NormArgs &a);

// Y (0 fp16, 1 bf16, 2 fp32) = codes * scales, a scale per row of K.
hipError_t launch_q8_dequant(const int8_t *Q, const float *S, void *Y, int y_dtype, int64_t M, int64_t K,
                             hipStream_t stream);

struct Q8Args {
    const int8_t *Q;     // [M,K]
    const float *XS;     // [M], or [M,K/128] where grouped is not 0
    int grouped;
    const uint8_t *W;    // [N,K/4]
    const uint16_t *S;   // [N,K/128] fp16 bits
    void *Y;             // [M,N]
    int y_dtype;         // 0 = fp16, 1 = bf16, 2 = fp32
    int64_t M, N, K;
    void *terms;         // workspace of launch_q8_gemm, and what it puts there
    const float *w_scales, *x_scales;
    hipStream_t stream;
};

// Products.  Few rows: waves split K, and each 32 rows read the weights.
bool q8_rows_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_q8_rows(const Q8Args &a);
// Tiles of 64 x 128 outputs.
hipError_t launch_q8_blocks(const Q8Args &a);
// Tiles of 128 x 384; the workspace that they need.
size_t q8_gemm_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_q8_gemm(const Q8Args &a);
// What each takes, about, in us.
double q8_rows_time(int64_t M, int64_t N, int64_t K);
double q8_blocks_time(int64_t M, int64_t N, int64_t K);
double q8_gemm_time(int64_t M, int64_t N, int64_t K);

}  // namespace tern
