// tern_mx.h -- host-side launchers and device helpers of the microscaled 4-bit
// float (e2m1, one power-of-two scale per 32) operators.  Every launcher
// assumes its arguments were validated by tern_api.hip.
//
// Format.  A row of K values is cut into blocks of 32; block b has a biased
// exponent byte e (the scale is 2^(e - 127), 255 means that the block is NaN)
// and 32 4-bit codes [sign, magnitude index] of the magnitudes 0, .5, 1, 1.5,
// 2, 3, 4, 6, two to a byte with the even element in the low nibble.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tern {

struct MxArgs {
    const void *X;        // [M,K] fp16/bf16, or e2m1 codes [M,K/2] (x_dtype 2)
    const uint8_t *XE;    // [M,K/32] exponents of X, x_dtype 2 only
    int x_dtype;          // 0 = fp16, 1 = bf16, 2 = microscaled
    const uint8_t *W;     // [N,K/2]
    const uint8_t *WE;    // [N,K/32]
    void *Y;              // [M,N]
    int y_dtype;          // 0 = fp16, 1 = bf16, 2 = fp32
    int64_t M, N, K;
    hipStream_t stream;
};

// codes / exps of X (x_dtype 0 fp16, 1 bf16, 2 fp32), over blocks = M*K/32.
hipError_t launch_mx_quantize(const void *X, int x_dtype, uint8_t *codes, uint8_t *exps, int64_t blocks,
                              hipStream_t stream);
// W (w_dtype 0 fp16, 1 bf16, 2 fp32) from codes and exps.
hipError_t launch_mx_dequant(const uint8_t *codes, const uint8_t *exps, void *W, int w_dtype, int64_t blocks,
                             hipStream_t stream);
// Product for few rows: waves split K, weights are read once per row chunk.
hipError_t launch_mx_gemv(const MxArgs &a);
// Product for many rows: LDS-staged tiles, and where they are the faster choice.
bool mx_gemm_wins(const MxArgs &a);
hipError_t launch_mx_gemm(const MxArgs &a);

}  // namespace tern
