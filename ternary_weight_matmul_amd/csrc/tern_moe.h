// tern_moe.h -- host-side launcher of the mixture-of-experts layer with ternary
// experts.  It assumes that its arguments were validated by tern_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace tern {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int64_t kMoeChunk = 64;   // tokens of one pass over the experts
constexpr int kMoeSmall = 4;        // tokens up to which two launches do
constexpr int64_t kMoeMaxWidth = 16384;   // H and F: four tokens' operands stay in LDS

struct MoeArgs {
    const void *X;               // [T,H] fp16/bf16
    int x_dtype;                 // 0 = fp16, 1 = bf16
    const void *logits;          // [T,E]
    int l_dtype;                 // 0 = fp16, 1 = bf16, 2 = fp32
    const int *ids;              // [T,top_k] experts with
    const float *weights;        // [T,top_k] weights in place of the logits, or null
    const uint8_t *GU;           // [E,2F,H/4]
    const uint16_t *GUS;         // [E,2F,H/128]
    const uint8_t *D;            // [E,H,F/4]
    const uint16_t *DS;          // [E,H,F/128]
    void *Y;                     // [T,H]
    int y_dtype;                 // 0 = fp16, 1 = bf16, 2 = fp32
    int64_t T, E, top_k, H, F;
    int renormalize;
    void *ws;
    hipStream_t stream;
};

// Bytes of workspace for T tokens (the chunk's pairs: expert ids, weights,
// hidden values and partial outputs).
size_t moe_workspace(int64_t T, int64_t top_k, int64_t H, int64_t F);
hipError_t launch_moe(const MoeArgs &a);

}  // namespace tern
