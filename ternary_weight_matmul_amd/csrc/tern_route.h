// tern_route.h -- host-side launcher of the routing of tokens to experts.  It
// assumes that its arguments were validated by tern_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tern {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
constexpr int kRouteMaxGroups = 64;   // a lane each

struct RouteArgs {
    const void *logits;   // [T,E]
    int l_dtype;          // 0 = fp16, 1 = bf16, 2 = fp32
    const float *bias;    // [E], or null
    int *ids;             // [T,top_k]
    float *weights;       // [T,top_k]
    int64_t T;
    int E, top_k, sigmoid, groups, keep, best, renormalize;
    float scale;
    hipStream_t stream;
};

hipError_t launch_route(const RouteArgs &a);

}  // namespace tern
