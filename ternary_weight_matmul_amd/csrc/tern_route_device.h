// tern_route_device.h -- what the routing kernels share: logits, keys in the order
// of values, and maxima over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_device.h"

namespace tern {

__device__ __forceinline__ float load_logit(const void *l, int dtype, int64_t i) {
    if (dtype == 2) return static_cast<const float *>(l)[i];
    if (dtype == 1) return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(l)[i] << 16);
    return f16_bits_to_float(static_cast<const uint16_t *>(l)[i]);
}

// Unsigned key in the order of the values, never 0: NaN above all, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v != v ? __builtin_bit_cast(float, 0x7FC00000u) : v + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, (k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// Maximum over the wave, the same for every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<0x128>(v));   // rotations within rows of 16
    v = max(v, dpp<0x124>(v));
    v = max(v, dpp<0x122>(v));
    v = max(v, dpp<0x121>(v));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    auto lane_of = [&](int l) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    };
    return (lane_of(0) + lane_of(16)) + (lane_of(32) + lane_of(48));
}

// The same for 64 bits.
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v != v ? __builtin_nan("") : v + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    const uint32_t hi = wave_max((uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

}  // namespace tern
