// tern_mx_device.h -- device helpers shared by the products with microscaled
// 4-bit weights.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_buffer.h"
#include "tern_device.h"
#include "tern_launch.h"

namespace tern {

typedef __bf16 bf168_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const bf162_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// The two bf16 terms of 8 fp16 values, hi (returned) and lo.  lo is the last 3 significant bits of
// the value, hi the rest: hi + lo is the value exactly.  An infinity leaves inf - inf behind, which
// the maximum replaces by a number (it returns the operand that is one): the infinity is in hi
// alone.  A NaN makes hi a NaN.
__device__ __forceinline__ uint4 fp16_terms(const uint4 &q, uint4 &lo) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const half2_t least = {(_Float16)-65504.f, (_Float16)-65504.f};
    uint32_t h[4], l[4];
    // the upper halves of two fp32: exact, both terms have 8 significant bits at most
    auto pair = [](float a, float b) {
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
    };
    float one = 1.f;   // hidden, for a multiply-add that takes 16-bit operands: no conversion of v - d
    asm("" : "+s"(one));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const half2_t v = __builtin_bit_cast(half2_t, w[i]), t = __builtin_bit_cast(half2_t, w[i] & 0xFFF8FFF8u);
        const half2_t d = __builtin_elementwise_max(v - t, least);
        h[i] = pair(fmaf((float)v[0], one, -(float)d[0]), fmaf((float)v[1], one, -(float)d[1]));
        l[i] = pair((float)d[0], (float)d[1]);
    }
    lo = make_uint4(l[0], l[1], l[2], l[3]);
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// 8 e2m1 codes -> 8 bf16 values times the scale s (exact: two significant bits).
__device__ __forceinline__ bf168_t decode8(uint32_t c, float s) {
    uint32_t w[4];
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    return __builtin_bit_cast(bf168_t, make_uint4(w[0], w[1], w[2], w[3]));
}

}  // namespace tern
