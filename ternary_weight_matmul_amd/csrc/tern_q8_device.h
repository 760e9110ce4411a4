// tern_q8_device.h -- ternary weights as 8-bit operands, shared by the products
// with 8-bit activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_buffer.h"
#include "tern_device.h"

namespace tern {

typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef float float4v_t __attribute__((ext_vector_type(4)));

// In both words of x, the fields under MASK change places with those S bits above them.
template <int S, uint32_t MASK>
__device__ __forceinline__ void swap_fields(uint64_t &x) {
    const uint64_t y = x >> S;
    uint32_t lo = (uint32_t)x, hi = (uint32_t)(x >> 32);
    const uint32_t t0 = __builtin_amdgcn_bitop3_b32(lo, (uint32_t)y, MASK, (0xF0 ^ 0xCC) & 0xAA);
    const uint32_t t1 = __builtin_amdgcn_bitop3_b32(hi, (uint32_t)(y >> 32), MASK, (0xF0 ^ 0xCC) & 0xAA);
    const uint64_t z = (t0 | (uint64_t)t1 << 32) << S;
    lo = __builtin_amdgcn_bitop3_b32(lo, t0, (uint32_t)z, 0xF0 ^ 0xCC ^ 0xAA);
    hi = __builtin_amdgcn_bitop3_b32(hi, t1, (uint32_t)(z >> 32), 0xF0 ^ 0xCC ^ 0xAA);
    x = lo | (uint64_t)hi << 32;
}

// 32 codes (two words of 16) -> 32 int8 in {-1, 0, +1} in their own order, which is that of the
// activations' bytes in memory: no byte of those is moved anywhere.
//
// A word is a 4 x 4 matrix of 2-bit fields, byte j and place i in it for weight 4 j + i.  A shift
// and a mask take one place of all bytes, weights i, 4 + i, 8 + i, 12 + i; so the matrix is
// transposed first, two swaps of off-diagonal fields (quarters, then within them), after which
// they are weights 4 i .. 4 i + 3.  A byte permutation then looks each code up in {0, 1, -1, 0}.
__device__ __forceinline__ void decode32(uint64_t x, int4v_t &a, int4v_t &b) {
    swap_fields<6, 0x00CC00CCu>(x);    // fields 1 and 3 of the even bytes with 0 and 2 of the odd ones
    swap_fields<12, 0x0000F0F0u>(x);   // fields 2 and 3 of the lower half with 0 and 1 of the upper one
    constexpr uint32_t VALUES = 0x00FF0100u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t f = (x >> (2 * i)) & 0x0303030303030303ull;
        a[i] = (int)__builtin_amdgcn_perm(0u, VALUES, (uint32_t)f);
        b[i] = (int)__builtin_amdgcn_perm(0u, VALUES, (uint32_t)(f >> 32));
    }
}

__device__ __forceinline__ int4v_t mfma_i8(const int4v_t &a, const int4v_t &b, const int4v_t &c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// `count` of 4 consecutive outputs from index `at` on; vec: all 4 at once where they are there.
__device__ __forceinline__ void store4(void *Y, int y_dtype, int64_t at, const float4v_t &d, int count, int vec) {
    if (vec && count == 4) {
        if (y_dtype == 2) {
            *reinterpret_cast<float4v_t *>(static_cast<float *>(Y) + at) = d;
        } else if (y_dtype == 1) {
            const bf162_t a = {(__bf16)d[0], (__bf16)d[1]}, b = {(__bf16)d[2], (__bf16)d[3]};
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + at) =
                make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
        } else {
            const half2_t a = {(_Float16)d[0], (_Float16)d[1]}, b = {(_Float16)d[2], (_Float16)d[3]};
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + at) =
                make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (v < count) {
            if (y_dtype == 2) store_out<2>(Y, at + v, d[v]);
            else if (y_dtype == 1) store_out<1>(Y, at + v, d[v]);
            else store_out<0>(Y, at + v, d[v]);
        }
}

}  // namespace tern
