// tern_buffer.h -- buffer loads whose bounds do not depend on a scalar offset.
//
// A raw buffer load reads base + vector offset + scalar offset.  Its bounds
// check compares the vector offset (with an immediate) against the size in the
// descriptor; that the scalar offset takes part in it is not promised.  So the
// scalar offset is 0 in every load: what decides whether a byte is there stands
// in the vector offset, which is one vector addition where it differs between
// the loads of a lane, and a load past the end returns zeros.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tern {

// The vector offset of a load that reads nothing.  Sizes and what is added to it stay below 2^31.
constexpr int OUT_OF_RANGE = (int)0x80000000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000);
}

template <int NT = 0>   // 2: non-temporal, for bytes that are read once
__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, int off) {
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint4, __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, NT)));
}

template <int NT = 0>
__device__ __forceinline__ uint2 load8(__amdgpu_buffer_rsrc_t r, int off) {
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint2, __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, NT)));
}

// Lane l's 16 or 4 bytes at off -> lds + 16 l or 4 l.
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t *lds, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t *lds, int off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 4, off, 0, 0, 0);
}

}  // namespace tern
