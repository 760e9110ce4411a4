// tern_tile.h -- LDS tiles of the products with many rows that go from memory
// straight to LDS: where the 16-byte chunks of a row lie, and the wait that ends
// a step.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tern {

// A 16-byte read of the wave is served in groups of lanes such as 0-3, 12-15, 20-27: rows 0-3
// and 12-15 of one lane group p and 4-11 of the next.  Their 16 chunks have to fall on distinct
// places of 256 bytes.
//
// Rows of 128 bytes, chunks 2 p (+ 1): the row pair h = (row / 2) mod 8, rotated left by a bit,
// is XORed in (h itself made every read a two-way conflict).
__device__ __forceinline__ int xor128(int row) { return ((row & 6) | ((row >> 3) & 1)) & 7; }
// Rows of 32 bytes, read 8 bytes a lane.
__device__ __forceinline__ int xor32(int row) { return (row >> 3) & 1; }

template <int ROWB>
__device__ __forceinline__ int swz(int row, int c) {
    return row * ROWB + ((c ^ (ROWB == 128 ? xor128(row) : xor32(row))) << 4);
}

// Lambdas of the kernel: left as calls, their captures live in scratch memory.
#define TERN_INLINE __attribute__((always_inline))

// At most LATER loads of this wave are still on their way, its LDS accesses are done, and every
// wave of the workgroup has got here.  In one piece: __syncthreads would wait for every load.
template <int LATER>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
}

// Loads that go to LDS without the compiler's knowledge.  It waits for those that it knows of where a
// loop begins anew, for all of them, whatever was asked for last; these are waited for by
// wait_and_meet alone, which every access to what they write must follow.  They have no registers to
// write, and `memory` keeps LDS accesses on their sides.  m0 is theirs: the compiler reserves it, and
// sets it anew for each instruction of its own that reads it.
typedef int tile_int4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ tile_int4 descriptor(const void *base, int bytes) {   // as buffer_of's
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    return (tile_int4){__builtin_amdgcn_readfirstlane((int)b), __builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF),
                       __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_of(const void *p) {   // a pointer into LDS as the offset there
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// Lane l's 16 or 4 bytes at off -> LDS offset lds + 16 l or 4 l.
__device__ __forceinline__ void to_lds16(tile_int4 r, uint32_t lds, int off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r) : "memory");
}
__device__ __forceinline__ void to_lds4(tile_int4 r, uint32_t lds, int off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r) : "memory");
}

}  // namespace tern
