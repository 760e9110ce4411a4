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

}  // namespace tern
