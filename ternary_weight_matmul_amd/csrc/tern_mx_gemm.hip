// tern_mx_gemm.hip -- Y[M,N] = X[M,K] . W^T for many rows M, with W in
// microscaled 4-bit floats and X in fp16, bf16 or the same 4-bit form.
//
// Mathematics as in tern_mx_gemv.hip: with 4-bit X both operands enter
// v_mfma_scale_f32_16x16x128_f8f6f4 as they are stored, with their scale
// bytes; with 16-bit X a weight times its scale is an exact bf16, and an fp16
// activation two bf16 terms, for v_mfma_f32_16x16x32_bf16.
//
// Work layout.  A workgroup of WM x WN waves computes BM x BN outputs, BM =
// 16 MB WM, BN = 16 NB WN.  Per step both operands are staged in LDS as they
// are stored: 64 values of a row of X in 128 bytes and the same 64 weights in
// 32, or 256 4-bit values of either in 128 bytes.  They go from memory straight
// to LDS, into one of ST buffers, ST - 1 steps before they are needed: every
// CU misses its XCD's L2 on its first touch of a line, and with two buffers the
// steps waited for memory (2.3 us a step for 0.6 us of matrix instructions
// with 4-bit X).  The weights stay 4-bit in LDS, so that the fragment reads of
// a wave are mostly X's; a wave decodes its own fragments (4 instructions for
// 8 weights, shared by MB matrix instructions).
//
// The rows of the matrix tile are weights and its columns activations: a lane
// then holds 4 consecutive outputs of one row of Y.  Which K indices share a
// matrix instruction does not matter as long as both operands agree: with
// 16-bit X lane group p = lane / 16 takes values 16 p .. 16 p + 15 of the 64,
// half of a block of weights.
//
// LDS rows are XOR-swizzled in 16-byte chunks so that the lanes of a fragment
// read that are served together fall on distinct banks.
//
// Bound: the matrix cores.  M = 2048, 5120 -> 7168, weights rotated over 2 GB:
// bf16 X 146 us, 4-bit X 74, fp16 X 320 (twice the matrix instructions, and
// every wave splits its fragments of X anew).
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "tern_device.h"
#include "tern_mx.h"
#include "tern_mx_device.h"

namespace tern {

namespace {

typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef float float4v_t __attribute__((ext_vector_type(4)));

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

// The order of a step's LDS reads and matrix instructions: the first operands and AHEAD more
// fragments of X are read, then a fragment goes out with every NB matrix instructions, so that
// a read has AHEAD times as long to arrive.  Left to itself the compiler waits for each pair of
// reads right after it issues them.
constexpr int AHEAD = 3;
template <bool MX, int MB, int NB, int TERMS>
__device__ __forceinline__ void interleave() {
    constexpr int DS = 0x100, MFMA = 0x008;
    __builtin_amdgcn_sched_group_barrier(DS, (MX ? MB + 3 * NB : 2 * NB) + AHEAD, 0);
#pragma unroll
    for (int g = 0; g < 2 * MB; ++g) {
        __builtin_amdgcn_sched_group_barrier(MFMA, NB * TERMS, 0);
        __builtin_amdgcn_sched_group_barrier(DS, 1, 0);
    }
}

// 32 4-bit values as the operand of a matrix instruction.
__device__ __forceinline__ int8v_t quarter(const uint8_t *at) {
    const uint4 q = *reinterpret_cast<const uint4 *>(at);
    return (int8v_t){(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

template <int XT, int WM, int WN, int MB, int NB, int ST>
struct Shape {
    static constexpr bool MX = XT == 2;
    static constexpr int WAVES = WM * WN, NT = 64 * WAVES;
    static constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN;
    static constexpr int BPS = MX ? 8 : 2;            // blocks of 32 per step
    static constexpr int XROW = 128;                  // bytes of a row of X per step
    static constexpr int WROW = MX ? 128 : 32;        // and of W
    static constexpr int A_LDS = BM * XROW, W_LDS = BN * WROW;
    static constexpr int AI = (A_LDS / 1024 + WAVES - 1) / WAVES;        // load instructions per wave
    static constexpr int WI = (W_LDS / 1024 + WAVES - 1) / WAVES;
    static constexpr int SROWS = MX ? BM + BN : BN;                      // rows with scale bytes
    static constexpr int SP = (SROWS + NT - 1) / NT;
    static constexpr int S_AT = (AI + WI) * WAVES * 1024;                // where they start
    static constexpr int BUF = S_AT + SP * NT * BPS;                     // every thread stores SP rows, no branch
    static constexpr int CH = 16 / BPS;                                  // steps per 16 scale bytes of a row
    static constexpr int LOADS = AI + WI;                                // tile loads of a wave per step
    static_assert(A_LDS % (1024 * WAVES) == 0 && W_LDS % 1024 == 0, "whole load instructions");
    static_assert(ST >= 2 && ST <= 4 && ST * BUF <= 160 * 1024, "buffers");
    static_assert(!MX || (ST == 2 && BM / 4 <= 64 && BN / 8 <= 64), "touched lines: one instruction, waited for in its step");
    static_assert(ST - 1 <= CH, "the first steps' scales come from one chunk");
    static_assert((ST - 2) * LOADS < 64, "the wait counter has 6 bits");
};

template <int XT, int WM, int WN, int MB, int NB, int ST>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_kernel(const uint8_t *__restrict__ X,
                                                             const uint8_t *__restrict__ XE,
                                                             const uint8_t *__restrict__ W,
                                                             const uint8_t *__restrict__ WE, void *__restrict__ Y,
                                                             int y_dtype, int M, int N, int blocks, int tiles_m,
                                                             int tiles_n, int vec) {
    typedef Shape<XT, WM, WN, MB, NB, ST> T;
    // One variable each, so that the compiler sees that an access to one need not wait for the loads
    // into another.
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::BUF], buf1[T::BUF];
    __shared__ __attribute__((aligned(16))) uint8_t buf2[ST > 2 ? T::BUF : 16], buf3[ST > 3 ? T::BUF : 16];
    __shared__ __attribute__((aligned(16))) uint8_t touched[T::MX ? 512 : 16];   // written, never read
    auto buf = [&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value % ST;
        if constexpr (I == 0) return buf0;
        else if constexpr (I == 1) return buf1;
        else if constexpr (I == 2) return buf2;
        else return buf3;
    };
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int p = lane >> 4, li = lane & 15;

    // Workgroups go round the 8 XCDs: each XCD gets a contiguous run of tiles, which goes down
    // bands of 8 tile rows, so that its 32 CUs share 8 row tiles and 4 column tiles in its L2.
    const int ntiles = tiles_m * tiles_n;
    int tile = blockIdx.x;
    if (ntiles % 8 == 0) tile = (blockIdx.x % 8) * (ntiles / 8) + blockIdx.x / 8;
    const int band = tile / (8 * tiles_n), in = tile - band * 8 * tiles_n, bandm = min(8, tiles_m - band * 8);
    const int m0 = (band * 8 + in % bandm) * T::BM, n0 = in / bandm * T::BN;

    const int xrow = blocks * (T::MX ? 16 : 64), wrow = blocks * 16;
    const int xrows = min(T::BM, M - m0), wrows = min(T::BN, N - n0);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(X + (int64_t)m0 * xrow, xrows * xrow);
    const __amdgpu_buffer_rsrc_t rw = buffer_of(W + (int64_t)n0 * wrow, wrows * wrow);
    const int steps = (blocks + T::BPS - 1) / T::BPS;

    // Tiles go from memory straight to LDS, 16 bytes a lane, 1 KB an instruction.  Rows past the
    // end, chunks past the end of a row in the last step, and instructions past the tile (every
    // wave issues as many) get an offset out of range and arrive as zeros.
    constexpr int XL = T::XROW / 16, WL = T::WROW / 16;   // lanes per row
    const int ar = wave * (64 / XL) + lane / XL, wr = wave * (64 / WL) + lane / WL;
    const int ac = (lane % XL) ^ xor128(ar);
    const int wc = (lane % WL) ^ (T::MX ? xor128(wr) : xor32(wr));
    const int aoff = ar * xrow + ac * 16, woff = wr * wrow + wc * 16;
    auto fetch = [&](uint8_t *to, int s) TERN_INLINE {
        const int left = blocks - s * T::BPS;   // blocks of this step
        const int ao = (ac < left * (T::MX ? 1 : 4) ? aoff : OUT_OF_RANGE) + s * T::XROW;
        const int wo = (wc < left ? woff : OUT_OF_RANGE) + s * T::WROW;
#pragma unroll
        for (int i = 0; i < T::AI; ++i)
            load16_to_lds(rx, to + (i * T::WAVES + wave) * 1024, ao + i * T::WAVES * (64 / XL) * xrow);
#pragma unroll
        for (int i = 0; i < T::WI; ++i)
            load16_to_lds(rw, to + T::A_LDS + (i * T::WAVES + wave) * 1024, wo + i * T::WAVES * (64 / WL) * wrow);
    };

    // With 4-bit X a step is short and its tiles come late: every line is new to the XCD's L2.  So
    // the lines of one step further are touched (4 bytes each, into a corner of LDS), every CU its
    // share of what the band's CUs read together: 4 of them a row tile, 8 a column tile.  Measured
    // at M = 2048, 5120 -> 17408: 140 -> 129 us; with 16-bit X, whose steps are longer, 158 -> 164.
    const bool tx = wave == 0;
    const __amdgpu_buffer_rsrc_t rt = tx ? rx : rw;
    const int tshare = tx ? in / bandm % 4 * (T::BM / 4) : in % bandm * (T::BN / 8);
    const int toff = lane < (tx ? T::BM / 4 : T::BN / 8) ? (tshare + lane) * (tx ? xrow : wrow) : OUT_OF_RANGE;
    auto touch = [&](int s) TERN_INLINE {
        if (T::MX && wave < 2 && s < steps)
            load4_to_lds(rt, touched + wave * 256, toff + s * T::XROW);
    };

    // Scale bytes go through registers, 16 of a row at a time (512 values): a load costs a request
    // to the L2 per row however short it is, and 4 bytes a step were as many requests as the tiles
    // themselves.  A step's bytes are stored just before its tiles are fetched into the same buffer.
    // Places past the end of a row get 127, the scale 1: a stray 255 would make NaN of the zeros
    // there.  Rows have no alignment; a load that would pass the end of the matrix starts earlier and
    // is shifted when it is taken (a matrix has at least 16 scale bytes).
    uint4 scur[T::SP], snext[T::SP];
    const uint8_t *srow[T::SP];   // the row's scale bytes
    int slast[T::SP];             // the last place in it that 16 bytes can be loaded from
#pragma unroll
    for (int i = 0; i < T::SP; ++i) {
        const int r = i * T::NT + tid;
        if (T::MX && r < T::BM) {
            const int64_t row = m0 + min(r, xrows - 1);
            srow[i] = XE + row * blocks;
            slast[i] = (int)min((M - row) * blocks - 16, (int64_t)1 << 30);
        } else {
            const int64_t row = n0 + min(r - (T::MX ? T::BM : 0), wrows - 1);
            srow[i] = WE + row * blocks;
            slast[i] = (int)min((N - row) * blocks - 16, (int64_t)1 << 30);
        }
    }
    auto load_scales = [&](int q) TERN_INLINE {
#pragma unroll
        for (int i = 0; i < T::SP; ++i) __builtin_memcpy(&snext[i], srow[i] + min(q * 16, slast[i]), 16);
    };
    auto take_scales = [&](int q) TERN_INLINE {   // chunk q becomes the current one, q + 1 goes out
#pragma unroll
        for (int i = 0; i < T::SP; ++i) {
            const int sh = 8 * min(max(q * 16 - slast[i], 0), 15);
            uint64_t lo = snext[i].x | (uint64_t)snext[i].y << 32, hi = snext[i].z | (uint64_t)snext[i].w << 32;
            if (sh >= 64) lo = hi, hi = 0;
            if (sh & 63) lo = lo >> (sh & 63) | hi << (64 - (sh & 63)), hi >>= sh & 63;
            scur[i] = make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
        }
        load_scales(q + 1);
    };
    auto store_scales = [&](uint8_t *to, int s) TERN_INLINE {
        const int left = min(max(blocks - s * T::BPS, 0), T::BPS);
        const uint64_t valid = left == 8 ? ~0ull : (1ull << (8 * left)) - 1;
        const int at = s % T::CH;   // its place in the chunk
#pragma unroll
        for (int i = 0; i < T::SP; ++i) {
            const uint4 &c = scur[i];
            const int r = i * T::NT + tid;
            if constexpr (T::MX) {
                const uint64_t v = at ? c.z | (uint64_t)c.w << 32 : c.x | (uint64_t)c.y << 32;
                *reinterpret_cast<uint64_t *>(to + T::S_AT + r * 8) = (v & valid) | (0x7F7F7F7F7F7F7F7Full & ~valid);
            } else {
                const uint32_t v = (at < 2 ? c.x : at < 4 ? c.y : at < 6 ? c.z : c.w) >> 16 * (at & 1);
                *reinterpret_cast<uint16_t *>(to + T::S_AT + r * 2) = (uint16_t)((v & valid) | (0x7F7Fu & ~valid));
            }
        }
    };

    float4v_t acc[NB][MB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[n][m] = (float4v_t){0.f, 0.f, 0.f, 0.f};

    const int arow = wm * 16 * MB + li, wrow0 = wn * 16 * NB + li;
    auto products = [&](const uint8_t *a) TERN_INLINE {
        const uint8_t *w = a + T::A_LDS;
        const uint8_t *sc = a + T::S_AT;
        if constexpr (T::MX) {
            uint32_t as[MB], bs[NB];   // two scale bytes each
            int8v_t bv[2][NB];
#pragma unroll
            for (int m = 0; m < MB; ++m) as[m] = *reinterpret_cast<const uint16_t *>(sc + (arow + 16 * m) * 8 + 2 * p);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                bs[n] = *reinterpret_cast<const uint16_t *>(sc + (T::BM + wrow0 + 16 * n) * 8 + 2 * p);
#pragma unroll
                for (int j = 0; j < 2; ++j) bv[j][n] = quarter(w + swz<T::WROW>(wrow0 + 16 * n, 2 * p + j));
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int8v_t av = quarter(a + swz<T::XROW>(arow + 16 * m, 2 * p + j));
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        // the byte selects are immediates
                        if (j == 0)
                            acc[n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[0][n], av, acc[n][m], 4, 4, 0,
                                                                                         (int)bs[n], 0, (int)as[m]);
                        else
                            acc[n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[1][n], av, acc[n][m], 4, 4, 1,
                                                                                         (int)bs[n], 1, (int)as[m]);
                    }
                }
        } else {
            uint2 code[NB];
            float sf[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                code[n] = *reinterpret_cast<const uint2 *>(w + swz<T::WROW>(wrow0 + 16 * n, p >> 1) + 8 * (p & 1));
                sf[n] = __builtin_bit_cast(float, (uint32_t)sc[(wrow0 + 16 * n) * 2 + (p >> 1)] << 23);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 xv[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m) xv[m] = *reinterpret_cast<const uint4 *>(a + swz<T::XROW>(arow + 16 * m, 2 * p + i));
                bf168_t bv[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) bv[n] = decode8(i ? code[n].y : code[n].x, sf[n]);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    uint4 lo;
                    const uint4 hi = XT == 0 ? fp16_terms(xv[m], lo) : xv[m];
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], __builtin_bit_cast(bf168_t, hi),
                                                                           acc[n][m], 0, 0, 0);
                    if constexpr (XT == 0) {
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], __builtin_bit_cast(bf168_t, lo),
                                                                               acc[n][m], 0, 0, 0);
                    }
                }
            }
        }
    };

    // Step s, in buffer I = s mod ST, fetches step s + ST - 1.  Past the end every offset is out of
    // range; a branch around the fetch would let the compiler move the products behind the wait.
    auto step = [&](auto i, int s) TERN_INLINE {
        constexpr int I = decltype(i)::value;
        constexpr auto fill = std::integral_constant<int, (I + ST - 1) % ST>();
        const int f = s + ST - 1;
        if (ST == T::CH ? fill.value == 0 : f % T::CH == 0) take_scales(f / T::CH);
        touch(f + 1);
        store_scales(buf(fill), f);
        fetch(buf(fill), f);
        __builtin_amdgcn_sched_barrier(0);   // the loads first
        products(buf(i));
        interleave<T::MX, MB, NB, XT == 0 ? 2 : 1>();
        __builtin_amdgcn_sched_barrier(0);   // and the wait last
        wait_and_meet<(ST - 2) * T::LOADS>();   // step s + 1 is there
    };
    auto each = [&](auto f) TERN_INLINE {   // f(0), ..., f(ST - 1) until one returns true
        typedef std::integral_constant<int, 0> I0;
        typedef std::integral_constant<int, 1> I1;
        if (f(I0()) || f(I1())) return true;
        if constexpr (ST > 2)
            if (f(std::integral_constant<int, 2>())) return true;
        if constexpr (ST > 3)
            if (f(std::integral_constant<int, 3>())) return true;
        return false;
    };
    load_scales(0);
    take_scales(0);
    each([&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value;
        if constexpr (I < ST - 1) {
            store_scales(buf(i), I);
            fetch(buf(i), I);
        }
        return false;
    });
    wait_and_meet<0>();
    int s = 0;
    while (!each([&](auto i) TERN_INLINE {
        step(i, s);
        return ++s >= steps;
    })) {
    }

    // lane (p, li): outputs n = 4 p + v of row li of each 16 x 16 block
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int row = m0 + arow + 16 * m, c0 = n0 + wn * 16 * NB + 16 * n + 4 * p;
            if (row >= M) continue;
            const float4v_t &d = acc[n][m];
            const int64_t at = (int64_t)row * N + c0;
            if (vec && c0 + 4 <= N) {
                if (y_dtype == 2) {
                    *reinterpret_cast<float4v_t *>(static_cast<float *>(Y) + at) = d;
                } else if (y_dtype == 1) {
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + at) =
                        make_uint2(bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3]));
                } else {
                    const half2_t a = {(_Float16)d[0], (_Float16)d[1]}, b = {(_Float16)d[2], (_Float16)d[3]};
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(Y) + at) =
                        make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
                }
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (c0 + v < N) {
                        if (y_dtype == 2) store_out<2>(Y, at + v, d[v]);
                        else if (y_dtype == 1) store_out<1>(Y, at + v, d[v]);
                        else store_out<0>(Y, at + v, d[v]);
                    }
            }
        }
}

template <int XT, int WM, int WN, int MB, int NB, int ST>
hipError_t launch_t(const MxArgs &a) {
    typedef Shape<XT, WM, WN, MB, NB, ST> T;
    constexpr auto kern = &mx_gemm_kernel<XT, WM, WN, MB, NB, ST>;
    const int tm = (int)((a.M + T::BM - 1) / T::BM), tn = (int)((a.N + T::BN - 1) / T::BN);
    const size_t unit = a.y_dtype == 2 ? 16 : 8;
    const int vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.Y) % unit == 0;
    hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tn)), dim3(T::NT), 0, a.stream, static_cast<const uint8_t *>(a.X),
                       a.XE, a.W, a.WE, a.Y, a.y_dtype, (int)a.M, (int)a.N, (int)(a.K / 32), tm, tn, vec);
    return hipGetLastError();
}

// Big tiles (256 x 256, with 4-bit X 256 x 192) or small ones (64 x 128).  A step of a big tile takes
// 2.4 times a small one's, 3.4 times when every CU has one (2.6 with 4-bit X, either way), and a CU
// holds one big tile at a time; up to 256 small ones take as long as one.  Measured, K = 5120, us:
//   16-bit X: 512 -> 5120: big 120, small 59; 256 -> 17408: 124, 104; 1024 -> 5120: 122, 95;
//   512 -> 17408: 133, 162.  4-bit X: 44, 28; 48, 45; 43, 36; 50, 64.
// A launch has fewer than 2^32 threads: 2^24 small tiles are too many.
template <int XT>
bool big_tiles(const MxArgs &a) {
    if (((a.M + 63) / 64) * ((a.N + 127) / 128) >= (1 << 24)) return true;
    const double big = (double)((a.M + 255) / 256) * (double)((a.N + (XT == 2 ? 191 : 255)) / (XT == 2 ? 192 : 256)) / 256;
    const double small = (double)((a.M + 63) / 64) * (double)((a.N + 127) / 128) / 256;
    const double step = XT == 2 ? 2.6 : 2.4 + (big < 1 ? big : 1);
    return ceil(big) * step < (small > 1 ? small : 1);
}

template <int XT>
hipError_t launch_x(const MxArgs &a) {
    if constexpr (XT == 2) return big_tiles<XT>(a) ? launch_t<XT, 2, 4, 8, 3, 2>(a) : launch_t<XT, 2, 2, 2, 4, 2>(a);
    else return big_tiles<XT>(a) ? launch_t<XT, 2, 4, 8, 4, 3>(a) : launch_t<XT, 2, 2, 2, 4, 4>(a);
}

}  // namespace

// Up to 32 rows, tiles have nothing to gain; up to 160, while the rows in sixteens times N stay
// small, too few tiles to fill the chip take longer than the weights read once for 16 rows.  Measured,
// K = 5120, us, in sixteens and in tiles: 16-bit X, 128 -> 5120 40 and 45, 64 -> 17408 59 and 49;
// 4-bit X, 64 -> 5120 18 and 25, 128 -> 5120 27 and 23; 37 x 1056 -> 1001: 4 and 13.
// More rows by a narrow W are as few tiles (a router over a prompt).  The border is a product of rows in
// sixteens and N again.  Measured, us: 16-bit X, 200 x 5120 -> 64 5 and 37, 2048 x 1056 -> 128 11.6 and
// 11.1, 1024 x 5120 -> 256 24 and 39, 512 x 5120 -> 1024 42 and 41, 1024 x 17408 -> 16 13 and 118; 4-bit
// X, 200 x 5120 -> 64 5 and 15, 512 x 5120 -> 256 12 and 17, 161 x 1056 -> 1024 5.3 and 6.1, 1024 x 5120
// -> 256 23 and 17.
// Scale bytes are loaded 16 at a time, offsets inside a tile are 32-bit, and so are the columns that a
// tile would have past the last one.  2^23 big tiles are too many threads for a launch.
bool mx_gemm_wins(const MxArgs &a) {
    const int64_t blocks = a.K / 32, chunks = (a.M + 15) / 16;
    const bool mx = a.x_dtype == 2;
    if (a.M <= 32 || chunks * a.N <= (chunks <= 10 ? (mx ? 32768 : 45056) : (mx ? 11264 : 16384))) return false;
    return a.M * blocks >= 16 && a.N * blocks >= 16 && a.K <= (1 << 21) && a.N < INT32_MAX - 256 &&
           ((a.M + 255) / 256) * ((a.N + 191) / 192) < (1 << 23);
}

hipError_t launch_mx_gemm(const MxArgs &a) {
    return a.x_dtype == 0 ? launch_x<0>(a) : (a.x_dtype == 1 ? launch_x<1>(a) : launch_x<2>(a));
}

}  // namespace tern
