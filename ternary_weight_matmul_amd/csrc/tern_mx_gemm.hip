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
// are stored, double-buffered, one barrier a step: 128 bytes of a row of X
// (64 or 256 values), and the same K range of a row of W (32 or 128 bytes).
// The weights stay 4-bit in LDS, so that the fragment reads of a wave are
// mostly X's; a wave decodes its own fragments (4 instructions for 8 weights,
// shared by MB matrix instructions).  The loads of step s + 1 go from memory
// straight to LDS while the products of step s run.
//
// The rows of the matrix tile are weights and its columns activations: a lane
// then holds 4 consecutive outputs of one row of Y.  Which K indices share a
// matrix instruction does not matter as long as both operands agree: lane
// group p = lane / 16 takes the 16-byte chunks 2 p and 2 p + 1 of a row of X,
// so that the scale bytes of a lane's two instructions lie side by side.
//
// LDS rows of 128 bytes have their 16-byte chunks XOR-swizzled by (row / 2)
// mod 8: the 16 lanes of a fragment read fall on 64 distinct banks.
//
// Bound: the matrix cores.
#include <hip/hip_runtime.h>

#include "tern_device.h"
#include "tern_mx.h"
#include "tern_mx_device.h"

namespace tern {

namespace {

typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef float float4v_t __attribute__((ext_vector_type(4)));

constexpr int ROWB = 128;   // bytes of a row of X per step

__device__ __forceinline__ int swz(int r, int c) { return r * ROWB + ((c ^ ((r >> 1) & 7)) << 4); }

// 16-bit X: rows of W are 32 bytes per step, two 16-byte blocks; their places
// alternate every 8 rows, so that the 16 lanes of a read cover all banks.
__device__ __forceinline__ int wswz(int r, int c) { return r * 32 + ((c ^ ((r >> 3) & 1)) << 4); }

constexpr int OUT_OF_RANGE = (int)0x80000000;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint8_t *base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0, bytes, 0x00020000);
}

// Lane l's 16 bytes at r[off + at] -> lds + 16 l; zeros where that is out of range.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, uint8_t *lds, int off, int at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, off, at, 0, 0);
}

// Every load of this wave has arrived (vmcnt 0).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// 32 4-bit values as the operand of a matrix instruction.
__device__ __forceinline__ int8v_t quarter(const uint8_t *at) {
    const uint4 q = *reinterpret_cast<const uint4 *>(at);
    return (int8v_t){(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

template <int XT, int WM, int WN, int MB, int NB>
struct Shape {
    static constexpr bool MX = XT == 2;
    static constexpr int NT = 64 * WM * WN;
    static constexpr int BM = 16 * MB * WM, BN = 16 * NB * WN;
    static constexpr int BPS = MX ? 8 : 2;            // blocks of 32 per step
    static constexpr int WROW = MX ? 128 : 32;        // bytes of a row of W per step
    static constexpr int WAVES = WM * WN;
    static constexpr int A_LDS = BM * ROWB, W_LDS = BN * WROW;
    static constexpr int AI = A_LDS / 1024 / WAVES;                      // load instructions per wave
    static constexpr int WI = (W_LDS / 1024 + WAVES - 1) / WAVES;
    static constexpr int SROWS = MX ? BM + BN : BN;                      // rows with scale bytes
    static constexpr int SP = (SROWS + NT - 1) / NT;
    static constexpr int BUF = A_LDS + W_LDS + SROWS * BPS;
    static_assert(A_LDS % (1024 * WAVES) == 0 && W_LDS % 1024 == 0, "whole load instructions");
    static_assert(WAVES % 2 == 0, "a lane's swizzle must not depend on the instruction");
};

template <int XT, int WM, int WN, int MB, int NB>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_kernel(const uint8_t *__restrict__ X,
                                                             const uint8_t *__restrict__ XE,
                                                             const uint8_t *__restrict__ W,
                                                             const uint8_t *__restrict__ WE, void *__restrict__ Y,
                                                             int y_dtype, int M, int N, int blocks, int tiles_m,
                                                             int tiles_n, int vec) {
    typedef Shape<XT, WM, WN, MB, NB> T;
    // two variables, so that the compiler sees that the reads of one need not wait for the loads into the other
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::BUF];
    __shared__ __attribute__((aligned(16))) uint8_t buf1[T::BUF];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int p = lane >> 4, li = lane & 15;

    // Each XCD takes a contiguous run of tiles (workgroups go round the 8 XCDs).
    const int ntiles = tiles_m * tiles_n;
    int tile = blockIdx.x;
    if (ntiles % 8 == 0) tile = (blockIdx.x % 8) * (ntiles / 8) + blockIdx.x / 8;
    const int m0 = tile / tiles_n * T::BM, n0 = tile % tiles_n * T::BN;

    const int xrow = blocks * (T::MX ? 16 : 64), wrow = blocks * 16;
    const int xrows = min(T::BM, M - m0), wrows = min(T::BN, N - n0);
    const __amdgpu_buffer_rsrc_t rx = rows_of(X + (int64_t)m0 * xrow, xrows * xrow);
    const __amdgpu_buffer_rsrc_t rw = rows_of(W + (int64_t)n0 * wrow, wrows * wrow);
    const uint8_t *xeb = T::MX ? XE + (int64_t)m0 * blocks : nullptr, *web = WE + (int64_t)n0 * blocks;
    const int steps = (blocks + T::BPS - 1) / T::BPS;

    // Tiles go from memory straight to LDS, 16 bytes a lane, 1 KB an instruction: 8 rows of 128
    // bytes, or 32 rows of 32.  Rows past the end, and in the last step the chunks past the end
    // of a row, get an offset out of range and arrive as zeros.
    const int ac = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));   // this lane's chunk (swz)
    const int wc = T::MX ? ac : (lane & 1) ^ ((lane >> 4) & 1);      // (wswz)
    const int aoff = (wave * 8 + (lane >> 3)) * xrow + ac * 16;
    const int woff = (T::MX ? wave * 8 + (lane >> 3) : wave * 32 + (lane >> 1)) * wrow + wc * 16;
    auto fetch = [&](uint8_t *buf, int s) {
        const int left = blocks - s * T::BPS;   // blocks of this step
        const int ao = ac < left * (T::MX ? 1 : 4) ? aoff : OUT_OF_RANGE;
        const int wo = wc < left ? woff : OUT_OF_RANGE;
#pragma unroll
        for (int i = 0; i < T::AI; ++i)
            to_lds(rx, buf + (i * T::WAVES + wave) * 1024, ao, i * T::WAVES * 8 * xrow + s * ROWB);
#pragma unroll
        for (int i = 0; i < T::WI; ++i)
            if (T::W_LDS / 1024 % T::WAVES == 0 || i * T::WAVES + wave < T::W_LDS / 1024)
                to_lds(rw, buf + T::A_LDS + (i * T::WAVES + wave) * 1024, wo,
                       i * T::WAVES * (T::MX ? 8 : 32) * wrow + s * T::WROW);
    };

    // Scale bytes go through registers (rows of blocks bytes have no alignment).  Places past the
    // end get 127, the scale 1: a stray 255 would make NaN of the zeros there.
    uint64_t sr[T::SP];
    auto load_scales = [&](int s) {
        const int left = blocks - s * T::BPS;
#pragma unroll
        for (int i = 0; i < T::SP; ++i) {
            const int r = i * T::NT + tid;
            const uint8_t *e = T::MX && r < T::BM ? xeb + (int64_t)min(r, xrows - 1) * blocks
                                                  : web + (int64_t)min(r - (T::MX ? T::BM : 0), wrows - 1) * blocks;
            e += s * T::BPS;
            if (left >= T::BPS) {
                sr[i] = 0;
                __builtin_memcpy(&sr[i], e, T::BPS);
            } else {
                sr[i] = 0x7F7F7F7F7F7F7F7Full;
                for (int b = 0; b < left; ++b) sr[i] ^= (uint64_t)(e[b] ^ 127) << (8 * b);
            }
        }
    };
    auto store_scales = [&](uint8_t *buf) {
        uint8_t *sc = buf + T::A_LDS + T::W_LDS;
#pragma unroll
        for (int i = 0; i < T::SP; ++i) {
            const int r = i * T::NT + tid;
            if (T::SROWS % T::NT == 0 || r < T::SROWS) {
                if constexpr (T::MX) *reinterpret_cast<uint64_t *>(sc + r * 8) = sr[i];
                else *reinterpret_cast<uint16_t *>(sc + r * 2) = (uint16_t)sr[i];
            }
        }
    };

    float4v_t acc[NB][MB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[n][m] = (float4v_t){0.f, 0.f, 0.f, 0.f};

    const int arow = wm * 16 * MB + li, wrow0 = wn * 16 * NB + li;
    auto products = [&](const uint8_t *a) {
        const uint8_t *w = a + T::A_LDS, *sc = w + T::W_LDS;
        if constexpr (T::MX) {
            uint32_t as[MB], bs[NB];
#pragma unroll
            for (int m = 0; m < MB; ++m) as[m] = *reinterpret_cast<const uint16_t *>(sc + (arow + 16 * m) * 8 + 2 * p);
#pragma unroll
            for (int n = 0; n < NB; ++n)
                bs[n] = *reinterpret_cast<const uint16_t *>(sc + (T::BM + wrow0 + 16 * n) * 8 + 2 * p);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int8v_t bv[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) bv[n] = quarter(w + swz(wrow0 + 16 * n, 2 * p + j));
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int8v_t av = quarter(a + swz(arow + 16 * m, 2 * p + j));
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        // the byte selects are immediates
                        if (j == 0)
                            acc[n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[n], av, acc[n][m], 4, 4, 0,
                                                                                         (int)bs[n], 0, (int)as[m]);
                        else
                            acc[n][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bv[n], av, acc[n][m], 4, 4, 1,
                                                                                         (int)bs[n], 1, (int)as[m]);
                    }
                }
                if (j == 0) __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            uint2 code[NB];
            float sf[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                code[n] = *reinterpret_cast<const uint2 *>(w + wswz(wrow0 + 16 * n, p >> 1) + 8 * (p & 1));
                sf[n] = __builtin_bit_cast(float, (uint32_t)sc[(wrow0 + 16 * n) * 2 + (p >> 1)] << 23);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint4 xv[MB];
#pragma unroll
                for (int m = 0; m < MB; ++m) xv[m] = *reinterpret_cast<const uint4 *>(a + swz(arow + 16 * m, 2 * p + i));
                bf168_t bv[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) bv[n] = decode8(i ? code[n].y : code[n].x, sf[n]);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const bf168_t hi = __builtin_bit_cast(bf168_t, XT == 0 ? fp16_term(xv[m], false) : xv[m]);
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], hi, acc[n][m], 0, 0, 0);
                    if constexpr (XT == 0) {
                        const bf168_t lo = __builtin_bit_cast(bf168_t, fp16_term(xv[m], true));
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            acc[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[n], lo, acc[n][m], 0, 0, 0);
                    }
                }
            }
        }
    };

    // One step: the products of `now` while `next` fills.
    auto step = [&](uint8_t *now, uint8_t *next, int s) {
        const bool more = s + 1 < steps;
        if (more) {
            fetch(next, s + 1);
            load_scales(s + 1);
        }
        products(now);
        if (more) store_scales(next);
        wait_loads();
        __syncthreads();
    };
    fetch(buf0, 0);
    load_scales(0);
    store_scales(buf0);
    wait_loads();
    __syncthreads();
    for (int s = 0;;) {
        step(buf0, buf1, s);
        if (++s >= steps) break;
        step(buf1, buf0, s);
        if (++s >= steps) break;
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

template <int XT, int WM, int WN, int MB, int NB>
hipError_t launch_t(const MxArgs &a) {
    typedef Shape<XT, WM, WN, MB, NB> T;
    constexpr auto kern = &mx_gemm_kernel<XT, WM, WN, MB, NB>;
    const int tm = (int)((a.M + T::BM - 1) / T::BM), tn = (int)((a.N + T::BN - 1) / T::BN);
    const size_t unit = a.y_dtype == 2 ? 16 : 8;
    const int vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.Y) % unit == 0;
    hipLaunchKernelGGL(kern, dim3((unsigned)(tm * tn)), dim3(T::NT), 0, a.stream, static_cast<const uint8_t *>(a.X),
                       a.XE, a.W, a.WE, a.Y, a.y_dtype, (int)a.M, (int)a.N, (int)(a.K / 32), tm, tn, vec);
    return hipGetLastError();
}

template <int XT>
hipError_t launch_x(const MxArgs &a) {
    if (a.M > 128) {
        if constexpr (XT == 2) return launch_t<XT, 2, 4, 8, 4>(a);
        else return launch_t<XT, 2, 4, 8, 4>(a);   // 256 x 256
    }
    return launch_t<XT, 2, 2, 2, 4>(a);                  // 64 x 128
}

}  // namespace

// Offsets inside a tile are 32-bit, tiles are counted in an int.
bool mx_gemm_fits(const MxArgs &a) {
    return a.K <= (1 << 21) && ((a.M + 63) / 64) * ((a.N + 63) / 64) < (int64_t(1) << 31);
}

hipError_t launch_mx_gemm(const MxArgs &a) {
    return a.x_dtype == 0 ? launch_x<0>(a) : (a.x_dtype == 1 ? launch_x<1>(a) : launch_x<2>(a));
}

}  // namespace tern
