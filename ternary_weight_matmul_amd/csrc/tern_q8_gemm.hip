// tern_q8_gemm.hip -- Y[M,N] = X . (T*S)^T for many rows M, with X in 8 bits with
// scales and ternary weights.
//
// Mathematics.  X[m,k] = q[m,k] s[m] (a scale per row) or q[m,k] s[m,k/128]; the
// weights t are -1, 0 or +1 with a scale S[n,k/128].  So
//   Y[m,n] = sum over blocks g of 128:  s[m,g] S[n,g] * sum over k in g of q t
// The inner sums are integers of up to 2^14.  A code is split by its magnitude,
// q = 16 a + b with both terms of its sign, |a| <= 8 and |b| <= 15.  As 6-bit floats
// they enter v_mfma_f32_32x32x64_f8f6f4 against the weights as 4-bit floats +-2 / 0:
// b / 8 as e2m3, whose codes 0 .. 15 are the multiples 0 .. 15 of 1/8, and 2 a, 16
// times that unit, as e3m2.  Products and sums are exact, and arrive as fp32: the
// integer instruction takes as long for one term as this one for two (4.5 against 8.6
// * 10^15 operations a second, measured), but its sums have to be converted, and its
// operand takes three times as many instructions to decode.  (The 16x16 forms of both
// run at half the rate.)
//
// Two kernels.  The first splits X, once, and leaves its terms in the workspace in
// the order in which the second reads them: for each 32 rows and each block of 128 k,
// the 24 operand registers of the 64 lanes.  Lane (h, i) = (lane / 32, lane % 32) has
// row i, k 64 h .. 64 h + 63.  It also turns the scales round, fp32, 64 rows' for a
// block side by side, so that all that the second kernel loads in its loop goes
// straight to LDS: a load to registers would be waited for behind every tile that
// was asked for before it.
//
// Work layout of the second.  A workgroup of WM x WN waves computes BM x BN outputs,
// BM = 32 MB WM, BN = 32 NB WN.  A step is one block of 128: the terms of BM rows of
// X, 192 bytes each, and the codes of BN weight rows, 32 bytes each, go from memory
// straight to LDS, into one of ST buffers, ST - 1 steps before they are needed (a
// line that comes from HBM takes 2 us).  X has the rows of the matrix tile, the
// weights its columns: a lane holds 16 rows of one column and needs one weight scale.
// A tile's sums are scaled while the next one's matrix instructions run.
//
// Bound: the issue of 2 waves a SIMD.  A wave's step has 24 matrix and 161 vector
// instructions, 96 of which scale its sums, of 32 and 4 cycles: 1.5 and 1.3 thousand
// cycles for both waves, of 2.0 GHz under this load, against 3.0 measured; loads
// alone take 0.6 us a step, products alone 0.7, both 1.4.  2048 x 5120 -> 17408: 212
// us, 1.7 * 10^15 operations a second, 12 of them for the first kernel (222 with 193
// vector instructions: offsets of loads counted up in vector registers, halves of
// operands moved together, codes decoded in 64-bit shifts).  Reading operands half a
// step ahead of their use, and decoding between the products, changed nothing.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "tern_fp4.h"
#include "tern_q8.h"
#include "tern_q8_device.h"
#include "tern_tile.h"

namespace tern {

namespace {

typedef float float16v_t __attribute__((ext_vector_type(16)));
typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef int int2v_t __attribute__((ext_vector_type(2)));

constexpr int T_ROWS = 32;            // rows whose terms lie together
constexpr int T_BLOCK = 6 * 1024;     // bytes of their terms of one block: [4][lane][16], then [4][lane][8]

// Both 6-bit terms of 4 codes, a byte each: 2 a as e3m2 (0, 2, 4, 6, ... are the codes 0, 16, 20, 22,
// 24, 25, 26, 27, 28) and b / 8 as e2m3.
__device__ __forceinline__ void terms4(uint32_t x, uint32_t &a, uint32_t &b) {
    const uint32_t neg = (x >> 7) & 0x01010101u, mag = (x ^ (neg * 255u)) + neg;   // -128 has the magnitude 128
    a = __builtin_amdgcn_perm(0x1B1A1918u, 0x16141000u, (mag >> 4) & 0x07070707u) | ((mag >> 7) & 0x01010101u) * 28u | neg << 5;
    b = (mag & 0x0F0F0F0Fu) | neg << 5;
}

// 32 6-bit codes, 4 to a word, in the order of the weights' decoding (fp4_weights: evens of the
// first 16, odds, evens and odds of the others), as 6 registers.
__device__ __forceinline__ void pack6(const uint32_t (&c)[8], uint32_t *r) {
    uint64_t d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[i] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t w = c[4 * (i >> 1) + k] >> (8 * (i & 1));
            d[i] |= (uint64_t)((w & 0x3Fu) | ((w >> 10) & 0xFC0u)) << (12 * k);
        }
    }
    r[0] = (uint32_t)d[0];
    r[1] = (uint32_t)(d[0] >> 32) | (uint32_t)d[1] << 16;
    r[2] = (uint32_t)(d[1] >> 16);
    r[3] = (uint32_t)d[2];
    r[4] = (uint32_t)(d[2] >> 32) | (uint32_t)d[3] << 16;
    r[5] = (uint32_t)(d[3] >> 16);
}

// Terms of 32 rows' block u, by one wave.
__device__ __forceinline__ void split_terms(const int8_t *Q, char *out, int M, int groups, int64_t u, int lane) {
    const int h = lane >> 5, i = lane & 31;
    const int64_t row = u / groups * T_ROWS + i;
    const int g = (int)(u % groups);
    uint32_t r[24];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
        if (row < M) {
            const uint4 *at = reinterpret_cast<const uint4 *>(Q + (row * groups + g) * 128 + 64 * h + 32 * j);
            v0 = at[0], v1 = at[1];
        }
        const uint32_t x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) terms4(x[k], a[k], b[k]);
        pack6(a, r + 12 * j);
        pack6(b, r + 12 * j + 6);
    }
    char *at = out + u * T_BLOCK;
#pragma unroll
    for (int c = 0; c < 4; ++c) {   // a, b of the first half, a, b of the second
        *reinterpret_cast<uint4 *>(at + c * 1024 + lane * 16) = make_uint4(r[6 * c], r[6 * c + 1], r[6 * c + 2], r[6 * c + 3]);
        *reinterpret_cast<uint2 *>(at + 4096 + c * 512 + lane * 8) = make_uint2(r[6 * c + 4], r[6 * c + 5]);
    }
}

// Scales of 64 rows, 8 blocks of each, by one wave: S[rows, groups] (fp16 or fp32) times 4 or 1 ->
// out[rows / 64][groups][64].
constexpr int S_ROWS = 64;
template <bool F32>
__device__ __forceinline__ void turn_scales(const void *S, float *out, int rows, int groups, int64_t u, int lane) {
    const int pieces = (groups + 7) / 8;
    const int64_t block = u / pieces;
    const int g0 = (int)(u % pieces) * 8;
    const int64_t row = block * S_ROWS + lane < rows ? block * S_ROWS + lane : rows - 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int g = g0 + j;
        if (g >= groups) break;
        const int64_t at = row * groups + g;
        // 4: the units of terms and weights are 1/8 and 2
        const float f = F32 ? static_cast<const float *>(S)[at] : 4.f * f16_bits_to_float(static_cast<const uint16_t *>(S)[at]);
        out[(block * groups + g) * S_ROWS + lane] = f;
    }
}

// Waves: the terms' blocks, then the weights' and the activations' scales.
__global__ __launch_bounds__(256) void q8_layout_kernel(const int8_t *__restrict__ Q, const uint16_t *__restrict__ S,
                                                        const float *__restrict__ XS, char *__restrict__ terms,
                                                        float *__restrict__ w_scales, float *__restrict__ x_scales, int M,
                                                        int N, int groups, int64_t t_units, int64_t w_units, int64_t units) {
    const int lane = threadIdx.x & 63;
    const int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (u < t_units) split_terms(Q, terms, M, groups, u, lane);
    else if (u < t_units + w_units) turn_scales<false>(S, w_scales, N, groups, u - t_units, lane);
    else if (u < units) turn_scales<true>(XS, x_scales, M, groups, u - t_units - w_units, lane);
}

// 16 codes a word -> their +-2 / 0 as 4-bit floats, the odd ones in the second word of each pair: sign
// and nonzero bit, 5 instructions.
__device__ __forceinline__ uint4 weights_of(uint32_t a, uint32_t b) {
    const uint32_t u = __builtin_amdgcn_bitop3_b32(a, a >> 1, 0x55555555u, 0xF0 ^ (0xCC & 0xAA));
    const uint32_t v = __builtin_amdgcn_bitop3_b32(b, b >> 1, 0x55555555u, 0xF0 ^ (0xCC & 0xAA));
    return make_uint4((u << 2) & 0xCCCCCCCCu, u & 0xCCCCCCCCu, (v << 2) & 0xCCCCCCCCu, v & 0xCCCCCCCCu);
}

template <int WM, int WN, int MB, int NB, int ST, bool GX>
struct Shape {
    static constexpr int WAVES = WM * WN, NT = 64 * WAVES, BM = 32 * MB * WM, BN = 32 * NB * WN;
    static constexpr int A_LDS = BM * 192, W_LDS = BN * 64;         // the terms of a step, the codes of two
    static constexpr int XI = A_LDS / 1024 / WAVES, WI = W_LDS / 1024 / WAVES;   // load instructions of a wave
    static constexpr int S_AT = A_LDS;                              // the weights' scales, fp32
    static constexpr int X_AT = S_AT + BN * 4;                      // GX: those of the activations
    static constexpr int BUF = X_AT + (GX ? BM * 4 : 0);
    static constexpr int ROW = 32 * NB + 4, OUT = 32 * ROW * 4;     // floats of a row, bytes of a wave's tiles on their way out
    static constexpr int PER = BUF / OUT;                           // waves whose tiles fit a buffer
    static constexpr int LOADS = XI + (GX ? 2 : 1);                 // of a wave a step: terms and scales
    static constexpr int SB = BN / S_ROWS, XB = BM / S_ROWS;        // blocks of scales
    static_assert(A_LDS % (1024 * WAVES) == 0 && W_LDS % (1024 * WAVES) == 0, "whole load instructions");
    static_assert(ST == 4 && ST * BUF + 2 * W_LDS <= 160 * 1024, "buffers");
    static_assert(BN % S_ROWS == 0 && BM % S_ROWS == 0 && SB <= WAVES && XB <= WAVES, "scales");
    static_assert(WAVES <= ST * PER, "outputs");
    static_assert(2 * LOADS + WI < 64, "the wait counter has 6 bits");
};

template <int WM, int WN, int MB, int NB, int ST, bool GX>
__global__ __launch_bounds__(64 * WM * WN, 2) void q8_gemm_kernel(Q8Args a, int tiles_m, int tiles_n, int vec) {
    typedef Shape<WM, WN, MB, NB, ST, GX> T;
    // One variable each, so that the compiler sees that an access to one need not wait for the loads
    // into another.
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::BUF], buf1[T::BUF], buf2[T::BUF], buf3[T::BUF];
    __shared__ __attribute__((aligned(16))) uint8_t codes0[T::W_LDS], codes1[T::W_LDS];
    auto codes = [&](auto i) TERN_INLINE {   // of step i
        if constexpr ((decltype(i)::value / 2 & 1) == 0) return codes0;
        else return codes1;
    };
    auto buf = [&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value % ST;
        if constexpr (I == 0) return buf0;
        else if constexpr (I == 1) return buf1;
        else if constexpr (I == 2) return buf2;
        else return buf3;
    };
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    const int h = lane >> 5, li = lane & 31;
    const int M = (int)a.M, N = (int)a.N, K = (int)a.K, groups = K >> 7;

    // Workgroups go round the 8 XCDs: each XCD gets a contiguous run of tiles, which goes down
    // bands of 8 tile rows, so that its 32 CUs share 8 row tiles and 4 column tiles in its L2.
    const int ntiles = tiles_m * tiles_n;
    int tile = blockIdx.x;
    if (ntiles % 8 == 0) tile = (blockIdx.x % 8) * (ntiles / 8) + blockIdx.x / 8;
    const int band = tile / (8 * tiles_n), in = tile - band * 8 * tiles_n, bandm = min(8, tiles_m - band * 8);
    const int m0 = __builtin_amdgcn_readfirstlane((band * 8 + in % bandm) * T::BM);
    const int n0 = __builtin_amdgcn_readfirstlane(in / bandm * T::BN);

    const int wrow = K >> 2, wrows = min(T::BN, N - n0);
    const int xband = groups * T_BLOCK;   // bytes of 32 rows' terms
    const int sblock = wave % T::SB, xblock = wave % T::XB, sband = groups * S_ROWS * 4;
    const char *const rx = static_cast<const char *>(a.terms) + (int64_t)(m0 / T_ROWS) * xband;
    const uint8_t *const rw = a.W + (int64_t)n0 * wrow;
    const float *const rs = a.w_scales + (int64_t)min(n0 / S_ROWS + sblock, (N - 1) / S_ROWS) * (groups * S_ROWS);
    const float *const rxs = GX ? a.x_scales + (int64_t)min(m0 / S_ROWS + xblock, (M - 1) / S_ROWS) * (groups * S_ROWS) : nullptr;
    // What step s reads of `bytes` from base: the step moves the descriptor, in scalar registers, and
    // the offsets of a lane stay as they are.  Its range ends where the bytes end: rows past the last one
    // are out of it, and so is the second step of a last pair that has none; steps past the end have
    // nothing in range.
    auto of_step = [&](const void *base, int s, int each, int bytes) TERN_INLINE {
        return descriptor(static_cast<const char *>(base) + (int64_t)s * each, s < groups ? bytes - s * each : 0);
    };

    // 16 bytes a lane, 1 KB an instruction: a sixth of 32 rows' terms, or 64 bytes, two steps, of 16 rows
    // of codes (32 bytes of 32 rows took twice as long as as many terms); 4 bytes a lane of scales, which
    // some waves load once more, so that all of them issue and count as many.  Rows past the end, and
    // steps past it, get an offset out of range and arrive as zeros.
    int xoff[T::XI], woff[T::WI];
#pragma unroll
    for (int i = 0; i < T::XI; ++i) {
        const int at = wave * T::XI + i;
        xoff[i] = at / 6 * xband + at % 6 * 1024 + lane * 16;
    }
#pragma unroll
    for (int i = 0; i < T::WI; ++i) {
        const int row = (wave * T::WI + i) * 16 + (lane >> 2);
        woff[i] = row * wrow + (((lane & 3) ^ ((row >> 2) & 3)) << 4);
    }
    auto fetch_terms = [&](uint32_t to, int s, int i) TERN_INLINE {   // and scales, load i of LOADS
        if (i < T::XI)
            to_lds16(of_step(rx, s, T_BLOCK, T::BM / T_ROWS * xband), to + (wave * T::XI + i) * 1024, xoff[i < T::XI ? i : 0]);
        else if (i == T::XI)
            to_lds4(of_step(rs, s, S_ROWS * 4, sband), to + T::S_AT + sblock * 256, lane * 4);
        else
            to_lds4(of_step(rxs, s, S_ROWS * 4, sband), to + T::X_AT + xblock * 256, lane * 4);
    };
    auto fetch_codes = [&](uint32_t to, int s, int i) TERN_INLINE {   // of steps s and s + 1
        to_lds16(of_step(rw, s, 32, wrows * wrow), to + (wave * T::WI + i) * 1024, woff[i]);
    };

    float16v_t acc[MB][NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[m][n][v] = 0.f;

    auto mfma = [&](const int4v_t &q0, const int2v_t &q1, const uint4 &w, const float16v_t &c, auto format) TERN_INLINE {
        const int8v_t av = {q0[0], q0[1], q0[2], q0[3], q1[0], q1[1], 0, 0};
        const int8v_t bv = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, decltype(format)::value, 4, 0, 0, 0, 0);
    };
    typedef std::integral_constant<int, 3> E3M2;
    typedef std::integral_constant<int, 2> E2M3;
    // The tiles of step s; between them load(0), load(1), ...: at the start of the step they would queue
    // up, and the waves with them.
    auto products = [&](auto i, auto load) TERN_INLINE {
        const uint8_t *b = buf(i), *cb = codes(i);
        uint4 w[NB][2];
        float sc[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int row = (wn * NB + n) * 32 + li;
            const int4v_t c = *reinterpret_cast<const int4v_t *>(cb + row * 64 + (((2 * (decltype(i)::value & 1) + h) ^ ((row >> 2) & 3)) << 4));
            w[n][0] = weights_of((uint32_t)c[0], (uint32_t)c[1]);
            w[n][1] = weights_of((uint32_t)c[2], (uint32_t)c[3]);
            sc[n] = *reinterpret_cast<const float *>(b + T::S_AT + row * 4);
        }
        float16v_t d[2];
        float16v_t xs[GX ? MB : 1];
        auto scale = [&](int t) TERN_INLINE {   // tile t = m NB + n
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                // the weights' scale first: the other may be anything
                const float e = GX ? d[t & 1][v] * sc[t % NB] : d[t & 1][v];
                acc[t / NB][t % NB][v] = fmaf(e, GX ? xs[GX ? t / NB : 0][v] : sc[t % NB], acc[t / NB][t % NB][v]);
            }
        };
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const uint8_t *xb = b + (wm * MB + m) * T_BLOCK;
            int4v_t x[4];
            int2v_t y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[c] = *reinterpret_cast<const int4v_t *>(xb + c * 1024 + lane * 16);
                // volatile: two of them read at once would have to be moved behind their x
                y[c] = *(const volatile __attribute__((address_space(3))) int2v_t *)(xb + 4096 + c * 512 + lane * 8);
            }
            if constexpr (GX) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float4v_t f = *reinterpret_cast<const float4v_t *>(b + T::X_AT + ((wm * MB + m) * 32 + 8 * v + 4 * h) * 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) xs[m][4 * v + k] = f[k];
                }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int t = m * NB + n;
                float16v_t z = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                load(t);
                z = mfma(x[0], y[0], w[n][0], z, E3M2());
                z = mfma(x[2], y[2], w[n][1], z, E3M2());
                z = mfma(x[1], y[1], w[n][0], z, E2M3());
                d[t & 1] = mfma(x[3], y[3], w[n][1], z, E2M3());
                if (t > 0) scale(t - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        scale(MB * NB - 1);
    };

    // Step s, in buffer I = s mod ST, asks for terms and scales of step s + 3, and if it is even for the
    // codes of steps s + 2 and s + 3 before them.  At its end, terms and codes of step s + 1 are there: no more are
    // on their way than what was asked for after them.
    auto step = [&](auto i, int s) TERN_INLINE {
        constexpr int I = decltype(i)::value, W = I % 2 == 0 ? T::WI : 0;
        constexpr auto fill = std::integral_constant<int, (I + 3) % ST>();
        constexpr auto next = std::integral_constant<int, (I + 2) % ST>();
        products(i, [&](int t) TERN_INLINE {   // at most two a tile
            constexpr int EACH = (T::LOADS + T::WI + MB * NB - 1) / (MB * NB);
#pragma unroll
            for (int j = t * EACH; j < (t + 1) * EACH; ++j) {
                if (j < W) fetch_codes(lds_of(codes(next)), s + 2, j);
                else if (j < W + T::LOADS) fetch_terms(lds_of(buf(fill)), s + 3, j - W);
            }
        });
        __builtin_amdgcn_sched_barrier(0);   // the wait last
        wait_and_meet<2 * T::LOADS + W>();
    };
    auto each = [&](auto f) TERN_INLINE {   // f(0), ..., f(ST - 1) until one returns true
        return f(std::integral_constant<int, 0>()) || f(std::integral_constant<int, 1>()) ||
               f(std::integral_constant<int, 2>()) || f(std::integral_constant<int, 3>());
    };
#pragma unroll
    for (int j = 0; j < T::WI; ++j) fetch_codes(lds_of(codes0), 0, j);
    each([&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value;
        if constexpr (I < ST - 1) {
#pragma unroll
            for (int j = 0; j < T::LOADS; ++j) fetch_terms(lds_of(buf(i)), I, j);
        }
        return false;
    });
    wait_and_meet<0>();
    int s = 0;
    while (!each([&](auto i) TERN_INLINE {
        step(i, s);
        return ++s >= groups;
    })) {
    }

    // Lane (h, li) holds rows 8 v + 4 h + k of column li of each 32 x 32 tile.  32 rows of the wave at a
    // time go through LDS, so that a lane stores 8 consecutive outputs (2 bytes a lane took 20 us a tile).
    wait_and_meet<0>();   // the last loads are past the end, but still write zeros
    float *out = reinterpret_cast<float *>((wave < T::PER ? buf0 : wave < 2 * T::PER ? buf1 : wave < 3 * T::PER ? buf2 : buf3) + wave % T::PER * T::OUT);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        wave_order();
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int v = 0; v < 16; ++v) out[(8 * (v >> 2) + 4 * h + (v & 3)) * T::ROW + 32 * n + li] = acc[m][n][v];
        wave_order();
        const int row0 = m0 + (wm * MB + m) * 32, col0 = n0 + wn * NB * 32;
#pragma unroll 2
        for (int o = lane; o < 32 * NB * 4; o += 64) {
            const int r = o / (NB * 4), c = o % (NB * 4) * 8, row = row0 + r, left = min(8, N - col0 - c);
            if (row >= M || left <= 0) continue;
            const float xs = GX ? 1.f : a.XS[row];
            const float4v_t y0 = *reinterpret_cast<const float4v_t *>(out + r * T::ROW + c) * xs;
            const float4v_t y1 = *reinterpret_cast<const float4v_t *>(out + r * T::ROW + c + 4) * xs;
            const int64_t at = (int64_t)row * N + col0 + c;
            store4(a.Y, a.y_dtype, at, y0, min(4, left), vec);
            if (left > 4) store4(a.Y, a.y_dtype, at + 4, y1, left - 4, vec);
        }
    }
}

template <int WM, int WN, int MB, int NB, int ST, bool GX>
hipError_t launch_t(const Q8Args &a) {
    typedef Shape<WM, WN, MB, NB, ST, GX> T;
    const int tm = (int)((a.M + T::BM - 1) / T::BM), tn = (int)((a.N + T::BN - 1) / T::BN);
    const size_t unit = a.y_dtype == 2 ? 16 : 8;
    const int vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.Y) % unit == 0;
    hipLaunchKernelGGL((q8_gemm_kernel<WM, WN, MB, NB, ST, GX>), dim3((unsigned)(tm * tn)), dim3(T::NT), 0, a.stream, a, tm, tn,
                       vec);
    return hipGetLastError();
}

constexpr int64_t T_PAD = 128;   // rows of the largest tile

template <bool GX>
hipError_t launch_x(const Q8Args &a) { return launch_t<2, 4, 2, 3, 4, GX>(a); }

// Bytes of the workspace's parts: terms, scales of the weights and of X.
size_t terms_bytes(int64_t M, int64_t K) { return (size_t)((M + T_PAD - 1) / T_PAD * (T_PAD / T_ROWS)) * (size_t)(K / 128) * T_BLOCK; }
size_t scales_bytes(int64_t rows, int64_t K) { return (size_t)((rows + S_ROWS - 1) / S_ROWS) * (size_t)(K / 128) * S_ROWS * 4; }

}  // namespace

size_t q8_gemm_workspace(int64_t M, int64_t N, int64_t K) { return terms_bytes(M, K) + scales_bytes(N, K) + scales_bytes(M, K); }

double q8_gemm_time(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = ((M + 127) / 128) * ((N + 383) / 384);
    return 18 + (double)(K / 128) * (1.75 * (double)((tiles + 255) / 256) - 0.5);
}

hipError_t launch_q8_gemm(const Q8Args &a0) {
    Q8Args a = a0;
    char *ws = static_cast<char *>(a.terms);
    float *w_scales = reinterpret_cast<float *>(ws + terms_bytes(a.M, a.K));
    float *x_scales = reinterpret_cast<float *>(ws + terms_bytes(a.M, a.K) + scales_bytes(a.N, a.K));
    a.w_scales = w_scales;
    a.x_scales = x_scales;
    const int groups = (int)(a.K / 128);
    const int64_t tu = (a.M + T_PAD - 1) / T_PAD * (T_PAD / T_ROWS) * groups, pieces = (groups + 7) / 8;
    const int64_t wu = (a.N + S_ROWS - 1) / S_ROWS * pieces;
    const int64_t units = tu + wu + (a.grouped ? (a.M + S_ROWS - 1) / S_ROWS * pieces : 0);
    hipLaunchKernelGGL(q8_layout_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, a.stream, a.Q, a.S, a.XS, ws, w_scales,
                       x_scales, (int)a.M, (int)a.N, groups, tu, wu, units);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return a.grouped ? launch_x<true>(a) : launch_x<false>(a);
}

}  // namespace tern
