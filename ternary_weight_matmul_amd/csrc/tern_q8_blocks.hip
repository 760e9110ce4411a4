// tern_q8_blocks.hip -- Y[M,N] = X . (T*S)^T for some hundred rows M, with X in 8 bits
// with scales and ternary weights.
//
// Mathematics.  X[m,k] = q[m,k] s[m] (a scale per row) or q[m,k] s[m,k/128]; the
// weights t are -1, 0 or +1 with a scale S[n,k/128].  So
//   Y[m,n] = sum over blocks g of 128:  s[m,g] S[n,g] * sum over k in g of q t
// whose inner sums are integers below 2^15: v_mfma_i32_16x16x64_i8 forms them
// without error.  They become fp32 and meet their scales there.
//
// Work layout.  A workgroup of 4 waves computes 64 x 128 outputs.  A step is one block
// of 128: the activations of all 64 rows, 128 bytes each, and the codes of all 128
// weight rows, 32 bytes each, go from memory straight to LDS, into one of ST buffers,
// ST - 1 steps before they are needed.  Each wave decodes the codes of its own 32
// weight rows, once, and every wave reads all activations.  The rows of the matrix
// tile are weights and its columns activations: a lane then holds 4 consecutive
// outputs of one row of Y.  Lane group p = lane / 16 takes weights 32 p .. 32 p + 31
// of the block, 8 bytes of codes, and the same 32 bytes of X.
//
// Bound: the way of a step's lines to LDS where a CU has one workgroup (0.61 us a
// step), then the conversion and scaling of the sums, one for every 2 matrix
// instructions of half rate (0.33 us for each workgroup more).  A buffer more, with
// scales asked for two steps ahead, changed nothing (512 x 5120 x 5120 38.8 us against
// 38.1), nor did tiles of 32 x 128 where there are few (256 rows 27.2 against 27.4; 64
// rows 21.9 against 27.7, which the kernel for few rows takes in 13.6).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "tern_q8.h"
#include "tern_q8_device.h"
#include "tern_tile.h"

namespace tern {

namespace {

// MFMAS matrix instructions, each followed by VALUS vector ones.
template <int MFMAS, int VALUS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int g = 0; g < MFMAS; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALUS, 0);
    }
}

constexpr int WV = 4, NB = 2, MB = 4;   // waves; sixteens of weight rows of a wave, and of rows of X
constexpr int ST = 3;                   // buffers

template <bool GX>
struct Shape {
    static constexpr int NT = 64 * WV, BM = 16 * MB, BN = 16 * NB * WV;
    static constexpr int A_LDS = BM * 128, W_LDS = BN * 32;
    static constexpr int AI = A_LDS / 1024 / WV, WI = W_LDS / 1024 / WV;   // load instructions per wave
    static constexpr int S_AT = A_LDS + W_LDS;                             // the weights' scales, fp32
    static constexpr int X_AT = S_AT + BN * 4;                             // GX: those of the activations
    static constexpr int BUF = X_AT + (GX ? BM * 4 : 0);
    static constexpr int LOADS = AI + WI;
    static constexpr int SP = (BN + NT - 1) / NT, XP = GX ? (BM + NT - 1) / NT : 0;
    static_assert(A_LDS % (1024 * WV) == 0 && W_LDS % (1024 * WV) == 0, "whole load instructions");
    static_assert(ST == 3 && ST * BUF <= 160 * 1024, "buffers");
    static_assert((ST - 2) * LOADS < 64, "the wait counter has 6 bits");
};

template <bool GX>
__global__ __launch_bounds__(64 * WV, 2) void q8_blocks_kernel(Q8Args a, int tiles_m, int tiles_n, int vec) {
    typedef Shape<GX> T;
    // One variable each, so that the compiler sees that an access to one need not wait for the loads
    // into another.
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::BUF], buf1[T::BUF], buf2[T::BUF];
    auto buf = [&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value % ST;
        if constexpr (I == 0) return buf0;
        else if constexpr (I == 1) return buf1;
        else return buf2;
    };
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p = lane >> 4, li = lane & 15;
    const int M = (int)a.M, N = (int)a.N, K = (int)a.K, groups = K >> 7;

    // Workgroups go round the 8 XCDs: each XCD gets a contiguous run of tiles, which goes down
    // bands of 8 tile rows, so that its 32 CUs share 8 row tiles and 4 column tiles in its L2.
    const int ntiles = tiles_m * tiles_n;
    int tile = blockIdx.x;
    if (ntiles % 8 == 0) tile = (blockIdx.x % 8) * (ntiles / 8) + blockIdx.x / 8;
    const int band = tile / (8 * tiles_n), in = tile - band * 8 * tiles_n, bandm = min(8, tiles_m - band * 8);
    const int m0 = (band * 8 + in % bandm) * T::BM, n0 = in / bandm * T::BN;

    const int wrow = K >> 2, xrows = min(T::BM, M - m0), wrows = min(T::BN, N - n0);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(a.Q + (int64_t)m0 * K, xrows * K);
    const __amdgpu_buffer_rsrc_t rw = buffer_of(a.W + (int64_t)n0 * wrow, wrows * wrow);

    // Tiles go from memory straight to LDS, 16 bytes a lane, 1 KB an instruction: 8 rows of X or 32 of
    // codes.  Rows past the end, and steps past it, get an offset out of range and arrive as zeros.
    const int ar = lane >> 3, wr = lane >> 1;
    auto fetch = [&](uint8_t *to, int s) TERN_INLINE {
        const int xs = s < groups ? s * 128 : OUT_OF_RANGE, ws = s < groups ? s * 32 : OUT_OF_RANGE;
#pragma unroll
        for (int i = 0; i < T::AI; ++i) {
            const int at = wave * T::AI + i, row = at * 8 + ar, off = row * K + (((lane & 7) ^ xor128(row)) << 4);
            load16_to_lds(rx, to + at * 1024, off + xs);
        }
#pragma unroll
        for (int i = 0; i < T::WI; ++i) {
            const int at = wave * T::WI + i, row = at * 32 + wr, off = row * wrow + (((lane & 1) ^ xor32(row)) << 4);
            load16_to_lds(rw, to + T::A_LDS + at * 1024, off + ws);
        }
    };
    // Scales go through registers, one step ahead of the tiles; past the end they are read again and
    // meet sums of zeros that are not added.
    uint16_t sw[T::SP];
    float sx[T::XP > 0 ? T::XP : 1];
    auto load_scales = [&](int s) TERN_INLINE {
        const int g = min(s, groups - 1);
#pragma unroll
        for (int i = 0; i < T::SP; ++i)
            sw[i] = a.S[(int64_t)(n0 + min(i * T::NT + tid, wrows - 1)) * groups + g];
#pragma unroll
        for (int i = 0; i < T::XP; ++i)
            sx[i] = a.XS[(int64_t)(m0 + min(i * T::NT + tid, xrows - 1)) * groups + g];
    };
    auto store_scales = [&](uint8_t *to) TERN_INLINE {
#pragma unroll
        for (int i = 0; i < T::SP; ++i)
            if (i * T::NT + tid < T::BN)
                reinterpret_cast<float *>(to + T::S_AT)[i * T::NT + tid] = f16_bits_to_float(sw[i]);
#pragma unroll
        for (int i = 0; i < T::XP; ++i)
            if (i * T::NT + tid < T::BM) reinterpret_cast<float *>(to + T::X_AT)[i * T::NT + tid] = sx[i];
    };

    float4v_t acc[NB][MB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[n][m] = (float4v_t){0.f, 0.f, 0.f, 0.f};

    const int wrow0 = wave * 16 * NB;
    auto products = [&](const uint8_t *b) TERN_INLINE {
        int4v_t w0[NB], w1[NB];
        float4v_t sc[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int row = wrow0 + 16 * n + li;
            decode32(*reinterpret_cast<const uint64_t *>(b + T::A_LDS + swz<32>(row, p >> 1) + 8 * (p & 1)), w0[n], w1[n]);
            sc[n] = *reinterpret_cast<const float4v_t *>(b + T::S_AT + (wrow0 + 16 * n + 4 * p) * 4);
        }
        // Activations are read a block of rows ahead, and a block's sums are scaled while the next
        // block's matrix instructions run.  The barriers keep the compiler from fetching everything
        // first, for which there are no registers.
        int4v_t x[2][2], d[2][NB];
        float xs[2] = {1.f, 1.f};
        auto read = [&](int m) TERN_INLINE {
            const int row = 16 * m + li;
            x[m & 1][0] = *reinterpret_cast<const int4v_t *>(b + swz<128>(row, 2 * p));
            x[m & 1][1] = *reinterpret_cast<const int4v_t *>(b + swz<128>(row, 2 * p + 1));
        };
        auto scale = [&](int m) TERN_INLINE {
            if constexpr (GX) xs[m & 1] = reinterpret_cast<const float *>(b + T::X_AT)[16 * m + li];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    // the weights' scale first: the other may be anything
                    const float e = GX ? (float)d[m & 1][n][v] * sc[n][v] : (float)d[m & 1][n][v];
                    acc[n][m][v] = fmaf(e, GX ? xs[m & 1] : sc[n][v], acc[n][m][v]);
                }
        };
        read(0);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (m + 1 < MB) read(m + 1);
#pragma unroll
            for (int n = 0; n < NB; ++n) d[m & 1][n] = mfma_i8(w0[n], x[m & 1][0], (int4v_t){0, 0, 0, 0});
#pragma unroll
            for (int n = 0; n < NB; ++n) d[m & 1][n] = mfma_i8(w1[n], x[m & 1][1], d[m & 1][n]);
            if (m > 0) scale(m - 1);
            interleave<2 * NB, GX ? 6 : 4>();
            __builtin_amdgcn_sched_barrier(0);
        }
        scale(MB - 1);
    };

    // Step s, in buffer I = s mod ST, fetches step s + ST - 1.
    auto step = [&](auto i, int s) TERN_INLINE {
        constexpr int I = decltype(i)::value;
        constexpr auto fill = std::integral_constant<int, (I + ST - 1) % ST>();
        const int f = s + ST - 1;
        store_scales(buf(fill));
        load_scales(f + 1);
        fetch(buf(fill), f);
        __builtin_amdgcn_sched_barrier(0);   // the loads first
        products(buf(i));
        __builtin_amdgcn_sched_barrier(0);   // and the wait last
        wait_and_meet<(ST - 2) * T::LOADS>();   // step s + 1 is there
    };
    auto each = [&](auto f) TERN_INLINE {   // f(0), ..., f(ST - 1) until one returns true
        return f(std::integral_constant<int, 0>()) || f(std::integral_constant<int, 1>()) ||
               f(std::integral_constant<int, 2>());
    };
    load_scales(0);
    each([&](auto i) TERN_INLINE {
        constexpr int I = decltype(i)::value;
        if constexpr (I < ST - 1) {
            store_scales(buf(i));
            load_scales(I + 1);
            fetch(buf(i), I);
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

    // lane (p, li): outputs n = 4 p + v of row li of each 16 x 16 block
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int row = m0 + 16 * m + li;
        if (row >= M) continue;
        const float xs = GX ? 1.f : a.XS[row];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int c0 = n0 + wrow0 + 16 * n + 4 * p;
            store4(a.Y, a.y_dtype, (int64_t)row * N + c0, acc[n][m] * xs, min(4, N - c0), vec);
        }
    }
}

template <bool GX>
hipError_t launch_t(const Q8Args &a) {
    typedef Shape<GX> T;
    const int tm = (int)((a.M + T::BM - 1) / T::BM), tn = (int)((a.N + T::BN - 1) / T::BN);
    const size_t unit = a.y_dtype == 2 ? 16 : 8;
    const int vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.Y) % unit == 0;
    hipLaunchKernelGGL(q8_blocks_kernel<GX>, dim3((unsigned)(tm * tn)), dim3(T::NT), 0, a.stream, a, tm, tn,
                       vec);
    return hipGetLastError();
}

}  // namespace

double q8_blocks_time(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = ((M + 63) / 64) * ((N + 127) / 128);
    return 3.5 + (double)(K / 128) * (0.28 + 0.33 * (double)((tiles + 255) / 256));
}

hipError_t launch_q8_blocks(const Q8Args &a) {
    return a.grouped ? launch_t<true>(a) : launch_t<false>(a);
}

}  // namespace tern
