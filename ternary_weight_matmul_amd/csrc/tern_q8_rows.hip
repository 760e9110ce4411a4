// tern_q8_rows.hip -- Y[M,N] = X . (T*S)^T for few rows, with X in 8 bits with scales
// and ternary weights.
//
// Mathematics as in tern_q8_blocks.hip: a block of 128's sum is an exact integer from
// v_mfma_i32_16x16x64_i8, its scales are applied in fp32.
//
// Work layout.  A workgroup owns 16 RW weight rows over all of K, for 32 rows of X.  Its waves are KW
// groups of RW: a group takes every KW-th step of 512 weights, and a wave of it 16
// weight rows.  A wave's codes, 128 bytes a row, go to registers as whole lines, 8
// rows an instruction, the first TT turns' at the start: a line that comes from HBM
// for the first time takes 2 us, so that few turns may wait for one (with codes
// loaded a turn ahead 17408 x 5120 took 14.0 us at 16 rows).  Their turn come, they
// are turned round in the wave's own piece of LDS.  The group's activations of a
// step, 512 bytes a row, go from memory straight to LDS, whole lines again, into one
// of two buffers.  (Loaded by each lane where it needs them, 32 bytes of 16 rows at a
// time, they took as long as the whole kernel: 16.8 us.)  Activations are the rows
// of the matrix tile: lane (p, i) takes 32 bytes of row i, the codes of the same 32
// weights of weight row i, and then holds rows 4 p .. 4 p + 3 of Y for that weight
// row, so that it reads one weight scale a block.
// Loads with nothing to fetch have offsets out of range and return zeros.
// Finally the groups' partial tiles meet in LDS and are summed in a fixed order.
//
// Bound: the lines' way from HBM and the decoding of the codes, some 200 vector
// instructions a wave and step, which overlap only in part.  16 rows, 5120 -> 5120,
// 5120 -> 17408 and 17408 -> 5120: 8.1, 13.2 and 17.0 us; the loads alone 6.5, 9.9 and
// 12.9, the codes' alone 5.4, 8.8 and 9.7, of which 2 are the launch.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "tern_q8.h"
#include "tern_q8_device.h"
#include "tern_tile.h"

namespace tern {

namespace {

constexpr int min(int a, int b) { return a < b ? a : b; }
constexpr int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }

// What every lane holds, in a scalar register: a buffer descriptor made from anything else is
// gathered lane by lane in a loop around each load.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int RW, int KW, int MT, int TT, bool GX>
struct Shape {
    static constexpr int NT = 64 * RW * KW;
    static constexpr int XI = (8 * MT + RW - 1) / RW;         // load instructions of a wave: activations, 2 rows each
    static constexpr int SI = GX ? (MT + RW - 1) / RW : 0;    // their scales, 16 rows each
    static constexpr int C_AT = XI * RW * 1024;               // the waves' codes of a turn
    static constexpr int S_AT = C_AT;
    static constexpr int GROUP = S_AT + SI * RW * 256;        // bytes of a group
    static constexpr int BUF = GROUP * KW;
    static constexpr int RED = KW * RW * MT * 1024;           // the partial tiles
    static_assert(2 * BUF + RW * KW * 2048 <= 160 * 1024 && RED <= BUF, "buffers");
    static_assert(TT % 2 == 0, "turns alternate between two buffers");
};

template <int RW, int KW, int MT, int TT, bool GX>
__global__ __launch_bounds__(64 * RW * KW) void q8_rows_kernel(Q8Args a) {
    typedef Shape<RW, KW, MT, TT, GX> T;
    // One variable each, so that the compiler sees that an access to one need not wait for the loads
    // into another.
    __shared__ __attribute__((aligned(16))) uint8_t buf0[T::BUF], buf1[T::BUF], images[RW * KW * 2048];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kw = wave / RW, rw = wave % RW;
    const int p = lane >> 4, li = lane & 15;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int M = uniform((int)min64(a.M - m0, 16 * MT)), N = (int)a.N, K = (int)a.K;   // M: of this workgroup
    const int groups = K >> 7, steps = (K + 511) >> 9, wrow = K >> 2;
    const int n0 = (blockIdx.x * RW + rw) * 16;
    const int first = uniform(min(n0, N)), rows = uniform(min(N - min(n0, N), 16));   // a minimum is a vector instruction
    const __amdgpu_buffer_rsrc_t rx = buffer_of(a.Q + m0 * K, M * K);
    const __amdgpu_buffer_rsrc_t rxs = buffer_of(a.XS + (GX ? m0 * groups : 0), GX ? M * groups * 4 : 0);
    const __amdgpu_buffer_rsrc_t rc = buffer_of(a.W + (int64_t)first * wrow, rows * wrow);
    const uint16_t *srow = a.S + (int64_t)min(n0 + li, N - 1) * groups;

    // A turn: step turn * KW + kw of the group.  16-byte chunks of a row of activations are XOR-swizzled
    // by the row, those of a row of codes by half of it: the rows that a read touches lie on distinct
    // banks.
    const int xrow = lane >> 5, xchunk = lane & 31, crow = lane >> 3, cpiece = lane & 7;
    auto fetch = [&](uint8_t *to, int turn) TERN_INLINE {
        const int s = turn * KW + kw, left = groups - 4 * s;   // blocks of this step
#pragma unroll
        for (int i = 0; i < T::XI; ++i) {
            const int at = rw * T::XI + i, row = 2 * at + xrow, c = xchunk ^ (row & 15);
            load16_to_lds(rx, to + kw * T::GROUP + at * 1024,
                          (c >> 3) < left && row < 16 * MT ? row * K + s * 512 + c * 16 : OUT_OF_RANGE);
        }
#pragma unroll
        for (int i = 0; i < T::SI; ++i) {
            const int at = rw * T::SI + i, row = 16 * at + (lane >> 2);
            load4_to_lds(rxs, to + kw * T::GROUP + T::S_AT + at * 256,
                         (lane & 3) < left && row < M ? (row * groups + 4 * s + (lane & 3)) * 4 : OUT_OF_RANGE);
        }
    };
    uint4 code[TT][2];
    uint64_t sc[TT];   // 4 fp16
    auto load_codes = [&](int j, int turn) TERN_INLINE {
        const int s = turn * KW + kw, left = groups - 4 * s;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code[j][i] = load16<2>(rc, (cpiece >> 1) < left ? (8 * i + crow) * wrow + s * 128 + cpiece * 16 : OUT_OF_RANGE);
        // the last 4 of the row at most, and shifted: zeros past the end
        __builtin_memcpy(&sc[j], srow + min(4 * s, groups - 4), 8);
    };
    auto scales_of = [&](int j, int turn, float (&f)[4]) TERN_INLINE {
        const int s = turn * KW + kw, past = 4 * s - min(4 * s, groups - 4);
        const uint64_t v = past < 4 ? sc[j] >> (16 * past) : 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = f16_bits_to_float((uint16_t)(v >> (16 * b)));
    };

    float4v_t acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = (float4v_t){0.f, 0.f, 0.f, 0.f};
    uint8_t *image = images + wave * 2048;
    auto products = [&](const uint8_t *b, const float (&scale)[4]) TERN_INLINE {
        const uint8_t *x = b + kw * T::GROUP;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            int4v_t w0, w1;
            decode32(*reinterpret_cast<const uint64_t *>(image + li * 128 + (((2 * g + (p >> 1)) ^ ((li >> 1) & 7)) << 4) + 8 * (p & 1)),
                     w0, w1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint8_t *at = x + (16 * m + li) * 512;
                const int4v_t x0 = *reinterpret_cast<const int4v_t *>(at + (((8 * g + 2 * p) ^ li) << 4));
                const int4v_t x1 = *reinterpret_cast<const int4v_t *>(at + (((8 * g + 2 * p + 1) ^ li) << 4));
                const int4v_t d = mfma_i8(x1, w1, mfma_i8(x0, w0, (int4v_t){0, 0, 0, 0}));
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float e = (float)d[v], s = scale[g];   // 0 past the end
                    // the weights' scale first: the other may be anything
                    if constexpr (GX)
                        e *= s, s = *reinterpret_cast<const float *>(x + T::S_AT + ((16 * m + 4 * p + v) * 4 + g) * 4);
                    acc[m][v] = fmaf(e, s, acc[m][v]);
                }
            }
        }
    };

    const int turns = (steps + KW - 1) / KW;
    // What a wave issues in a turn's end: TURN loads to LDS, then 3 to registers.  They are counted in
    // order, so that a turn's activations are there once all but the newest few have arrived.
    constexpr int TURN = T::XI + T::SI;
    fetch(buf0, 0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(buf1, 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < TT; ++j) load_codes(j, j);
    __builtin_amdgcn_sched_barrier(0);
    wait_and_meet<min(TURN + 3 * TT, 63)>();
    for (int t0 = 0; t0 < turns; t0 += TT) {
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int t = t0 + j;
            if (t >= turns) break;
            float now[4];
            scales_of(j, t, now);
            wave_order();   // the image before is read
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint4 *>(image + (8 * i + crow) * 128 + ((cpiece ^ (((8 * i + crow) >> 1) & 7)) << 4)) = code[j][i];
            wave_order();
            products(j & 1 ? buf1 : buf0, now);
            __builtin_amdgcn_sched_barrier(0);
            // turn t + 1 is there, and turn t's buffer is free: past turn 0 all but this wave's newest
            // loads to registers
            if (t == 0) wait_and_meet<min(3 * TT, 63)>();
            else wait_and_meet<3>();
            fetch(j & 1 ? buf1 : buf0, t + 2);
            __builtin_amdgcn_sched_barrier(0);   // in this order, which the counts rely on
            load_codes(j, t + TT);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The last turns' loads are past the end, but still write zeros: all of them before the buffer is
    // used anew.
    wait_and_meet<0>();
    float4v_t *red = reinterpret_cast<float4v_t *>(buf0);
#pragma unroll
    for (int m = 0; m < MT; ++m) red[(wave * MT + m) * 64 + lane] = acc[m];
    __syncthreads();
    for (int o = tid; o < RW * MT * 64; o += T::NT) {
        float4v_t y = red[o];
#pragma unroll
        for (int w = 1; w < KW; ++w) y += red[w * (RW * MT * 64) + o];
        const int l = o & 63, t = o >> 6, n = (blockIdx.x * RW + t / MT) * 16 + (l & 15);
        if (n >= N) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int m = 16 * (t % MT) + 4 * (l >> 4) + v;
            if (m >= M) continue;
            const float r = GX ? y[v] : y[v] * a.XS[m0 + m];
            const int64_t at = (m0 + m) * N + n;
            if (a.y_dtype == 2) store_out<2>(a.Y, at, r);
            else if (a.y_dtype == 1) store_out<1>(a.Y, at, r);
            else store_out<0>(a.Y, at, r);
        }
    }
}

int64_t chunks(int64_t M) { return M <= 16 ? 1 : (M + 31) / 32; }   // of the rows of X

template <int RW, int KW, int MT, int TT, bool GX>
hipError_t launch_t(const Q8Args &a) {
    const unsigned grid = (unsigned)((a.N + 16 * RW - 1) / (16 * RW));
    hipLaunchKernelGGL((q8_rows_kernel<RW, KW, MT, TT, GX>), dim3(grid, (unsigned)chunks(a.M)), dim3(64 * RW * KW), 0,
                       a.stream, a);
    return hipGetLastError();
}

// Weight rows of a workgroup, in sixteens: the busiest CU takes ceil(workgroups / CUs) of them, plus
// about one sixteen's worth of work that every workgroup has.  Measured at M = 16, K = 5120, in us, for
// 1, 2, 3, 4, 5 sixteens: 5120 rows 11.4, 7.8, 9.2, 9.7, 11.6; 17408 rows 27.2, 16.9, 18.0, 16.0, 12.8.
struct Split {
    int sixteens;
    int64_t cost;
};
Split split(int64_t M, int64_t N) {
    const int64_t blocks = (N + 15) / 16, times = chunks(M);
    Split best = {1, 0};
    for (int i = 1; i <= 5; ++i) {
        const int64_t cost = ((blocks + i - 1) / i * times + 255) / 256 * (i + 1);
        if (i == 1 || cost < best.cost) best = {i, cost};
    }
    return best;
}

// Groups that split K: 8 to 10 waves a workgroup (more of them take longer to start than they save:
// two sixteens of 5120 x 5120 with 4, 5, 6, 8 groups 7.8, 8.0, 9.2, 11.9 us).  Codes in registers for 4
// turns ahead pay with long K (17408: 16.4 us against 16.9 with 2), not with 3 turns (8.0 against 7.8).
template <int MT, bool GX>
hipError_t launch_m(const Q8Args &a) {
    switch (split(a.M, a.N).sixteens) {
    case 1: return launch_t<1, MT == 1 ? 5 : 4, MT, 2, GX>(a);
    case 2: return a.K > 12288 ? launch_t<2, 4, MT, 4, GX>(a) : launch_t<2, 4, MT, 2, GX>(a);
    case 3: return launch_t<3, 3, MT, 2, GX>(a);
    case 4: return launch_t<4, 2, MT, 2, GX>(a);
    default: return launch_t<5, 2, MT, 2, GX>(a);
    }
}

template <bool GX>
hipError_t launch_x(const Q8Args &a) { return a.M > 16 ? launch_m<2, GX>(a) : launch_m<1, GX>(a); }

}  // namespace

// 4 scales are loaded at a time, and a grid has 65535 chunks.  Offsets: 32 rows of up to 2^23 bytes.
bool q8_rows_fits(int64_t M, int64_t, int64_t K) { return K >= 512 && chunks(M) <= 65535; }

double q8_rows_time(int64_t M, int64_t N, int64_t K) { return 2 + 0.23 * (double)split(M, N).cost * (double)((K + 511) / 512); }

hipError_t launch_q8_rows(const Q8Args &a) { return a.grouped ? launch_x<true>(a) : launch_x<false>(a); }

}  // namespace tern
