// tern_mx_gemv.hip -- Y[M,N] = X[M,K] . W^T for few rows M, with W in
// microscaled 4-bit floats and X in fp16, bf16 or the same 4-bit form.
//
// Mathematics.  Y[m,n] = sum_b 2^(e[n,b] - 127) sum_{k in b} q[n,k] X[m,k].
// A weight q 2^(e - 127) has two significant bits and is exact in bf16, so
// with 16-bit X the block scale is folded into the bf16 weight as it is
// decoded, the products are exact and the matrix cores sum them in fp32
// (v_mfma_f32_16x16x32_bf16).  An fp16 activation (11 significant bits) is
// written exactly as two bf16 terms, its first 8 bits and the rest, each
// multiplied by the weights.  (fp16 weights would do with one product, but a
// scale outside [2^-23, 2^13] does not fit them, and a choice by the scales at
// hand would let a row's last bit depend on its neighbours.)  With 4-bit X both
// operands go into v_mfma_scale_f32_16x16x128_f8f6f4 as they are stored.
//
// Work layout.  Waves of a workgroup split K into 256-weight steps, a run of
// them each; a workgroup owns 8 NB weight rows.  Lane (p = lane / 16, col =
// 2 r + c) loads the 16 code bytes of block 4 c + p of the step in row r: one
// instruction reads 8 rows x 128 contiguous bytes (whole lines).  The two
// halves c of a row are separate columns of the matrix tile, so tile row i =
// 8 c' + s holds activation row s in half c' and only the results with c' = c
// are used.  Partial sums of the waves meet in LDS and are added in a fixed
// order.
//
// A lane's activation operand is 64 bytes of one row of X.  A wave loads its
// step's activations 16 bytes a lane in order and passes them through its own
// corner of LDS: loaded straight to where they are used, 16 bytes out of every
// 64, they cost 4 to 6 us of 16 to 18 at 5120 -> 17408.  Scale bytes are loaded
// 4 a lane for four steps at once and handed to the lanes that need them.
//
// A wave holds the loads of one step (NB code loads) and refills each as soon as
// it has used it.  8 waves and up to 9 row groups a workgroup, one workgroup a
// CU where the rows allow it: fewer rows (3 groups, more workgroups than CUs)
// took 12.7 to 16.9 us at M = 1 / 4, 5120 -> 17408 where this takes 12.9 /
// 13.6, two steps of loads in flight or 12 waves 0.5 to 1 us more.
//
// Bound: HBM (the code bytes) and, from 16 rows, vector work.  Weights rotated
// over 2 GB: M = 1, 5120 -> 5120 5.8 us (a plain read of the bytes 3.7); 5120 ->
// 17408 (8.6) M = 4 13.6, M = 16 17.4, with fp16 X 15.0 and 21.5, 4-bit X 12.6
// and 14.0.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "tern_device.h"
#include "tern_mx.h"
#include "tern_mx_device.h"

namespace tern {

namespace {

typedef float float4v_t __attribute__((ext_vector_type(4)));
typedef int int8v_t __attribute__((ext_vector_type(8)));

// The place of 16-byte chunk c (0..31) of activation row t in a wave's corner.  Lanes that are
// served together read two chunks 4 apart of each of 8 rows: XORed with these they fall on 16
// distinct places of 256 bytes.
__device__ __forceinline__ int chunk_at(int t, int c) { return t * 512 + ((c ^ ((t & 3) | ((t & 4) << 1))) << 4); }

// XT: X is fp16 (0), bf16 (1) or 4-bit (2).  TC: activation rows it has room for.  SC4: rows of
// scale bytes can be loaded 4 at a time.  NT: cache policy of the code loads.
constexpr int kMaxWaves = 8;

template <int XT, int TC, int NB>
struct Shape {
    static constexpr int SETS = (TC + 7) / 8;              // matrix tiles of 8 activation rows
    static constexpr int XL = XT == 2 ? 0 : (TC + 1) / 2;  // activation loads of a step
    static constexpr int CORNER = XL * 1024;               // bytes of a wave's corner
};

// What a wave holds of one step: code and scale bytes of NB row groups, activations.
template <int XT, int TC, int NB>
struct Stage {
    typedef Shape<XT, TC, NB> T;
    uint4 code[NB];
    uint32_t scale[NB];                // without SC4
    uint4 x[XT == 2 ? T::SETS : T::XL];
    uint32_t xscale[T::SETS];          // XT == 2
};

template <int XT, int TC, int NB, bool SC4, int NT>
__global__ __launch_bounds__(64 * kMaxWaves) void mx_gemv_kernel(
    const uint8_t *__restrict__ X, const uint8_t *__restrict__ XE, const uint8_t *__restrict__ W,
    const uint8_t *__restrict__ WE, void *__restrict__ Y, int y_dtype, int64_t M, int64_t N, int blocks, int nw,
    int per_wave) {
    typedef Shape<XT, TC, NB> T;
    typedef Stage<XT, TC, NB> S;
    constexpr int SETS = T::SETS;
    extern __shared__ uint4 lds4[];
    char *corners = reinterpret_cast<char *>(lds4);
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    float *red = reinterpret_cast<float *>(corners + nw * T::CORNER);   // [nw][SETS][NB][2 halves][8 slots][8 rows]
    char *corner = corners + wave * T::CORNER;
    const int p = lane >> 4, col = lane & 15;
    const int r = col >> 1, c = col & 1;      // as a weight column
    const int ah = col >> 3, as = col & 7;    // as an activation row: half, slot
    const int64_t n0 = (int64_t)blockIdx.x * 8 * NB;
    const int64_t m0 = (int64_t)blockIdx.y * TC;

    // Loads past the end of a row (the last step), of rows past N and of activation rows past M
    // have offsets out of range: they read no memory and return zeros (a zero scale byte is a
    // finite scale).
    const int steps = (blocks + 7) / 8;
    const int wrows = (int)min((int64_t)8 * NB, N - n0), xrows = (int)min((int64_t)TC, M - m0);
    const int xrow = blocks * (XT == 2 ? 16 : 64);
    const __amdgpu_buffer_rsrc_t rw = buffer_of(W + n0 * blocks * 16, wrows * blocks * 16);
    const __amdgpu_buffer_rsrc_t re = buffer_of(WE + n0 * blocks, wrows * blocks);
    const __amdgpu_buffer_rsrc_t rx = buffer_of(X + m0 * xrow, xrows * xrow);
    const __amdgpu_buffer_rsrc_t rxe = buffer_of(XT == 2 ? XE + m0 * blocks : nullptr, XT == 2 ? xrows * blocks : 0);

    float4v_t acc[SETS][NB];
#pragma unroll
    for (int t = 0; t < SETS; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] = (float4v_t){0.f, 0.f, 0.f, 0.f};

    const int first = wave * per_wave, last = min(first + per_wave, steps);
    // Loads of step s; one that is not this wave's costs nothing.
    auto load_x = [&](S &st, int s) __attribute__((always_inline)) {
        const bool mine = s < last;
        if constexpr (XT == 2) {
            const int ab = 8 * s + 4 * ah + p;
#pragma unroll
            for (int t = 0; t < SETS; ++t) {
                const int at = (8 * t + as) * blocks + ab;
                const bool ok = mine && ab < blocks && 8 * t + as < xrows;
                st.x[t] = load16(rx, ok ? at * 16 : OUT_OF_RANGE);
                st.xscale[t] = __builtin_amdgcn_raw_buffer_load_b8(rxe, ok ? at : OUT_OF_RANGE, 0, 0);
            }
        } else {
            const int chunk = 32 * s + (lane & 31);   // 8 activations
            const int off = mine && chunk < 4 * blocks ? (lane >> 5) * xrow + chunk * 16 : OUT_OF_RANGE;
#pragma unroll
            for (int i = 0; i < T::XL; ++i) st.x[i] = load16(rx, off + 2 * i * xrow);
        }
    };
    auto load_group = [&](S &st, int s, int b) __attribute__((always_inline)) {
        const int wb = 8 * s + 4 * c + p;   // this lane's block
        const int at = s < last && wb < blocks ? r * blocks + wb : OUT_OF_RANGE;
        if constexpr (!SC4) st.scale[b] = __builtin_amdgcn_raw_buffer_load_b8(re, at + 8 * b * blocks, 0, 0);
        st.code[b] = load16<NT>(rw, (at < 0 ? OUT_OF_RANGE : at * 16) + 8 * b * blocks * 16);
    };
    // Scale bytes of steps s .. s + 3: lane (u, 2 r + c) holds the 4 of half c of step s + u, row r.
    auto load_scales = [&](uint32_t (&sc)[NB], int s) __attribute__((always_inline)) {
        const int at = 8 * (s + p) + 4 * c;
        const int off = at < blocks ? r * blocks + at : OUT_OF_RANGE;
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[b] = __builtin_amdgcn_raw_buffer_load_b32(re, off + 8 * b * blocks, 0, 0);
    };
    // Computes step s (the u-th of its four) and refills what it has used with step s + 1.
    auto step = [&](S &st, const uint32_t (&sc)[NB], int s, int u) __attribute__((always_inline)) {
        uint32_t e[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if constexpr (SC4) e[b] = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * u + col) * 4, (int)sc[b]);
        uint4 a[SETS][4], lo[XT == 0 ? SETS : 1][4];
        uint32_t as4[SETS];
        if constexpr (XT == 2) {
#pragma unroll
            for (int t = 0; t < SETS; ++t) a[t][0] = st.x[t], as4[t] = st.xscale[t];
        } else {
            // the wave's LDS accesses are served in order: only the compiler has to keep it
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < T::XL; ++i)
                *reinterpret_cast<uint4 *>(corner + chunk_at(2 * i + (lane >> 5), lane & 31)) = st.x[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int t = 0; t < SETS; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[t][i] = *reinterpret_cast<const uint4 *>(
                        corner + chunk_at((8 * t + as) % (2 * T::XL), 4 * (4 * ah + p) + i));
                    if constexpr (XT == 0) a[t][i] = fp16_terms(a[t][i], lo[t][i]);
                }
        }
        load_x(st, s + 1);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t scale = SC4 ? (e[b] >> (8 * p)) & 255u : st.scale[b];
            const uint4 q = st.code[b];
            if constexpr (XT == 2) {
                const int8v_t bv = {(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < SETS; ++t) {
                    const int8v_t av = {(int)a[t][0].x, (int)a[t][0].y, (int)a[t][0].z, (int)a[t][0].w, 0, 0, 0, 0};
                    acc[t][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[t][b], 4, 4, 0, (int)as4[t],
                                                                                 0, (int)scale);
                }
            } else {
                const uint32_t cw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf168_t bv = decode8(cw[i], __builtin_bit_cast(float, scale << 23));
#pragma unroll
                    for (int t = 0; t < SETS; ++t) {
                        acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168_t, a[t][i]), bv,
                                                                           acc[t][b], 0, 0, 0);
                        if constexpr (XT == 0)
                            acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168_t, lo[t][i]), bv,
                                                                               acc[t][b], 0, 0, 0);
                    }
                }
            }
            load_group(st, s + 1, b);
            // the refill stays here: moved up it would need more registers, moved down it would come late
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    S st;
    uint32_t sc[NB], next[NB];
    if constexpr (SC4) load_scales(next, first);
    load_x(st, first);
#pragma unroll
    for (int b = 0; b < NB; ++b) load_group(st, first, b);
    auto take_scales = [&](int s) __attribute__((always_inline)) {
        if (!SC4 || (s - first) % 4 != 0) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[b] = next[b];
        load_scales(next, s + 4);
    };
    for (int s = first;;) {   // (with the test at the top the compiler's order of the loads cost 5 to 10%)
        take_scales(s);
        step(st, sc, s, (s - first) % 4);
        if (++s >= last) break;
    }

    // Lane (p, col) holds tile rows 4 p + v, i.e. half p / 2, slots 4 (p % 2)
    // + v, of column (r, c): it is used where p / 2 = c.  Every lane stores
    // (an unused one into its own spare word), so that no matrix instruction
    // is moved under a partial EXEC mask.
    const bool used = (p >> 1) == c;
    const int spare = nw * SETS * NB * 128 + lane;
#pragma unroll
    for (int t = 0; t < SETS; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int at = (((wave * SETS + t) * NB + b) * 2 + c) * 64 + (4 * (p & 1) + v) * 8 + r;
                red[used ? at : spare] = acc[t][b][v];
            }
    __syncthreads();
    for (int o = tid; o < TC * NB * 8; o += 64 * nw) {
        const int rr = o & 7, b = (o >> 3) % NB, mm = (o >> 3) / NB;
        const int64_t m = m0 + mm, n = n0 + 8 * b + rr;
        if (m >= M || n >= N) continue;
        const float *q = red + ((mm / 8) * NB + b) * 128 + (mm % 8) * 8 + rr;
        float y = 0.f;
        for (int w = 0; w < nw; ++w) y += q[w * SETS * NB * 128] + q[w * SETS * NB * 128 + 64];
        if (y_dtype == 2) store_out<2>(Y, m * N + n, y);
        else if (y_dtype == 1) store_out<1>(Y, m * N + n, y);
        else store_out<0>(Y, m * N + n, y);
    }
}

template <int XT, int TC, int NB>
hipError_t launch_t(const MxArgs &a) {
    typedef Shape<XT, TC, NB> T;
    const int blocks = (int)(a.K / 32), steps = (blocks + 7) / 8;
    const int per_wave = (steps + kMaxWaves - 1) / kMaxWaves;
    const int nw = (steps + per_wave - 1) / per_wave;
    const size_t lds = (size_t)nw * T::CORNER + ((size_t)nw * T::SETS * NB * 128 + 64) * 4;
    const dim3 grid((unsigned)((a.N + 8 * NB - 1) / (8 * NB)), (unsigned)((a.M + TC - 1) / TC));
    auto go = [&](auto sc4, auto nt) {
        constexpr auto kern = &mx_gemv_kernel<XT, TC, NB, decltype(sc4)::value, decltype(nt)::value>;
        const hipError_t e = raise_lds_limit<kern>(lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, grid, dim3(64 * nw), lds, a.stream, static_cast<const uint8_t *>(a.X), a.XE, a.W, a.WE,
                           a.Y, a.y_dtype, a.M, a.N, blocks, nw, per_wave);
        return hipGetLastError();
    };
    const std::integral_constant<int, 2> once;
    const std::integral_constant<int, 0> cached;
    if (blocks % 4 == 0 && reinterpret_cast<uintptr_t>(a.WE) % 4 == 0)
        return grid.y == 1 ? go(std::true_type(), once) : go(std::true_type(), cached);
    return grid.y == 1 ? go(std::false_type(), once) : go(std::false_type(), cached);
}

// Row groups per workgroup.  The busiest CU runs ceil(grid / 256) workgroups of NB groups each,
// plus about one group's worth of work of its own per workgroup.
int groups_per_workgroup(int64_t N, int most) {
    const int64_t groups = (N + 7) / 8;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int nb = 1; nb <= most; ++nb) {
        const int64_t grid = (groups + nb - 1) / nb, cost = (grid + 255) / 256 * (nb + 1);
        if (cost <= least) least = cost, best = nb;
    }
    return best;
}

template <int XT, int TC>
hipError_t launch_tc(const MxArgs &a) {
    switch (groups_per_workgroup(a.N, 9)) {
    case 1: return launch_t<XT, TC, 1>(a);
    case 2: return launch_t<XT, TC, 2>(a);
    case 3: return launch_t<XT, TC, 3>(a);
    case 4: return launch_t<XT, TC, 4>(a);
    case 5: return launch_t<XT, TC, 5>(a);
    case 6: return launch_t<XT, TC, 6>(a);
    case 7: return launch_t<XT, TC, 7>(a);
    case 8: return launch_t<XT, TC, 8>(a);
    default: return launch_t<XT, TC, 9>(a);
    }
}

template <int XT>
hipError_t launch_x(const MxArgs &a) {
    if constexpr (XT == 2) {
        return a.M <= 8 ? launch_tc<XT, 8>(a) : launch_tc<XT, 16>(a);
    } else {
        if (a.M <= 2) return launch_tc<XT, 2>(a);
        if (a.M <= 4) return launch_tc<XT, 4>(a);
        return a.M <= 8 ? launch_tc<XT, 8>(a) : launch_tc<XT, 16>(a);
    }
}

}  // namespace

hipError_t launch_mx_gemv(const MxArgs &a0) {
    MxArgs a = a0;
    const int64_t rows = 65535 * (int64_t)16;   // the grid's second dimension holds 65535 chunks
    const int64_t ysize = a.y_dtype == 2 ? 4 : 2;
    const int64_t xrow = a.x_dtype == 2 ? a.K / 2 : a.K * 2;
    for (int64_t m = 0; m < a0.M; m += rows) {
        a.M = a0.M - m < rows ? a0.M - m : rows;
        a.X = static_cast<const char *>(a0.X) + m * xrow;
        a.XE = a0.XE == nullptr ? nullptr : a0.XE + m * (a.K / 32);
        a.Y = static_cast<char *>(a0.Y) + m * a.N * ysize;
        const hipError_t e = a.x_dtype == 0 ? launch_x<0>(a) : (a.x_dtype == 1 ? launch_x<1>(a) : launch_x<2>(a));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tern
