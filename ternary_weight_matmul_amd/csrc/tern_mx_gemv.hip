// tern_mx_gemv.hip -- Y[M,N] = X[M,K] . W^T for few rows M, with W in
// microscaled 4-bit floats and X in fp16, bf16 or the same 4-bit form.
//
// Mathematics.  Y[m,n] = sum_b 2^(e[n,b] - 127) sum_{k in b} q[n,k] X[m,k].
// A weight q 2^(e - 127) has two significant bits and is exact in bf16, so
// with 16-bit X the block scale is folded into the bf16 weight as it is
// decoded, the products are exact and the matrix cores sum them in fp32
// (v_mfma_f32_16x16x32_bf16).  An fp16 activation (11 significant bits) is
// written exactly as two bf16 terms, hi = bf16(x) and lo = x - hi, which take
// separate rows of the matrix tile.  With 4-bit X both operands go into
// v_mfma_scale_f32_16x16x128_f8f6f4 as they are stored.
//
// Work layout.  Waves of a workgroup split K into 256-weight steps; a
// workgroup owns 8 NB weight rows.  Lane (p = lane / 16, col = 2 r + c) loads
// the 16 code bytes of block 4 c + p of the step in row r: one instruction
// reads 8 rows x 128 contiguous bytes (whole lines).  The two halves c of a
// row are separate columns of the matrix tile, so tile row i = 8 c' + s holds
// activation slot s of half c' and only the results with c' = c are used.
// The activation operand of a lane is 64 contiguous bytes of one row of X,
// loaded straight from memory.  Partial sums of the waves meet in LDS and are
// added in a fixed order.
//
// Bound: HBM (the code bytes).
#include <hip/hip_runtime.h>

#include "tern_device.h"
#include "tern_mx.h"
#include "tern_mx_device.h"

namespace tern {

namespace {

typedef float float4v_t __attribute__((ext_vector_type(4)));
typedef int int8v_t __attribute__((ext_vector_type(8)));

constexpr int G_STEP = 256;
constexpr int G_MAX_WAVES = 16;

// Activation rows of one matrix tile: 8 slots; an fp16 row takes two.
constexpr int rows_per_set(int xt) { return xt == 0 ? 4 : 8; }

template <int XT, int SETS, int NB>
struct Stage {
    uint4 code[NB];
    uint32_t scale[NB];
    uint4 a[SETS][XT == 2 ? 1 : 4];
    uint32_t ascale[SETS];
};

template <int XT, int SETS, int NB>
__global__ __launch_bounds__(64 * G_MAX_WAVES) void mx_gemv_kernel(const uint8_t *__restrict__ X,
                                                                 const uint8_t *__restrict__ XE,
                                                                 const uint8_t *__restrict__ W,
                                                                 const uint8_t *__restrict__ WE,
                                                                 void *__restrict__ Y, int y_dtype, int64_t M,
                                                                 int64_t N, int64_t blocks, int nw) {
    constexpr int RPS = rows_per_set(XT);
    extern __shared__ float red[];   // [nw][SETS][NB][2 halves][8 slots][8 rows]
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p = lane >> 4, col = lane & 15;
    const int r = col >> 1, c = col & 1;      // as a weight column
    const int ah = col >> 3, as = col & 7;    // as an activation row: half, slot
    const int64_t n0 = (int64_t)blockIdx.x * 8 * NB;
    const int64_t m0 = (int64_t)blockIdx.y * RPS * SETS;
    const int64_t steps = (blocks + 7) / 8;

    const uint8_t *wrow[NB];
    const uint8_t *erow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t n = min(n0 + 8 * b + r, N - 1);
        wrow[b] = W + n * blocks * 16;
        erow[b] = WE + n * blocks;
    }
    int64_t arow[SETS];
#pragma unroll
    for (int t = 0; t < SETS; ++t) arow[t] = min(m0 + t * RPS + (XT == 0 ? as & 3 : as), M - 1);

    float4v_t acc[SETS][NB];
#pragma unroll
    for (int t = 0; t < SETS; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[t][b] = (float4v_t){0.f, 0.f, 0.f, 0.f};

    typedef Stage<XT, SETS, NB> S;
    // A block past the end is read at the last block's address; its weights
    // get the scale 1 (finite) and its activations are zeros.
    auto load = [&](S &st, int64_t s) {
        const int64_t wb = min(8 * s + 4 * c + p, blocks - 1);
        const int64_t ab = min(8 * s + 4 * ah + p, blocks - 1);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            st.code[b] = *reinterpret_cast<const uint4 *>(wrow[b] + wb * 16);
            st.scale[b] = erow[b][wb];
        }
#pragma unroll
        for (int t = 0; t < SETS; ++t) {
            if constexpr (XT == 2) {
                st.a[t][0] = *reinterpret_cast<const uint4 *>(X + (arow[t] * blocks + ab) * 16);
                st.ascale[t] = XE[arow[t] * blocks + ab];
            } else {
                const uint4 *x = reinterpret_cast<const uint4 *>(X + (arow[t] * blocks + ab) * 64);
#pragma unroll
                for (int i = 0; i < 4; ++i) st.a[t][i] = x[i];
            }
        }
    };
    auto compute = [&](S &st, int64_t s) {
        const bool wok = 8 * s + 4 * c + p < blocks;
        const uint32_t keep = 8 * s + 4 * ah + p < blocks ? ~0u : 0u;
#pragma unroll
        for (int t = 0; t < SETS; ++t) {
#pragma unroll
            for (int i = 0; i < (XT == 2 ? 1 : 4); ++i) {
                uint4 &q = st.a[t][i];
                q.x &= keep, q.y &= keep, q.z &= keep, q.w &= keep;
                if constexpr (XT == 0) q = fp16_term(q, as >= 4);
            }
            if constexpr (XT == 2) st.ascale[t] = keep ? st.ascale[t] : 127u;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t e = wok ? st.scale[b] : 127u;
            if constexpr (XT == 2) {
                const int8v_t bv = {(int)st.code[b].x, (int)st.code[b].y, (int)st.code[b].z, (int)st.code[b].w, 0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < SETS; ++t) {
                    const uint4 &q = st.a[t][0];
                    const int8v_t av = {(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                    acc[t][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[t][b], 4, 4, 0,
                                                                                 (int)st.ascale[t], 0, (int)e);
                }
            } else {
                const float f = __builtin_bit_cast(float, e << 23);
                const uint32_t cw[4] = {st.code[b].x, st.code[b].y, st.code[b].z, st.code[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf168_t bv = decode8(cw[i], f);
#pragma unroll
                    for (int t = 0; t < SETS; ++t)
                        acc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168_t, st.a[t][i]), bv,
                                                                           acc[t][b], 0, 0, 0);
                }
            }
        }
    };

    S s0, s1;
    int64_t s = wave;
    if (s < steps) {
        load(s0, s);
        for (;;) {
            if (s + nw < steps) load(s1, s + nw);
            compute(s0, s);
            s += nw;
            if (s >= steps) break;
            if (s + nw < steps) load(s0, s + nw);
            compute(s1, s);
            s += nw;
            if (s >= steps) break;
        }
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
    for (int o = tid; o < SETS * RPS * NB * 8; o += 64 * nw) {
        const int rr = o & 7, b = (o >> 3) % NB, mm = (o >> 3) / NB;
        const int64_t m = m0 + mm, n = n0 + 8 * b + rr;
        if (m >= M || n >= N) continue;
        const int t = mm / RPS, slot = mm % RPS;
        float y = 0.f;
        for (int w = 0; w < nw; ++w) {
            const float *q = red + ((w * SETS + t) * NB + b) * 128 + slot * 8 + rr;
            y += q[0] + q[64];
            if constexpr (XT == 0) y += q[32] + q[96];   // the lo terms' slots
        }
        if (y_dtype == 2) store_out<2>(Y, m * N + n, y);
        else if (y_dtype == 1) store_out<1>(Y, m * N + n, y);
        else store_out<0>(Y, m * N + n, y);
    }
}

template <int XT, int SETS, int NB>
hipError_t launch_t(const MxArgs &a) {
    const int64_t blocks = a.K / 32, steps = (blocks + 7) / 8;
    const int nw = (int)(steps < G_MAX_WAVES ? steps : G_MAX_WAVES);
    const size_t lds = ((size_t)nw * SETS * NB * 128 + 64) * 4;
    const int64_t per = rows_per_set(XT) * SETS;
    const dim3 grid((unsigned)((a.N + 8 * NB - 1) / (8 * NB)), (unsigned)((a.M + per - 1) / per));
    hipLaunchKernelGGL((mx_gemv_kernel<XT, SETS, NB>), grid, dim3(64 * nw), lds, a.stream,
                       static_cast<const uint8_t *>(a.X), a.XE, a.W, a.WE, a.Y, a.y_dtype, a.M, a.N, blocks, nw);
    return hipGetLastError();
}

template <int XT>
hipError_t launch_x(const MxArgs &a) {
    return a.M <= rows_per_set(XT) ? launch_t<XT, 1, 2>(a) : launch_t<XT, 2, 2>(a);
}

}  // namespace

hipError_t launch_mx_gemv(const MxArgs &a0) {
    MxArgs a = a0;
    // the grid's second dimension holds 65535 chunks
    const int64_t rows = 65535 * (int64_t)rows_per_set(0) * 2;
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
