// tern_norm.hip -- root-mean-square norm of rows, with the addition to a residual
// stream before it and outputs in 16 or 32 bits, in 8 bits with scales, or both.
//
// Mathematics, for a row of K values:
//   h = x + r, rounded to the stream's type: the norm takes what the stream holds
//   f = 1 / sqrt(mean of h^2 + eps),  y = (h f) w
//   a = largest |h w| of the row (or of each 128 of it),  q = rint(127 h w / a),
//   scale = a f / 127
// f is the same for a whole row, so that the codes q do not depend on it: they
// follow from h and w alone, and are the same on every machine and in any order
// of the sum.  a is held as an fp32, h w is taken exactly.  In fp32 127 h w / a is
// off by less than 2^-15 (three roundings of a value up to 127): where that could
// change the code, one value in 16000, it is formed anew in 64 bits, in which the
// quotient of these numbers is rounded to the right side of any border.
//
// Squares are summed in 64 bits: no row of any of the types leaves the range, and
// two conversions and additions an element hide behind the loads.  f is applied as
// a power of two and the rest, so that it need not fit an fp32.
//
// Work layout.  TPR threads hold a row in registers, NV times 8 consecutive values
// each, so that everything is read once and written once; a workgroup takes rows
// in turn and keeps its weights.  Rows of up to 2048 values are a wave's or a part
// of one and need no barrier, longer ones one each.
//
// Bound: HBM.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tern_device.h"
#include "tern_q8.h"

namespace tern {

namespace {

template <int T>
struct Elem;
template <>
struct Elem<0> {
    typedef _Float16 type;
};
template <>
struct Elem<1> {
    typedef __bf16 type;
};
template <>
struct Elem<2> {
    typedef float type;
};

// 8 consecutive elements at any address that their type allows, `n` of them (the rest is `fill`).
template <typename E>
__device__ __forceinline__ void load8_of(const E *at, int n, float fill, float (&v)[8]) {
    if (n >= 8) {
        E e[8];
        __builtin_memcpy(e, at, sizeof(e));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)at[i] : fill;
    }
}

template <typename E>
__device__ __forceinline__ void store8_of(E *at, int n, const float (&v)[8]) {
    if (n >= 8) {
        E e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = (E)v[i];
        __builtin_memcpy(at, e, sizeof(e));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) at[i] = (E)v[i];
    }
}

__device__ __forceinline__ void load8_any(const void *at, int dtype, int64_t i, int n, float fill, float (&v)[8]) {
    if (dtype == 2) load8_of(static_cast<const float *>(at) + i, n, fill, v);
    else if (dtype == 1) load8_of(static_cast<const __bf16 *>(at) + i, n, fill, v);
    else load8_of(static_cast<const _Float16 *>(at) + i, n, fill, v);
}

__device__ __forceinline__ void store8_any(void *at, int dtype, int64_t i, int n, const float (&v)[8]) {
    if (dtype == 2) store8_of(static_cast<float *>(at) + i, n, v);
    else if (dtype == 1) store8_of(static_cast<__bf16 *>(at) + i, n, v);
    else store8_of(static_cast<_Float16 *>(at) + i, n, v);
}

template <int CTRL>
__device__ __forceinline__ uint32_t move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ double move(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)move<CTRL>((uint32_t)b) | (uint64_t)move<CTRL>((uint32_t)(b >> 32)) << 32);
}

// Sums and maxima over a row of 16 lanes, the same for each of them.
__device__ __forceinline__ double row_sum(double v) {
    v += move<0x128>(v);
    v += move<0x124>(v);
    v += move<0x122>(v);
    v += move<0x121>(v);
    return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, move<0x128>(v));
    v = max(v, move<0x124>(v));
    v = max(v, move<0x122>(v));
    v = max(v, move<0x121>(v));
    return v;
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); }
__device__ __forceinline__ double lane_of(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)lane_of((uint32_t)b, l) | (uint64_t)lane_of((uint32_t)(b >> 32), l) << 32);
}

// The codes of 8 values h w, whose neighbours' largest magnitude is a, a byte each.
__device__ __forceinline__ uint64_t codes_of(const float (&h)[8], const float (&w)[8], float a) {
    const float inv = 127.f / a;
    bool sure = a >= 0x1p-100f;   // 127 / a fits an fp32
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = h[i] * w[i] * inv, r = __builtin_rintf(t);
        sure = sure && __builtin_fabsf(t - r) < 0.5f - 0x1p-15f;
        n[i] = (int)r;
    }
    if (!sure) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float hi = h[0], wi = w[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) hi = i == j ? h[j] : hi, wi = i == j ? w[j] : wi;
            const int c = (int)__builtin_rint(127.0 * ((double)hi * (double)wi) / (double)a);
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] = i == j ? c : n[j];
        }
    }
    uint32_t b[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        b[j] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[4 * j + 3], n[4 * j + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(n[4 * j + 1], n[4 * j], 0x0C0C0400u), 0x05040100u);
    return b[0] | (uint64_t)b[1] << 32;
}

// XT: type of X; RT: of the residual, -1 without one.
template <int XT, int RT, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
    constexpr int NT = TPR < 256 ? 256 : TPR, ROWS = NT / TPR, WAVES = NT / 64;
    typedef typename Elem<XT>::type X;
    typedef typename Elem<(RT < 0 ? 0 : RT)>::type R;
    __shared__ double sums[2][WAVES];
    __shared__ uint32_t tops[2][WAVES];
    const int tid = threadIdx.x, t = tid % TPR, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = (int)a.K;
    const bool grouped = a.grouped != 0, coded = a.Q != nullptr;
    // Read twice, by then from the L1: held in registers they cost as many as the row itself.
    auto weights = [&](int k, float (&w)[8]) __attribute__((always_inline)) {
        if (a.W != nullptr) {
            load8_any(a.W, a.w_dtype, k, K - k, 1.f, w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
        }
    };
    int slot = 0;
    // every thread of a workgroup takes part in each turn: rows past the last one are read as row M - 1
    // and not written
    for (int64_t row0 = (int64_t)blockIdx.x * ROWS; row0 < a.M; row0 += (int64_t)gridDim.x * ROWS) {
        const bool there = row0 + tid / TPR < a.M;
        const int64_t row = there ? row0 + tid / TPR : a.M - 1, at = row * K;
        float h[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int k = (v * TPR + t) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = 0.f;
            if (k < K) load8_of(static_cast<const X *>(a.X) + at + k, K - k, 0.f, h[v]);
        }
        if constexpr (RT >= 0) {
            float r[NV][8];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int k = (v * TPR + t) * 8;
                if (k < K) load8_of(static_cast<const R *>(a.R) + at + k, K - k, 0.f, r[v]);
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int k = (v * TPR + t) * 8;
                if (k >= K) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] = (float)(R)(h[v][i] + r[v][i]);
                if (there) store8_of(static_cast<R *>(a.H) + at + k, K - k, h[v]);
            }
        }
        double sum = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)h[v][i], (double)h[v][i], sum);
        }
        sum = row_sum(sum);
        // magnitudes as integers: their order is that of the values, NaN above infinity
        uint32_t top[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) top[v] = 0;
        if (coded) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int k = (v * TPR + t) * 8;
                float w[8];
                if (k < K) {
                    weights(k, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        top[v] = max(top[v], __builtin_bit_cast(uint32_t, h[v][i] * w[i]) & 0x7FFFFFFFu);
                }
            }
            if (grouped) {   // 128 values are 16 lanes' 8
#pragma unroll
                for (int v = 0; v < NV; ++v) top[v] = row_max(top[v]);
            } else {
#pragma unroll
                for (int v = 1; v < NV; ++v) top[0] = max(top[0], top[v]);
                top[0] = row_max(top[0]);
            }
        }
        if constexpr (TPR >= 64) {
            sum = (lane_of(sum, 0) + lane_of(sum, 16)) + (lane_of(sum, 32) + lane_of(sum, 48));
            if (!grouped)
                top[0] = max(max(lane_of(top[0], 0), lane_of(top[0], 16)), max(lane_of(top[0], 32), lane_of(top[0], 48)));
        }
        if constexpr (TPR > 64) {
            // two slots in turn: a wave writes one again only after a barrier that follows its last read
            if (lane == 0) {
                sums[slot][wave] = sum;
                if (!grouped) tops[slot][wave] = top[0];
            }
            __syncthreads();
            sum = 0;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) sum += sums[slot][i];
            if (!grouped) {
#pragma unroll
                for (int i = 0; i < WAVES; ++i) top[0] = max(top[0], tops[slot][i]);
            }
            slot ^= 1;
        }
        // f = f1 f2, f1 a power of two
        double f = 1.0;
        if (a.normalize) f = 1.0 / __builtin_sqrt(sum / K + (double)a.eps);
        const int e = min(max((int)(__builtin_bit_cast(uint64_t, f) >> 52 & 0x7FF) - 1023, -126), 127);
        const float f1 = __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
        const float f2 = (float)(f / (double)f1);
        if (!there) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int k = (v * TPR + t) * 8;
            if (k >= K) continue;
            float w[8];
            weights(k, w);
            if (a.Y != nullptr) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = h[v][i] * f1 * f2 * w[i];
                store8_any(a.Y, a.y_dtype, at + k, K - k, y);
            }
            if (coded) {
                const uint32_t bits = grouped ? top[v] : top[0];
                // 0 for a block of zeros, NaN for one with an infinity or a NaN; the codes are 0 in both
                const float most = __builtin_bit_cast(float, bits);
                const bool some = bits - 1 < 0x7F7FFFFFu;
                float scale = (float)((double)most * f / 127.0);
                if (!some) scale = bits != 0 ? __builtin_nanf("") : f == f ? 0.f : (float)f;
                const uint64_t q = some ? codes_of(h[v], w, most) : 0;
                int8_t *qp = a.Q + at + k;
                if (K - k >= 8) {
                    __builtin_memcpy(qp, &q, 8);
                } else {
                    for (int i = 0; i < K - k; ++i) qp[i] = (int8_t)(q >> (8 * i));
                }
                if (grouped ? k % 128 == 0 : k == 0) a.S[grouped ? (at + k) / 128 : row] = scale;
            }
        }
    }
}

template <int XT, int RT, int TPR, int NV>
hipError_t launch_t(const NormArgs &a) {
    constexpr int NT = TPR < 256 ? 256 : TPR, ROWS = NT / TPR;
    // enough workgroups to fill every CU, each with rows left to take in turn
    const int64_t need = (a.M + ROWS - 1) / ROWS, most = 256 * (2048 / NT);
    hipLaunchKernelGGL((norm_kernel<XT, RT, TPR, NV>), dim3((unsigned)std::min(need, most)), dim3(NT), 0, a.stream, a);
    return hipGetLastError();
}

template <int XT, int RT>
hipError_t launch_row(const NormArgs &a) {
    if (a.K <= 128) return launch_t<XT, RT, 16, 1>(a);
    if (a.K <= 512) return launch_t<XT, RT, 64, 1>(a);
    if (a.K <= 1024) return launch_t<XT, RT, 64, 2>(a);
    if (a.K <= 2048) return launch_t<XT, RT, 256, 1>(a);
    if (a.K <= 4096) return launch_t<XT, RT, 256, 2>(a);
    if (a.K <= 6144) return launch_t<XT, RT, 256, 3>(a);
    if (a.K <= 12288) return launch_t<XT, RT, 512, 3>(a);
    if (a.K <= 20480) return launch_t<XT, RT, 512, 5>(a);
    if (a.K <= 32768) return launch_t<XT, RT, 1024, 4>(a);
    return launch_t<XT, RT, 1024, 8>(a);
}

template <int YT>
__global__ __launch_bounds__(256) void q8_dequant_kernel(const int8_t *__restrict__ Q, const float *__restrict__ S,
                                                         void *__restrict__ Y, int64_t M, int K, int lanes) {
    typedef typename Elem<YT>::type E;
    const int rows = 256 / lanes, t = threadIdx.x % lanes;
    for (int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / lanes; row < M; row += (int64_t)gridDim.x * rows) {
        const float s = S[row];
        const int64_t at = row * K;
        for (int k = (blockIdx.y * lanes + t) * 8; k < K; k += gridDim.y * lanes * 8) {
            float q[8];
            load8_of(Q + at + k, K - k, 0.f, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] *= s;
            store8_of(static_cast<E *>(Y) + at + k, K - k, q);
        }
    }
}

}  // namespace

// The residual has X's type or is fp32.
hipError_t launch_norm(const NormArgs &a) {
    if (a.R == nullptr) {
        if (a.x_dtype == 0) return launch_row<0, -1>(a);
        return a.x_dtype == 1 ? launch_row<1, -1>(a) : launch_row<2, -1>(a);
    }
    if (a.r_dtype == 2) {
        if (a.x_dtype == 0) return launch_row<0, 2>(a);
        return a.x_dtype == 1 ? launch_row<1, 2>(a) : launch_row<2, 2>(a);
    }
    return a.x_dtype == 0 ? launch_row<0, 0>(a) : launch_row<1, 1>(a);
}

hipError_t launch_q8_dequant(const int8_t *Q, const float *S, void *Y, int y_dtype, int64_t M, int64_t K,
                             hipStream_t stream) {
    int lanes = 16;
    while (lanes < 256 && lanes * 8 < K) lanes *= 2;
    const int64_t rows = 256 / lanes, need = (M + rows - 1) / rows, across = (K + lanes * 8 - 1) / (lanes * 8);
    const dim3 g((unsigned)std::min<int64_t>(need, 8192), (unsigned)std::min<int64_t>(across, 64)), b(256);
    if (y_dtype == 0) hipLaunchKernelGGL(q8_dequant_kernel<0>, g, b, 0, stream, Q, S, Y, M, (int)K, lanes);
    else if (y_dtype == 1) hipLaunchKernelGGL(q8_dequant_kernel<1>, g, b, 0, stream, Q, S, Y, M, (int)K, lanes);
    else hipLaunchKernelGGL(q8_dequant_kernel<2>, g, b, 0, stream, Q, S, Y, M, (int)K, lanes);
    return hipGetLastError();
}

}  // namespace tern
