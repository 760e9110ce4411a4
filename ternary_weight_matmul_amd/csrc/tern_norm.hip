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
// change the code, one value in 16000, it is decided in 64 bits: h w is exact there,
// and so is any border (n + 1/2) a, so that one fused multiply-add tells on which side
// of it 127 h w lies.  (The quotient itself may round to the border: 127 h w has up to
// 55 bits.)
//
// Squares are summed in 64 bits: no row of any of the types leaves the range.  f is
// applied as a power of two and the rest, so that it need not fit an fp32.
//
// Work layout.  A row of up to 32768 values stays in the registers of its threads, NV
// times 8 consecutive values each, so that everything is read once and written once;
// a workgroup takes rows in turn, keeps its weights, and asks for the next row while
// it works on one.
// Rows of up to 1024 values are a wave's or a part of one and need no barrier,
// longer ones one each.
//
// Bound: HBM where there are thousands of rows (2048 x 5120 with a residual stream
// 20.9 us, 4.0 TB/s, inputs and outputs over more than the last-level cache), else
// the way of the first row's lines from memory.  With 8-bit outputs it is the vector
// instructions and what they wait for, one after the other: 2048 x 5120 takes 24.5
// us, of which 31 instructions a value (squares in 64 bits, codes) keep a SIMD busy
// for 8, and the 10 waves of a CU wait for memory or for each other for 53% of their
// time.  Above 12288 values there is one workgroup a CU, and nothing of its next row
// on the way: 333 x 17408 22.9 us (the copy's rate gives 11.9), two rows one after
// the other on 77 of the CUs; 2048 x 17408 without a norm 67 (20.0).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tern_device.h"
#include "tern_q8.h"
#include "tern_tile.h"

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

// 8 consecutive elements at any address that their type allows.
template <typename E>
__device__ __forceinline__ void load8_of(const E *at, float (&v)[8]) {
    E e[8];
    __builtin_memcpy(e, at, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
}

template <typename E>
__device__ __forceinline__ void store8_of(E *at, const float (&v)[8]) {
    E e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = (E)v[i];
    __builtin_memcpy(at, e, sizeof(e));
}

__device__ __forceinline__ void load8_any(const void *at, int dtype, int64_t i, float (&v)[8]) {
    if (dtype == 2) load8_of(static_cast<const float *>(at) + i, v);
    else if (dtype == 1) load8_of(static_cast<const __bf16 *>(at) + i, v);
    else load8_of(static_cast<const _Float16 *>(at) + i, v);
}

__device__ __forceinline__ void store8_any(void *at, int dtype, int64_t i, const float (&v)[8]) {
    if (dtype == 2) store8_of(static_cast<float *>(at) + i, v);
    else if (dtype == 1) store8_of(static_cast<__bf16 *>(at) + i, v);
    else store8_of(static_cast<_Float16 *>(at) + i, v);
}

__device__ __forceinline__ float load_any(const void *at, int dtype, int64_t i) {
    if (dtype == 2) return static_cast<const float *>(at)[i];
    return dtype == 1 ? (float)static_cast<const __bf16 *>(at)[i] : (float)static_cast<const _Float16 *>(at)[i];
}

__device__ __forceinline__ void store_any(void *at, int dtype, int64_t i, float v) {
    if (dtype == 2) static_cast<float *>(at)[i] = v;
    else if (dtype == 1) static_cast<__bf16 *>(at)[i] = (__bf16)v;
    else static_cast<_Float16 *>(at)[i] = (_Float16)v;
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

// 1 / sqrt(x) in 64 bits: the instruction's estimate, good to 2^-24, and a Newton step.  x = 0 and
// infinity have no step.
__device__ __forceinline__ double inverse_root(double x) {
    const double y = __builtin_amdgcn_rsq(x), z = y * __builtin_fma(-0.5 * x * y, y, 1.5);
    return z == z ? z : y;
}

// The codes of 8 values h w, whose neighbours' largest magnitude is a, a byte each.  127 h w / a plus
// 1.5 2^23 has the nearest integer in its low bits.
__device__ __forceinline__ uint64_t codes_of(const float (&h)[8], const float (&w)[8], float a) {
    const float about = __builtin_amdgcn_rcpf(a), inv = 127.f * fmaf(fmaf(-a, about, 1.f), about, about);
    float u[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = h[i] * w[i];
        u[i] = fmaf(p, inv, 0x1.8p23f);
        off = fmaxf(off, __builtin_fabsf(fmaf(p, inv, -(u[i] - 0x1.8p23f))));
    }
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = __builtin_bit_cast(uint32_t, u[i]);
    if (!(off < 0.5f - 0x1p-15f && a >= 0x1p-100f && a <= 0x1p100f)) {   // beyond, 1 / a leaves fp32
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            float hi = h[0], wi = w[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) hi = i == j ? h[j] : hi, wi = i == j ? w[j] : wi;
            const double p = (double)hi * (double)wi;
            // the instruction's estimate is good to 2^-20 at least, and next to an integer either of the codes
            // beside it will do as `below`
            const int below = (int)floor(127.0 * p * __builtin_amdgcn_rcp((double)a));
            // (below + 1/2) a is exact, and its difference to 127 p has the right sign
            const double past = __builtin_fma(127.0, p, -((double)below + 0.5) * (double)a);
            // an a below the normal range may be a third less than the value that it stands for: cut off
            const uint32_t c = (uint32_t)max(min(below + (past > 0.0 || (past == 0.0 && (below & 1))), 127), -127);
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

// f = f1 f2, f1 a power of two.
struct Factor {
    double f;
    float f1, f2;
};
__device__ __forceinline__ Factor factor_of(double sum, double per, double eps, bool normalize) {
    const double f = normalize ? inverse_root(__builtin_fma(sum, per, eps)) : 1.0;
    const int e = min(max((int)(__builtin_bit_cast(uint64_t, f) >> 52 & 0x7FF) - 1023, -126), 127);
    return {f, __builtin_bit_cast(float, (uint32_t)(e + 127) << 23),
            (float)(f * __builtin_bit_cast(double, (uint64_t)(1023 - e) << 52))};
}

// The scale of a block whose largest magnitude has these bits: 0 for a block of zeros, NaN for one
// with an infinity or a NaN; the codes are 0 in both.
__device__ __forceinline__ bool has_codes(uint32_t bits) { return bits - 1 < 0x7F7FFFFFu; }
__device__ __forceinline__ float scale_of(uint32_t bits, double f) {
    if (has_codes(bits)) return (float)((double)__builtin_bit_cast(float, bits) * f * (1.0 / 127.0));
    return bits != 0 ? __builtin_nanf("") : f == f ? 0.f : (float)f;
}

// XT: type of X; RT: of the residual, -1 without one.  TPR: threads of a row, 16 or 64 of a workgroup
// of 256, or 0: the workgroup's, up to MOST.  8 <= K <= 8 NV threads.
// The last of a row's eights begins at K - 8 and shares values with the one before it: every load is
// whole.  What is shared counts once in the sum, and is written twice alike.
template <int XT, int RT, int TPR, int NV, int MOST>
__global__ __launch_bounds__(MOST) void norm_kernel(NormArgs a) {
    constexpr int ROWS = TPR > 0 ? MOST / TPR : 1;
    // The next row is asked for while this one is worked on, where there are registers for it.
    constexpr bool AHEAD = NV <= 3;
    typedef typename Elem<XT>::type X;
    typedef typename Elem<(RT < 0 ? 0 : RT)>::type R;
    __shared__ double sums[2][16];
    __shared__ uint32_t tops[2][16];
    const int tid = threadIdx.x, threads = TPR > 0 ? TPR : blockDim.x, t = TPR > 0 ? tid % threads : tid, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int my_row = TPR > 0 ? tid / threads : 0;
    const int K = (int)a.K;
    const bool grouped = a.grouped != 0, coded = a.Q != nullptr;
    auto first = [&](int v) __attribute__((always_inline)) { return min((v * threads + t) * 8, K - 8); };
    struct Eights {
        X x[8];
        R r[8];
    };
    auto ask = [&](Eights (&e)[NV], int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int v = 0; v < NV; ++v) __builtin_memcpy(e[v].x, static_cast<const X *>(a.X) + row * K + first(v), sizeof(e[v].x));
        if constexpr (RT >= 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) __builtin_memcpy(e[v].r, static_cast<const R *>(a.R) + row * K + first(v), sizeof(e[v].r));
        }
    };
    // every thread of a workgroup takes part in each turn: rows past the last one are read as row M - 1
    // and not written
    auto mine = [&](int64_t row0) __attribute__((always_inline)) { return min(row0 + my_row, a.M - 1); };
    const double per = 1.0 / K;
    int64_t row0 = (int64_t)blockIdx.x * ROWS;
    Eights e[NV];
    ask(e, mine(row0));
    float w[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (a.W != nullptr) {
            load8_any(a.W, a.w_dtype, first(v), w[v]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[v][i] = 1.f;
        }
    }
    int slot = 0;
    for (;;) {
        const bool there = row0 + my_row < a.M;
        const int64_t row = mine(row0), at = row * K;
        row0 += (int64_t)gridDim.x * ROWS;
        float h[NV][8];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[v][i] = (float)e[v].x[i];
                if constexpr (RT >= 0) h[v][i] = (float)(R)(h[v][i] + (float)e[v].r[i]);
            }
        }
        if constexpr (AHEAD) {
            if (row0 < a.M) ask(e, mine(row0));
        }
        double sum = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int twice = (v * threads + t) * 8 - first(v);
            double s = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) s = __builtin_fma((double)h[v][i], (double)h[v][i], s);
            if (twice > 0) {
                s = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= twice) s = __builtin_fma((double)h[v][i], (double)h[v][i], s);
            }
            sum += s;
        }
        sum = row_sum(sum);
        // magnitudes as integers: their order is that of the values, NaN above infinity
        uint32_t top[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) top[v] = 0;
        if (coded) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top[v] = max(top[v], __builtin_bit_cast(uint32_t, h[v][i] * w[v][i]) & 0x7FFFFFFFu);
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
        if constexpr (TPR != 16) {
            sum = (lane_of(sum, 0) + lane_of(sum, 16)) + (lane_of(sum, 32) + lane_of(sum, 48));
            if (!grouped)
                top[0] = max(max(lane_of(top[0], 0), lane_of(top[0], 16)), max(lane_of(top[0], 32), lane_of(top[0], 48)));
        }
        if constexpr (TPR == 0) {
            // two slots in turn: a wave writes one again only after a barrier that follows its last read
            if (lane == 0) {
                sums[slot][wave] = sum;
                if (!grouped) tops[slot][wave] = top[0];
            }
            wait_and_meet<63>();   // not for loads and stores
            // 16 lanes take the waves'
            const int i = lane & 15, waves = threads >> 6;
            sum = row_sum(i < waves ? sums[slot][i] : 0.0);
            if (!grouped) top[0] = row_max(i < waves ? tops[slot][i] : 0u);
            slot ^= 1;
        }
        const Factor f = factor_of(sum, per, (double)a.eps, a.normalize != 0);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int k = first(v);
            if (!there || (v * threads + t) * 8 >= K) continue;
            // all of the row has been read by now: H may be R
            if constexpr (RT >= 0) store8_of(static_cast<R *>(a.H) + at + k, h[v]);
            if (a.Y != nullptr) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = h[v][i] * f.f1 * f.f2 * w[v][i];
                store8_any(a.Y, a.y_dtype, at + k, y);
            }
            if (coded) {
                const uint32_t bits = grouped ? top[v] : top[0];
                const uint64_t q = has_codes(bits) ? codes_of(h[v], w[v], __builtin_bit_cast(float, bits)) : 0;
                __builtin_memcpy(a.Q + at + k, &q, 8);
                if (t % 16 == 0 && (grouped || v * threads + t == 0)) a.S[grouped ? (at + k) / 128 : row] = scale_of(bits, f.f);
            }
        }
        if (row0 >= a.M) break;
        if constexpr (!AHEAD) ask(e, mine(row0));
    }
}

// Rows too long for registers: a workgroup of 1024 reads one twice, the second time from the L2 (64 rows of
// 65536 to 8 bits 37 us; read once, with 94 to 160 registers in scratch memory, 1.6 times as long.  Two
// registers still are there).  8 values a thread in turn, 4 turns' asked for at once; the last ones one by
// one, as the stream may be written in place and no value may be read after that as if it were x or r.
template <int XT, int RT>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    constexpr int NT = 1024, TOGETHER = 4;
    typedef typename Elem<XT>::type X;
    typedef typename Elem<(RT < 0 ? XT : RT)>::type R;   // of the stream
    __shared__ double sums[2][16];
    __shared__ uint32_t tops[2][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = (int)a.K;
    const bool grouped = a.grouped != 0, coded = a.Q != nullptr;
    auto load = [&](const auto *from, int k, auto (&e)[8]) __attribute__((always_inline)) {
        if (k + 8 <= K) {
            __builtin_memcpy(e, from + k, sizeof(e));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = k + i < K ? from[k + i] : 0;
        }
    };
    auto weights = [&](int k, float (&w)[8]) __attribute__((always_inline)) {
        if (a.W != nullptr && k + 8 <= K) {
            load8_any(a.W, a.w_dtype, k, w);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = a.W != nullptr && k + i < K ? load_any(a.W, a.w_dtype, k + i) : 1.f;
        }
    };
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const int64_t at = row * K;
        const X *x = static_cast<const X *>(a.X) + at;
        double sum = 0;
        uint32_t top = 0;
        for (int k0 = tid * 8; k0 < K; k0 += TOGETHER * NT * 8) {
            X ex[TOGETHER][8];
            R er[TOGETHER][8];
#pragma unroll
            for (int v = 0; v < TOGETHER; ++v) {
                load(x, k0 + v * NT * 8, ex[v]);
                if constexpr (RT >= 0) load(static_cast<const R *>(a.R) + at, k0 + v * NT * 8, er[v]);
            }
#pragma unroll
            for (int v = 0; v < TOGETHER; ++v) {
                const int k = k0 + v * NT * 8;
                float h[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[i] = (float)ex[v][i];
                    if constexpr (RT >= 0) h[i] = (float)(R)(h[i] + (float)er[v][i]);
                    sum = __builtin_fma((double)h[i], (double)h[i], sum);   // zeros past the end
                }
                if constexpr (RT >= 0) {
                    R *stream = static_cast<R *>(a.H) + at;
                    if (k + 8 <= K) {
                        store8_of(stream + k, h);
                    } else {
                        for (int i = 0; i < 8; ++i)
                            if (k + i < K) stream[k + i] = (R)h[i];
                    }
                }
                if (coded && !grouped) {
                    float w[8];
                    weights(k, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, h[i] * w[i]) & 0x7FFFFFFFu);
                }
            }
        }
        sum = row_sum(sum), top = row_max(top);
        sum = (lane_of(sum, 0) + lane_of(sum, 16)) + (lane_of(sum, 32) + lane_of(sum, 48));
        top = max(max(lane_of(top, 0), lane_of(top, 16)), max(lane_of(top, 32), lane_of(top, 48)));
        if (lane == 0) sums[slot][wave] = sum, tops[slot][wave] = top;
        wait_and_meet<63>();   // as above
        sum = row_sum(sums[slot][lane & 15]), top = row_max(tops[slot][lane & 15]);
        slot ^= 1;
        const Factor f = factor_of(sum, 1.0 / K, (double)a.eps, a.normalize != 0);
        if (coded && !grouped && tid == 0) a.S[row] = scale_of(top, f.f);
        const R *stream = static_cast<const R *>(RT >= 0 ? a.H : a.X) + at;
        for (int k0 = tid * 8; k0 < K; k0 += TOGETHER * NT * 8) {
            R e[TOGETHER][8];
#pragma unroll
            for (int v = 0; v < TOGETHER; ++v) load(stream, k0 + v * NT * 8, e[v]);
#pragma unroll
            for (int v = 0; v < TOGETHER; ++v) {
                const int k = k0 + v * NT * 8;
                if (k >= K) continue;
                float h[8], w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = (float)e[v][i];
                weights(k, w);
                if (a.Y != nullptr) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = h[i] * f.f1 * f.f2 * w[i];
                    if (k + 8 <= K) {
                        store8_any(a.Y, a.y_dtype, at + k, y);
                    } else {
                        for (int i = 0; i < K - k; ++i) store_any(a.Y, a.y_dtype, at + k + i, y[i]);
                    }
                }
                if (coded) {
                    uint32_t bits = top;
                    if (grouped) {   // 128 values are 16 lanes' 8, all of them here
                        bits = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) bits = max(bits, __builtin_bit_cast(uint32_t, h[i] * w[i]) & 0x7FFFFFFFu);
                        bits = row_max(bits);
                        if (tid % 16 == 0) a.S[(at + k) / 128] = scale_of(bits, f.f);
                    }
                    const uint64_t q = has_codes(bits) ? codes_of(h, w, __builtin_bit_cast(float, bits)) : 0;
                    if (k + 8 <= K) {
                        __builtin_memcpy(a.Q + at + k, &q, 8);
                    } else {
                        for (int i = 0; i < K - k; ++i) a.Q[at + k + i] = (int8_t)(q >> (8 * i));
                    }
                }
            }
        }
    }
}

// Rows of fewer than 8 values, one to a thread.
__global__ __launch_bounds__(256) void norm_short_kernel(NormArgs a) {
    const int K = (int)a.K;
    for (int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x; row < a.M; row += (int64_t)gridDim.x * 256) {
        const int64_t at = row * K;
        float h[8], w[8];
        double sum = 0;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = min(i, K - 1);
            h[i] = i < K ? load_any(a.X, a.x_dtype, at + k) : 0.f;
            if (a.R != nullptr && i < K) {
                h[i] = h[i] + load_any(a.R, a.r_dtype, at + k);
                store_any(a.H, a.r_dtype, at + k, h[i]);
                h[i] = load_any(a.H, a.r_dtype, at + k);
            }
            w[i] = a.W != nullptr ? load_any(a.W, a.w_dtype, k) : 1.f;
            sum = __builtin_fma((double)h[i], (double)h[i], sum);
            if (i < K) top = max(top, __builtin_bit_cast(uint32_t, h[i] * w[i]) & 0x7FFFFFFFu);
        }
        const Factor f = factor_of(sum, 1.0 / K, (double)a.eps, a.normalize != 0);
        const uint64_t q = a.Q != nullptr && has_codes(top) ? codes_of(h, w, __builtin_bit_cast(float, top)) : 0;
        if (a.Q != nullptr) a.S[row] = scale_of(top, f.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= K) continue;
            if (a.Y != nullptr) store_any(a.Y, a.y_dtype, at + i, h[i] * f.f1 * f.f2 * w[i]);
            if (a.Q != nullptr) a.Q[at + i] = (int8_t)(q >> (8 * i));
        }
    }
}

template <int XT, int RT, int TPR, int NV, int MOST>
hipError_t launch_t(const NormArgs &a) {
    const int threads = TPR > 0 ? MOST : (int)((a.K + 512 * NV - 1) / (512 * NV)) * 64;
    constexpr int ROWS = TPR > 0 ? MOST / TPR : 1;
    // Up to 16 waves a CU, in as many workgroups as give the busiest CU the fewest rows: 2048 x 5120 with
    // a residual took 18.3 us (outputs in the cache), against 22.3 with up to 20 waves, and 20.9 with the
    // most workgroups of 16 waves that there is room for.
    const int64_t need = (a.M + ROWS - 1) / ROWS;
    int64_t grid = 0, least = 0;
    for (int64_t c = std::max(16 * 64 / threads, 1); c >= 1; --c) {
        const int64_t rows = (need + 256 * c - 1) / (256 * c) * c;
        if (grid == 0 || rows < least) least = rows, grid = 256 * c;
    }
    grid = std::min(grid, need);
    hipLaunchKernelGGL((norm_kernel<XT, RT, TPR, NV, MOST>), dim3((unsigned)grid), dim3(threads), 0, a.stream, a);
    return hipGetLastError();
}

// Two eights a thread up to 8192, which leaves room for many waves (three: 2048 x 8192 29.7 us against
// 25.4, 2048 x 5119 24.5 against 21.8), then as few as the workgroup's threads allow.  Without a residual
// three would gain at some sizes (4096 x 6144 19.9 against 22.6); they follow the same rule.
template <int XT, int RT>
hipError_t launch_row(const NormArgs &a) {
    if (a.K <= 128) return launch_t<XT, RT, 16, 1, 256>(a);
    if (a.K <= 512) return launch_t<XT, RT, 64, 1, 256>(a);
    if (a.K <= 1024) return launch_t<XT, RT, 64, 2, 256>(a);
    if (a.K <= 8192) return launch_t<XT, RT, 0, 2, 512>(a);
    if (a.K <= 12288) return launch_t<XT, RT, 0, 3, 512>(a);
    if (a.K <= 32768) return launch_t<XT, RT, 0, 4, 1024>(a);
    hipLaunchKernelGGL((norm_long_kernel<XT, RT>), dim3((unsigned)std::min<int64_t>(a.M, 512)), dim3(1024), 0, a.stream, a);
    return hipGetLastError();
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
            if (K - k >= 8) {
                float q[8];
                load8_of(Q + at + k, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] *= s;
                store8_of(static_cast<E *>(Y) + at + k, q);
            } else {
                for (int i = k; i < K; ++i) static_cast<E *>(Y)[at + i] = (E)((float)Q[at + i] * s);
            }
        }
    }
}

}  // namespace

// The residual has X's type or is fp32.
hipError_t launch_norm(const NormArgs &a) {
    if (a.K < 8) {
        hipLaunchKernelGGL(norm_short_kernel, dim3((unsigned)std::min<int64_t>((a.M + 255) / 256, 4096)), dim3(256), 0, a.stream, a);
        return hipGetLastError();
    }
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
