// tern_mx.hip -- quantisation to microscaled 4-bit floats and back.
//
// Mathematics.  For a block of 32 values with largest magnitude a, the scale
// is 2^E with E = max(floor(log2 a) - 2, -127): the top binade of e2m1 is
// [4, 8), so a / 2^E lies in it.  Each value is rounded to the nearest of the
// 8 magnitudes of value / 2^E, ties to the even code; what exceeds 6 becomes
// 6 (the format has nothing above).  A block with an infinity or a NaN gets
// the exponent byte 255 and zero codes: it reads back as NaN.  Scaling by a
// power of two is exact in fp32, so the rounding to 4 bits is the only one.
//
// In bits: floor(log2 a) + 127 is the exponent field of a as fp32 (fields 0
// and 1 both end at the lower limit), so the byte is max(field - 2, 0).
//
// Bound: HBM.
#include <hip/hip_runtime.h>

#include "tern_device.h"
#include "tern_mx.h"

namespace tern {

namespace {

typedef float float2v_t __attribute__((ext_vector_type(2)));

// 8 consecutive elements as fp32.
template <int XT>
__device__ __forceinline__ void load8(const void *X, int64_t octet, float (&v)[8]) {
    if constexpr (XT == 2) {
        const float4 a = static_cast<const float4 *>(X)[2 * octet], b = static_cast<const float4 *>(X)[2 * octet + 1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 q = static_cast<const uint4 *>(X)[octet];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (XT == 1) {
                v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
                v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
            } else {
                v[2 * i] = f16_bits_to_float((uint16_t)w[i]);
                v[2 * i + 1] = f16_bits_to_float((uint16_t)(w[i] >> 16));
            }
        }
    }
}

// One lane per octet, the 4 lanes of a DPP quad per block.
template <int XT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void *__restrict__ X, uint32_t *__restrict__ codes,
                                                          uint8_t *__restrict__ exps, int64_t octets) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    // octets is a multiple of 4, so a quad is in range or out of it as a whole
    for (int64_t o = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; o < octets; o += stride) {
        float v[8];
        load8<XT>(X, o, v);
        uint32_t mag = 0;   // fp32 magnitudes compare as integers, NaN above infinity
#pragma unroll
        for (int i = 0; i < 8; ++i) mag = max(mag, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
        mag = max(mag, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mag, 0xB1, 0xF, 0xF, true));
        mag = max(mag, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)mag, 0x4E, 0xF, 0xF, true));
        const uint32_t field = mag >> 23;
        const bool bad = field == 255;
        const uint32_t e = bad ? 255u : (field > 2 ? field - 2 : 0u);
        const float inv = __builtin_bit_cast(float, (bad ? 0u : 254u - e) << 23);   // 2^(127 - e)
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.0f, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.0f, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.0f, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.0f, 3);
        codes[o] = bad ? 0u : c;
        if ((o & 3) == 0) exps[o >> 2] = (uint8_t)e;
    }
}

typedef uint32_t uint4v_t __attribute__((ext_vector_type(4)));

template <bool STREAM, typename T>
__device__ __forceinline__ void store16(void *to, int64_t at, T a, T b, T c, T d) {
    const uint4v_t v = {__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                        __builtin_bit_cast(uint32_t, d)};
    if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<uint4v_t *>(to) + at);
    else static_cast<uint4v_t *>(to)[at] = v;
}

// One lane per octet (4 code bytes).
template <int WT, bool STREAM>
__global__ __launch_bounds__(256) void mx_dequant_kernel(const uint32_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ exps, void *__restrict__ W,
                                                         int64_t octets) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t o = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; o < octets; o += stride) {
        const uint32_t c = codes[o];
        // the conversion reads the exponent field of its scale operand: 0 is
        // 2^-127 and 255 gives NaN (checked over every byte and code)
        const float s = __builtin_bit_cast(float, (uint32_t)exps[o >> 2] << 23);
        float2v_t f[4];
        f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
        f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
        f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
        f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
        if constexpr (WT == 2) {
            store16<STREAM>(W, 2 * o, f[0][0], f[0][1], f[1][0], f[1][1]);
            store16<STREAM>(W, 2 * o + 1, f[2][0], f[2][1], f[3][0], f[3][1]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (WT == 1) {
                    const bf162_t b = {(__bf16)f[i][0], (__bf16)f[i][1]};
                    w[i] = __builtin_bit_cast(uint32_t, b);
                } else {
                    const half2_t b = {(_Float16)f[i][0], (_Float16)f[i][1]};
                    w[i] = __builtin_bit_cast(uint32_t, b);
                }
            }
            store16<STREAM>(W, o, w[0], w[1], w[2], w[3]);
        }
    }
}

unsigned octet_grid(int64_t octets) {
    const int64_t g = (octets + 255) / 256;
    return (unsigned)(g < 8192 ? g : 8192);
}

}  // namespace

hipError_t launch_mx_quantize(const void *X, int x_dtype, uint8_t *codes, uint8_t *exps, int64_t blocks,
                              hipStream_t stream) {
    const int64_t octets = blocks * 4;
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
    const dim3 g(octet_grid(octets)), b(256);
    if (x_dtype == 0) hipLaunchKernelGGL(mx_quantize_kernel<0>, g, b, 0, stream, X, c, exps, octets);
    else if (x_dtype == 1) hipLaunchKernelGGL(mx_quantize_kernel<1>, g, b, 0, stream, X, c, exps, octets);
    else hipLaunchKernelGGL(mx_quantize_kernel<2>, g, b, 0, stream, X, c, exps, octets);
    return hipGetLastError();
}

// A matrix that the L2s cannot hold is written past them: what it would leave behind there is
// written back while the next kernel runs (17408 x 5120 to bf16: 41 -> 34 us, and 87 -> 72 for the
// quantisation after it).
constexpr int64_t kStreamBytes = 32 << 20;

template <int WT>
hipError_t dequant(const uint32_t *codes, const uint8_t *exps, void *W, int64_t octets, hipStream_t stream) {
    const bool past = octets * (WT == 2 ? 32 : 16) > kStreamBytes;
    constexpr auto past_l2 = &mx_dequant_kernel<WT, true>, through_l2 = &mx_dequant_kernel<WT, false>;
    hipLaunchKernelGGL(past ? past_l2 : through_l2, dim3(octet_grid(octets)), dim3(256), 0, stream, codes, exps, W, octets);
    return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t *codes, const uint8_t *exps, void *W, int w_dtype, int64_t blocks,
                             hipStream_t stream) {
    const uint32_t *c = reinterpret_cast<const uint32_t *>(codes);
    const int64_t octets = blocks * 4;
    if (w_dtype == 0) return dequant<0>(c, exps, W, octets, stream);
    return w_dtype == 1 ? dequant<1>(c, exps, W, octets, stream) : dequant<2>(c, exps, W, octets, stream);
}

}  // namespace tern
