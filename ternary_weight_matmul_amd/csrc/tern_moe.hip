// tern_moe.hip -- a mixture-of-experts layer with ternary experts, from the
// router's logits to the summed outputs, for a few tokens.
//
// Mathematics, for token t with logits l:
//   S = the top_k experts by logit (ties to the lowest index; NaN counts as
//       the largest; an expert whose logit is -inf is never taken)
//   w[e] = exp(l[e]) / sum of exp(l) over S (renormalised) or over all experts
//   h[e] = silu(Wg[e] x) * (Wu[e] x),  y = sum over e in S of w[e] Wd[e] h[e]
// with ternary Wg, Wu (the two halves of gate_up) and Wd.  The weights become
// +-2 / 0 operands (tern_device.h) of the 16-bit matrix instructions, a
// 128-weight block's fp32 sum is multiplied by its fp16 scale.  The hidden
// values stay fp32 and enter the down product as two bf16 terms, hi = bf16(h)
// and lo = bf16(h - hi): 16 significant bits, so that this product adds no
// rounding that a 16-bit output would show.
//
// Work layout of both products.  Waves of a workgroup split K into 512-weight
// steps.  Lane (p = lane / 16, col = 4 r + c) loads the 8 code bytes of slice
// p of block c of row r of a 4-row quad: one instruction reads 4 rows x 128
// contiguous bytes.  Tile row i = 4 c' + s holds activation slot s in block c',
// so that only the results with c' = c are used, each with its own scale.
//
// Bound: HBM (the codes of the experts that are taken, once for all of their
// tokens).
#include <hip/hip_runtime.h>

#include "tern_device.h"
#include "tern_moe.h"

namespace tern {

namespace {

typedef __bf16 bf168_t __attribute__((ext_vector_type(8)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4v_t __attribute__((ext_vector_type(4)));

constexpr int E_STEP = 512;
constexpr int E_MAX_WAVES = 16;

// ---- routing ------------------------------------------------------------------

__device__ __forceinline__ float load_logit(const void *l, int dtype, int64_t i) {
    if (dtype == 2) return static_cast<const float *>(l)[i];
    if (dtype == 1) return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(l)[i] << 16);
    return f16_bits_to_float(static_cast<const uint16_t *>(l)[i]);
}

// Unsigned key in the order of the values: NaN above all, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v != v ? __builtin_bit_cast(float, 0x7FC00000u) : v + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

// One wave routes one token: lane j < top_k returns the j-th expert and its
// weight (-1 and 0 where there is none).
__device__ void route_token(const void *logits, int l_dtype, int64_t row, int E, int top_k, bool renorm, int lane,
                            int &id, float &weight) {
    const int64_t base = row * E;
    id = -1;
    float mine = 0.f;       // logit of this lane's choice
    uint64_t last = ~0ull;  // key of the choice before
    float top = 0.f;
    for (int j = 0; j < top_k; ++j) {
        // the largest (value, lowest index) key below the last one taken
        uint64_t best = 0;
        for (int e = lane; e < E; e += 64) {
            const uint64_t k = ((uint64_t)order_key(load_logit(logits, l_dtype, base + e)) << 32) | (uint32_t)(~e);
            if (k < last && k > best) best = k;
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)best, m);
            best = o > best ? o : best;
        }
        last = best;
        const int e = (int)~(uint32_t)best;
        const float v = load_logit(logits, l_dtype, base + e);
        if (j == 0) top = v;
        if (lane == j) {
            id = v == -__builtin_inff() ? -1 : e;
            mine = v;
        }
    }
    float part;
    if (renorm) {
        part = lane < top_k && id >= 0 ? expf(mine - top) : 0.f;
    } else {
        part = 0.f;
        for (int e = lane; e < E; e += 64) {
            const float v = load_logit(logits, l_dtype, base + e);
            if (v != -__builtin_inff()) part += expf(v - top);
        }
    }
    const float total = wave_sum(part);
    weight = id >= 0 ? expf(mine - top) / total : 0.f;
}

__global__ __launch_bounds__(64) void moe_route_kernel(const void *__restrict__ logits, int l_dtype, int E, int top_k,
                                                       int renorm, int *__restrict__ ids, float *__restrict__ weights) {
    const int lane = threadIdx.x;
    int id;
    float w;
    route_token(logits, l_dtype, blockIdx.x, E, top_k, renorm != 0, lane, id, w);
    if (lane < top_k) {
        ids[blockIdx.x * top_k + lane] = id;
        weights[blockIdx.x * top_k + lane] = w;
    }
}

// ---- the expert of a workgroup and its (token, choice) pairs ----------------------

// The pairs [0, P) of the idx-th taken expert, in order, in `list`; returns
// their number (0: fewer experts are taken) and the expert.  Called by the
// whole workgroup.  `flags` holds kMoeMaxExperts / 32 words and two more.
__device__ int expert_pairs(const int *__restrict__ ids, int P, int E, int idx, int tid, int nthreads, uint32_t *flags,
                            uint16_t *list, int &expert) {
    const int words = (E + 31) / 32;
    for (int i = tid; i < words; i += nthreads) flags[i] = 0;
    __syncthreads();
    for (int i = tid; i < P; i += nthreads) {
        const int e = ids[i];
        if (e >= 0) atomicOr(&flags[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (tid < 64) {
        int left = idx, e = -1;
        for (int w = 0; w < words && e < 0; ++w) {
            uint32_t f = flags[w];
            const int n = __popc(f);
            if (left >= n) {
                left -= n;
                continue;
            }
            for (; left > 0; --left) f &= f - 1;
            e = 32 * w + __ffs(f) - 1;
        }
        int count = 0;
        if (e >= 0) {
            for (int b = 0; b < P; b += 64) {
                const bool hit = b + tid < P && ids[b + tid] == e;
                const uint64_t m = __ballot(hit);
                if (hit) list[count + __popcll(m & ((1ull << tid) - 1))] = (uint16_t)(b + tid);
                count += __popcll(m);
            }
        }
        if (tid == 0) {
            flags[kMoeMaxExperts / 32] = (uint32_t)count;
            flags[kMoeMaxExperts / 32 + 1] = (uint32_t)e;
        }
    }
    __syncthreads();
    expert = (int)flags[kMoeMaxExperts / 32 + 1];
    return (int)flags[kMoeMaxExperts / 32];
}

// ---- the product --------------------------------------------------------------

// AT: activations fp16 (0), bf16 (1) or fp32 (2: hi and lo bf16 terms).
constexpr int slots_rows(int at) { return at == 2 ? 2 : 4; }

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const bf162_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// hi or lo bf16 terms of 8 fp32 values.
__device__ __forceinline__ uint4 fp32_term(const uint4 &a, const uint4 &b, bool lo) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __builtin_bit_cast(float, w[2 * i]), y = __builtin_bit_cast(float, w[2 * i + 1]);
        const uint32_t hi = bf16_pair(x, y);
        const float xh = __builtin_bit_cast(float, hi << 16), yh = __builtin_bit_cast(float, hi & 0xFFFF0000u);
        // an infinite hi (infinity itself, or a value that rounds to it) has no rest
        const uint32_t rest = bf16_pair(__builtin_isinf(xh) ? 0.f : x - xh, __builtin_isinf(yh) ? 0.f : y - yh);
        o[i] = lo ? rest : hi;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int AT>
__device__ __forceinline__ float4v_t mfma16(const uint4 &a, const uint4 &b, const float4v_t &c) {
    if constexpr (AT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168_t, a), __builtin_bit_cast(bf168_t, b), c,
                                                       0, 0, 0);
}

// The wave's share (steps wave, wave + nw, ...) of Q quads times SETS tiles of
// activation rows.  row[q] / srow[q]: this lane's weight row and its scales;
// arow[t]: this lane's activation row.  acc[t][q][v]: slot v, used where p = c.
template <int AT, int SETS, int Q>
__device__ __forceinline__ void product(const uint8_t *const (&row)[Q], const uint16_t *const (&srow)[Q],
                                        const char *const (&arow)[SETS], int groups, int wave, int nw, int lane,
                                        float4v_t (&acc)[SETS][Q]) {
    constexpr int AQ = AT == 2 ? 8 : 4;   // 16-byte loads of a lane's 32 activations
    const int p = lane >> 4, col = lane & 15, c = col & 3, ca = col >> 2;
    const int steps = (groups + 3) / 4;
    const bool lo = AT == 2 && (col & 3) >= 2;
    for (int s = wave; s < steps; s += nw) {
        const int wb = min(4 * s + c, groups - 1);
        const int ab = min(4 * s + ca, groups - 1);
        const bool wok = 4 * s + c < groups;
        const uint32_t keep = 4 * s + ca < groups ? ~0u : 0u;
        uint2 code[Q];
        uint16_t sc[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            code[q] = *reinterpret_cast<const uint2 *>(row[q] + (int64_t)wb * 32 + p * 8);
            sc[q] = srow[q][wb];
        }
        uint4 a[SETS][4];   // the 4 operands of a lane's 32 activations, pair-interleaved
#pragma unroll
        for (int t = 0; t < SETS; ++t) {
            const uint4 *x = reinterpret_cast<const uint4 *>(arow[t] + ((int64_t)ab * 128 + p * 32) * (AT == 2 ? 4 : 2));
            uint4 raw[AQ];
#pragma unroll
            for (int i = 0; i < AQ; ++i) {
                raw[i] = x[i];
                raw[i].x &= keep, raw[i].y &= keep, raw[i].z &= keep, raw[i].w &= keep;
            }
            uint4 e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (AT == 2) e[i] = fp32_term(raw[2 * i], raw[2 * i + 1], lo);
                else e[i] = raw[i];
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t w[8];
                interleave16(e[2 * g], e[2 * g + 1], w);
                a[t][2 * g] = make_uint4(w[0], w[1], w[2], w[3]);
                a[t][2 * g + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint64_t v = sign_nz_fields64<true>((uint64_t)code[q].x | ((uint64_t)code[q].y << 32));
            uint32_t l[8], h[8];
            weight_pairs2<0, true>(v, l[0], h[0]);
            weight_pairs2<1, true>(v, l[1], h[1]);
            weight_pairs2<2, true>(v, l[2], h[2]);
            weight_pairs2<3, true>(v, l[3], h[3]);
            weight_pairs2<4, true>(v, l[4], h[4]);
            weight_pairs2<5, true>(v, l[5], h[5]);
            weight_pairs2<6, true>(v, l[6], h[6]);
            weight_pairs2<7, true>(v, l[7], h[7]);
            const uint4 b[4] = {make_uint4(l[0], l[1], l[2], l[3]), make_uint4(l[4], l[5], l[6], l[7]),
                                make_uint4(h[0], h[1], h[2], h[3]), make_uint4(h[4], h[5], h[6], h[7])};
            const float scale = wok ? f16_bits_to_float(sc[q]) : 0.f;
#pragma unroll
            for (int t = 0; t < SETS; ++t) {
                float4v_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i) d = mfma16<AT>(a[t][i], b[i], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][q][i] = fmaf(scale, d[i], acc[t][q][i]);
            }
        }
    }
}

// The wave's sums into red[wave][t][q][slot][r][c] (unused lanes into a spare word).
template <int SETS, int Q>
__device__ __forceinline__ void store_sums(float *red, int wave, int nw, int lane, const float4v_t (&acc)[SETS][Q]) {
    const int p = lane >> 4, col = lane & 15, r = col >> 2, c = col & 3;
    const int spare = nw * SETS * Q * 64 + lane;
#pragma unroll
    for (int t = 0; t < SETS; ++t)
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int at = ((wave * SETS + t) * Q + q) * 64 + v * 16 + r * 4 + c;
                red[p == c ? at : spare] = acc[t][q][v];
            }
}

template <int SETS, int Q>
__device__ __forceinline__ float sum_of(const float *red, int nw, int t, int q, int slot, int r) {
    float y = 0.f;
    for (int w = 0; w < nw; ++w) {
        const float4 v = *reinterpret_cast<const float4 *>(red + ((w * SETS + t) * Q + q) * 64 + slot * 16 + r * 4);
        y += (v.x + v.y) + (v.z + v.w);
    }
    return 0.5f * y;   // the weights were +-2
}

// LDS: sums, then the expert flags, then the pair list.
template <int SETS, int Q>
constexpr size_t red_words(int nw) {
    return (size_t)nw * SETS * Q * 64 + 64;
}
constexpr int FLAG_WORDS = kMoeMaxExperts / 32 + 2;

// h[pair][f] = silu(g) * u.  Quads [0, Q/2) are gate rows, the rest the up rows of the same f.
template <int AT, int SETS, int Q>
__global__ __launch_bounds__(64 * E_MAX_WAVES) void moe_up_kernel(const char *__restrict__ X,
                                                                const uint8_t *__restrict__ GU,
                                                                const uint16_t *__restrict__ GUS,
                                                                const int *__restrict__ ids, float *__restrict__ Hid,
                                                                int P, int E, int top_k, int H, int F, int nw) {
    static_assert(Q % 2 == 0, "gate and up quads");
    extern __shared__ float4 lds4[];
    float *red = reinterpret_cast<float *>(lds4);
    uint32_t *flags = reinterpret_cast<uint32_t *>(red + red_words<SETS, Q>(nw));
    uint16_t *list = reinterpret_cast<uint16_t *>(flags + FLAG_WORDS);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int e;
    const int count = expert_pairs(ids, P, E, blockIdx.y, tid, 64 * nw, flags, list, e);
    if (count == 0) return;
    const int groups = H >> 7;
    const int f0 = blockIdx.x * 2 * Q;
    const int col = lane & 15, r = col >> 2, slot = col & 3;
    const uint8_t *row[Q];
    const uint16_t *srow[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int f = min(f0 + 4 * (q % (Q / 2)) + r, F - 1);
        const int64_t n = (int64_t)e * 2 * F + (q < Q / 2 ? 0 : F) + f;
        row[q] = GU + n * (H / 4);
        srow[q] = GUS + n * groups;
    }
    constexpr int RPS = slots_rows(AT);
    for (int base = 0; base < count; base += RPS * SETS) {
        const char *arow[SETS];
#pragma unroll
        for (int t = 0; t < SETS; ++t)
            arow[t] = X + (int64_t)(list[min(base + t * RPS + slot, count - 1)] / top_k) * H * 2;
        float4v_t acc[SETS][Q];
#pragma unroll
        for (int t = 0; t < SETS; ++t)
#pragma unroll
            for (int q = 0; q < Q; ++q) acc[t][q] = (float4v_t){0.f, 0.f, 0.f, 0.f};
        product<AT, SETS, Q>(row, srow, arow, groups, wave, nw, lane, acc);
        if (base > 0) __syncthreads();   // the sums of the chunk before are read
        store_sums<SETS, Q>(red, wave, nw, lane, acc);
        __syncthreads();
        for (int o = tid; o < SETS * RPS * 2 * Q; o += 64 * nw) {
            const int ff = o % (2 * Q), i = o / (2 * Q);
            if (base + i >= count || f0 + ff >= F) continue;
            const float g = sum_of<SETS, Q>(red, nw, i / RPS, ff / 4, i % RPS, ff % 4);
            const float u = sum_of<SETS, Q>(red, nw, i / RPS, ff / 4 + Q / 2, i % RPS, ff % 4);
            Hid[(int64_t)list[base + i] * F + f0 + ff] = g / (1.f + expf(-g)) * u;
        }
    }
}

// part[pair][n] = weight * (Wd h)[n].
template <int SETS, int Q>
__global__ __launch_bounds__(64 * E_MAX_WAVES) void moe_down_kernel(const float *__restrict__ Hid,
                                                                  const uint8_t *__restrict__ D,
                                                                  const uint16_t *__restrict__ DS,
                                                                  const int *__restrict__ ids,
                                                                  const float *__restrict__ weights,
                                                                  float *__restrict__ part, int P, int E, int H, int F,
                                                                  int nw) {
    extern __shared__ float4 lds4[];
    float *red = reinterpret_cast<float *>(lds4);
    uint32_t *flags = reinterpret_cast<uint32_t *>(red + red_words<SETS, Q>(nw));
    uint16_t *list = reinterpret_cast<uint16_t *>(flags + FLAG_WORDS);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int e;
    const int count = expert_pairs(ids, P, E, blockIdx.y, tid, 64 * nw, flags, list, e);
    if (count == 0) return;
    const int groups = F >> 7;
    const int n0 = blockIdx.x * 4 * Q;
    const int col = lane & 15, r = col >> 2, slot = col & 3;
    const uint8_t *row[Q];
    const uint16_t *srow[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int64_t n = (int64_t)e * H + min(n0 + 4 * q + r, H - 1);
        row[q] = D + n * (F / 4);
        srow[q] = DS + n * groups;
    }
    constexpr int RPS = slots_rows(2);
    for (int base = 0; base < count; base += RPS * SETS) {
        const char *arow[SETS];
#pragma unroll
        for (int t = 0; t < SETS; ++t)
            arow[t] = reinterpret_cast<const char *>(Hid + (int64_t)list[min(base + t * RPS + (slot & 1), count - 1)] * F);
        float4v_t acc[SETS][Q];
#pragma unroll
        for (int t = 0; t < SETS; ++t)
#pragma unroll
            for (int q = 0; q < Q; ++q) acc[t][q] = (float4v_t){0.f, 0.f, 0.f, 0.f};
        product<2, SETS, Q>(row, srow, arow, groups, wave, nw, lane, acc);
        if (base > 0) __syncthreads();   // the sums of the chunk before are read
        store_sums<SETS, Q>(red, wave, nw, lane, acc);
        __syncthreads();
        for (int o = tid; o < SETS * RPS * 4 * Q; o += 64 * nw) {
            const int nn = o % (4 * Q), i = o / (4 * Q);
            if (base + i >= count || n0 + nn >= H) continue;
            const int t = i / RPS, k = i % RPS;
            const float y = sum_of<SETS, Q>(red, nw, t, nn / 4, k, nn % 4) +
                            sum_of<SETS, Q>(red, nw, t, nn / 4, k + 2, nn % 4);
            const int pair = list[base + i];
            part[(int64_t)pair * H + n0 + nn] = weights[pair] * y;
        }
    }
}

// y[t][n] = the sum of the token's parts, in the order of its choices.
__global__ __launch_bounds__(256) void moe_sum_kernel(const float *__restrict__ part, const int *__restrict__ ids,
                                                      void *__restrict__ Y, int y_dtype, int top_k, int H) {
    const int t = blockIdx.y;
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= H) return;
    float y = 0.f;
    for (int j = 0; j < top_k; ++j)
        if (ids[t * top_k + j] >= 0) y += part[((int64_t)t * top_k + j) * H + n];
    const int64_t at = (int64_t)t * H + n;
    if (y_dtype == 2) store_out<2>(Y, at, y);
    else if (y_dtype == 1) store_out<1>(Y, at, y);
    else store_out<0>(Y, at, y);
}

int waves_of(int64_t K) {
    const int64_t steps = (K + E_STEP - 1) / E_STEP;
    return (int)(steps < E_MAX_WAVES ? steps : E_MAX_WAVES);
}

template <int SETS, int Q>
size_t lds_bytes(int nw, int64_t P) {
    return (red_words<SETS, Q>(nw) + FLAG_WORDS) * 4 + (size_t)P * 2;
}

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// One chunk of at most kMoeChunk tokens.
hipError_t launch_chunk(const MoeArgs &a) {
    const int P = (int)(a.T * a.top_k);
    char *w = static_cast<char *>(a.ws);
    int *ids = reinterpret_cast<int *>(w);
    w += align256((size_t)P * 4);
    float *weights = reinterpret_cast<float *>(w);
    w += align256((size_t)P * 4);
    float *hid = reinterpret_cast<float *>(w);
    w += align256((size_t)P * a.F * 4);
    float *part = reinterpret_cast<float *>(w);
    hipLaunchKernelGGL(moe_route_kernel, dim3((unsigned)a.T), dim3(64), 0, a.stream, a.logits, a.l_dtype, (int)a.E,
                       (int)a.top_k, a.renormalize, ids, weights);
    const unsigned slots = (unsigned)(a.E < P ? a.E : P);
    {
        constexpr int SETS = 1, Q = 4;
        const int nw = waves_of(a.H);
        const dim3 g((unsigned)((a.F + 2 * Q - 1) / (2 * Q)), slots), b(64 * nw);
        const size_t lds = lds_bytes<SETS, Q>(nw, P);
        if (a.x_dtype == 0)
            hipLaunchKernelGGL((moe_up_kernel<0, SETS, Q>), g, b, lds, a.stream, static_cast<const char *>(a.X), a.GU,
                               a.GUS, ids, hid, P, (int)a.E, (int)a.top_k, (int)a.H, (int)a.F, nw);
        else
            hipLaunchKernelGGL((moe_up_kernel<1, SETS, Q>), g, b, lds, a.stream, static_cast<const char *>(a.X), a.GU,
                               a.GUS, ids, hid, P, (int)a.E, (int)a.top_k, (int)a.H, (int)a.F, nw);
    }
    {
        constexpr int SETS = 1, Q = 4;
        const int nw = waves_of(a.F);
        const dim3 g((unsigned)((a.H + 4 * Q - 1) / (4 * Q)), slots), b(64 * nw);
        const size_t lds = lds_bytes<SETS, Q>(nw, P);
        hipLaunchKernelGGL((moe_down_kernel<SETS, Q>), g, b, lds, a.stream, hid, a.D, a.DS, ids, weights, part, P,
                           (int)a.E, (int)a.H, (int)a.F, nw);
    }
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), dim3(256), 0, a.stream, part,
                       ids, a.Y, a.y_dtype, (int)a.top_k, (int)a.H);
    return hipGetLastError();
}

}  // namespace

size_t moe_workspace(int64_t T, int64_t top_k, int64_t H, int64_t F) {
    const int64_t P = (T < kMoeChunk ? T : kMoeChunk) * top_k;
    return 2 * align256((size_t)P * 4) + align256((size_t)P * F * 4) + align256((size_t)P * H * 4);
}

hipError_t launch_moe(const MoeArgs &a0) {
    MoeArgs a = a0;
    const int64_t lsize = a.l_dtype == 2 ? 4 : 2, ysize = a.y_dtype == 2 ? 4 : 2;
    for (int64_t t = 0; t < a0.T; t += kMoeChunk) {
        a.T = a0.T - t < kMoeChunk ? a0.T - t : kMoeChunk;
        a.X = static_cast<const char *>(a0.X) + t * a.H * 2;
        a.logits = static_cast<const char *>(a0.logits) + t * a.E * lsize;
        a.Y = static_cast<char *>(a0.Y) + t * a.H * ysize;
        const hipError_t e = launch_chunk(a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tern
