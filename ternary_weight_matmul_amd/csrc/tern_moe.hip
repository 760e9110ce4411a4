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
// 128-weight block's fp32 sum is multiplied by its fp16 scale.  v = w h, an
// fp32, is handed to the down product as bf16 terms that sum up to it: t1 =
// bf16(v), t2 = bf16(v - t1), t3 = v - t1 - t2.  An fp32 output takes all three,
// which is v exactly.  A 16-bit output takes two, which is v to 2^-16, a 32nd of
// the half step of fp16: an error of sum |v Wd| 2^-16, for half the slots (an
// fp32 output instead of a 16-bit one: 1 token 12.9 us either way, 32 tokens of
// the sizes below 68 -> 85, 4 tokens of 8 experts of 5120 x 2048 25 -> 41).  The
// terms are those of v / 4, so that no term and no product with +-2 leaves the
// fp32 range before v does.
//
// Launches.  Up to kMoeSmall tokens take two: the up kernel, whose workgroups
// each route every token anew (a microsecond, against two for a launch of its
// own), and a down kernel whose workgroups own output rows, go through all
// taken experts and sum in registers.  More tokens take four: routing and the
// list of each expert's tokens, up, down with a partial output per (token,
// choice), and the sum of a token's partials.
//
// Work layout of up and down.  A workgroup works for one expert: it holds the
// activations of the expert's tokens in LDS, as the matrix instructions take
// them, and each wave takes units of Q quads of weight rows over all of K.
// Lane (p = lane / 16, col = 4 r + c) loads the 8 code bytes of slice p of
// block c of row r of a quad: one instruction reads 4 rows x 128 contiguous
// bytes.  Tile row i = 4 c' + s holds activation slot s in block c', so that
// only the results with c' = c are used, each with its own scale.  A quad's
// loads are refilled, G steps of 512 weights ahead, as soon as it is used; the
// first are on their way before the activations are fetched.
//   With K split over the waves instead, sums met in LDS once a block of rows,
// each behind a barrier: 107 us for both products at 32 tokens of the sizes
// below, against 58.
//
// Bound: latency for one token (E = 64, k = 8, 2048 x 1024: 12.6 MB of codes,
// 3.7 us for a plain read; up 8.4 us, routing first, and down 5.4).  At 32
// tokens (97 MB, 16 us) decoding the codes, 36 vector instructions a quad and
// step, and the 4 or 8 matrix instructions they feed: 29 + 28 us, and 7 + 5
// for the plan and the sum.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "tern_buffer.h"
#include "tern_device.h"
#include "tern_launch.h"
#include "tern_moe.h"

namespace tern {

namespace {

typedef __bf16 bf168_t __attribute__((ext_vector_type(8)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4v_t __attribute__((ext_vector_type(4)));

// What every lane holds, in a scalar register: a buffer descriptor made from anything else is
// gathered lane by lane in a loop around each load.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- routing ------------------------------------------------------------------

__device__ __forceinline__ float load_logit(const void *l, int dtype, int64_t i) {
    if (dtype == 2) return static_cast<const float *>(l)[i];
    if (dtype == 1) return __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(l)[i] << 16);
    return f16_bits_to_float(static_cast<const uint16_t *>(l)[i]);
}

// Unsigned key in the order of the values, never 0: NaN above all, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v != v ? __builtin_bit_cast(float, 0x7FC00000u) : v + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
    return __builtin_bit_cast(float, (k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// Maximum over the wave, the same for every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<0x128>(v));   // rotations within rows of 16
    v = max(v, dpp<0x124>(v));
    v = max(v, dpp<0x122>(v));
    v = max(v, dpp<0x121>(v));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    auto lane_of = [&](int l) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
    };
    return (lane_of(0) + lane_of(16)) + (lane_of(32) + lane_of(48));
}

// One wave routes one token: lane j < top_k gets the j-th expert and its
// weight (-1 and 0 where there is none).  E <= 64 R.
template <int R>
__device__ __forceinline__ void route_token(const void *logits, int l_dtype, int64_t row, int E, int top_k, bool renorm,
                                            int lane, int &id, float &weight) {
    uint32_t key[R], all[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = 64 * i + lane;
        const float v = load_logit(logits, l_dtype, row * E + min(e, E - 1));
        all[i] = key[i] = e < E ? order_key(v) : 0u;
    }
    id = -1;
    uint32_t mine = 0, top = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < R; ++i) m = max(m, key[i]);
        m = wave_max(m);
        if (j == 0) top = m;
        int e = -1;   // the lowest index that holds it
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint64_t hit = __ballot(key[i] == m);
            if (e < 0 && hit != 0) {
                e = 64 * i + __ffsll((unsigned long long)hit) - 1;
                if (lane == (e & 63)) key[i] = 0;
            }
        }
        if (lane == j) id = e, mine = m;
    }
    const float t = key_value(top), v = key_value(mine), ninf = -__builtin_inff();
    if (lane >= top_k || v == ninf) id = -1;
    float part = 0.f;
    if (renorm) {
        if (id >= 0) part = expf(v - t);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float l = key_value(all[i]);
            if (all[i] != 0 && l != ninf) part += expf(l - t);
        }
    }
    const float total = wave_sum(part);
    weight = id >= 0 ? expf(v - t) / total : 0.f;
}

__device__ __forceinline__ void route_any(const void *logits, int l_dtype, int64_t row, int E, int top_k, bool renorm,
                                          int lane, int &id, float &weight) {
    if (E <= 64) route_token<1>(logits, l_dtype, row, E, top_k, renorm, lane, id, weight);
    else if (E <= 128) route_token<2>(logits, l_dtype, row, E, top_k, renorm, lane, id, weight);
    else if (E <= 256) route_token<4>(logits, l_dtype, row, E, top_k, renorm, lane, id, weight);
    else route_token<16>(logits, l_dtype, row, E, top_k, renorm, lane, id, weight);
}

// Index of the n-th set bit over `words` words, -1 if there are fewer.
__device__ __forceinline__ int nth_bit(const uint32_t *bits, int words, int n) {
    for (int w = 0; w < words; ++w) {
        uint32_t f = bits[w];
        const int c = __popc(f);
        if (n >= c) {
            n -= c;
            continue;
        }
        for (; n > 0; --n) f &= f - 1;
        return 32 * w + __ffs(f) - 1;
    }
    return -1;
}

// 16-bit words of a pair's hidden values in so many terms.
__host__ __device__ constexpr int64_t hid_words(int64_t F, int terms) { return (F + 511) / 512 * 512 * terms; }

// What the kernels hand on in the workspace.
struct Plan {
    int *ids;            // [P] expert of a (token, choice) pair, -1: none
    float *weights;      // [P]
    int *experts;        // [slots] the taken experts
    int *start;          // [slots + 1] where an expert's pairs start, start[i] = start[i + 1]: not taken
    int *pairs;          // [P] pairs by expert
    uint16_t *hid;       // [P, steps of F, 2 or 3 terms, 512] bf16: weight * hidden value / 4
    float *part;         // [P, H]
};

// More tokens: routing and the lists, by one workgroup of 16 waves.
__global__ __launch_bounds__(1024) void moe_plan_kernel(const void *__restrict__ logits, int l_dtype, int T, int E,
                                                        int top_k, int renorm, int slots, Plan plan) {
    __shared__ int ids[kMoeChunk * kMoeMaxTopK];
    __shared__ int count[kMoeMaxExperts], place[kMoeMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int P = T * top_k;
    for (int e = tid; e < E; e += 1024) count[e] = 0;
    for (int t = wave; t < T; t += 16) {
        int id;
        float w;
        route_any(logits, l_dtype, t, E, top_k, renorm != 0, lane, id, w);
        if (lane < top_k) {
            ids[t * top_k + lane] = id;
            plan.ids[t * top_k + lane] = id;
            plan.weights[t * top_k + lane] = w;
        }
    }
    __syncthreads();
    for (int i = tid; i < P; i += 1024)
        if (ids[i] >= 0) atomicAdd(&count[ids[i]], 1);
    __syncthreads();
    if (wave == 0) {   // running sums over the experts: slots and starts
        int slot = 0, start = 0;
        for (int b = 0; b < E; b += 64) {
            const int e = b + lane, n = e < E ? count[e] : 0;
            int sum = n;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(sum, d);
                if (lane >= d) sum += o;
            }
            const uint64_t taken = __ballot(n > 0);
            if (n > 0) {
                const int s = slot + __popcll(taken & ((1ull << lane) - 1));
                plan.experts[s] = e;
                plan.start[s] = start + sum - n;
                place[e] = start + sum - n;
            }
            slot += __popcll(taken);
            start += __shfl(sum, 63);
        }
        for (int s = slot + lane; s <= slots; s += 64) plan.start[s] = start;
    }
    __syncthreads();
    // Where a pair stands within its expert's changes the slot it is worked in, not its sums.
    for (int i = tid; i < P; i += 1024)
        if (ids[i] >= 0) plan.pairs[atomicAdd(&place[ids[i]], 1)] = i;
}

// ---- the products' parts --------------------------------------------------------

template <int AT>
__device__ __forceinline__ float4v_t mfma16(const uint4 &a, const uint4 &b, const float4v_t &c) {
    if constexpr (AT == 0)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf168_t, a), __builtin_bit_cast(bf168_t, b), c,
                                                       0, 0, 0);
}

// AT: activations fp16 (0), bf16 (1) or fp32 in that many bf16 terms (2, 3).  Term m of row j of a
// set is in slot j + rows_per_set m; with three terms the fourth slot is empty.
__host__ __device__ constexpr int rows_per_set(int at) { return at == 3 ? 1 : at == 2 ? 2 : 4; }

// Rows of weights and scales: quads [0, Q / 2) in a, the others in b.
struct Rows {
    __amdgpu_buffer_rsrc_t a, b, sa, sb;
};

__device__ __forceinline__ Rows rows_of(const uint8_t *W, const uint16_t *S, int64_t na, int64_t nb, int ra, int rb,
                                        int groups) {
    ra = uniform(max(ra, 0)), rb = uniform(max(rb, 0));   // a clamp is a vector instruction
    return {buffer_of(W + na * groups * 32, ra * groups * 32), buffer_of(W + nb * groups * 32, rb * groups * 32),
            buffer_of(S + na * groups, ra * groups * 2), buffer_of(S + nb * groups, rb * groups * 2)};
}

// What a wave holds of one step's weights.  Loads with nothing to read (past the
// end of a row, rows that are not there) have offsets out of range and return
// zeros.
template <int Q>
struct Step {
    uint2 code[Q];
    uint32_t scale[Q];
};

// Offsets of step s in the weight rows, and in their scales.
struct At {
    int code, scale;
};
__device__ __forceinline__ At place_of(int s, int groups, int lane, bool live) {
    const int p = lane >> 4, col = lane & 15, r = col >> 2, blk = 4 * s + (col & 3), at = r * groups + blk;
    if (!live || blk >= groups) return {OUT_OF_RANGE, OUT_OF_RANGE};
    return {at * 32 + p * 8, at * 2};
}

template <int Q>
__device__ __forceinline__ void load_quad(Step<Q> &st, const Rows &w, const At &at, int groups, int q) {
    const int row = 4 * (q % (Q / 2)) * groups;
    st.scale[q] = __builtin_amdgcn_raw_buffer_load_b16(q < Q / 2 ? w.sa : w.sb, at.scale + row * 2, 0, 0);
    st.code[q] = load8<2>(q < Q / 2 ? w.a : w.b, at.code + row * 32);
}

// Activations of the tiles' rows into LDS: operand i of set t of step s at ((s SETS + t) 4 + i) KB,
// 16 bytes a lane, pair-interleaved.  Row j is read from x + off[j] bytes, none if negative.  A
// thread takes 16 values of a row at a time.
template <int SETS>
__device__ __forceinline__ void stage(char *ops, const char *x, const int64_t *off, int groups, int tid, int nthreads) {
    const int per_row = (groups + 3) / 4 * 32;
    for (int i = tid; i < SETS * 4 * per_row; i += nthreads) {
        const int j = i / per_row, k = i - j * per_row;   // row, sixteen of the row
        const int s = k >> 5, ca = (k >> 3) & 3, p = (k >> 1) & 3, g = k & 1;
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
        if (off[j] >= 0 && k < groups * 8) {
            const uint4 *v = reinterpret_cast<const uint4 *>(x + off[j] + k * 32);
            v0 = v[0], v1 = v[1];
        }
        uint32_t w[8];
        interleave16(v0, v1, w);
        char *at = ops + ((s * SETS + j / 4) * 4 + 2 * g) * 1024 + (16 * p + 4 * ca + j % 4) * 16;
        *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(at + 1024) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Where the up kernel leaves hidden value f of a pair, in 16-bit words, each term 512 behind the
// one before: a step's operands in the order in which the down kernels take them, [operand][ca][p][8].
__device__ __forceinline__ int hidden_at(int f, int terms) {
    const int k = f & 511, ca = k >> 7, p = (k >> 5) & 3, x = k & 15, j = x & 7;
    const int i = ((k >> 4) & 1) * 2 + (j >> 2);
    return (f >> 9) * 512 * terms + ((i * 4 + ca) * 4 + p) * 8 + (j & 3) * 2 + (x >> 3);
}

// Hidden values of pairs rowpair[j] into LDS (-1: none), row j in set j / rows_per_set.
template <int AT, int SETS>
__device__ __forceinline__ void stage_hidden(char *ops, const uint16_t *hid, const int *rowpair, int groups, int tid,
                                             int nthreads) {
    constexpr int R = rows_per_set(AT), TERMS = 4 / R;   // with the empty one
    const int steps = (groups + 3) / 4, per_row = steps * TERMS * 64;   // chunks of 16 bytes
    for (int i = tid; i < SETS * R * per_row; i += nthreads) {
        const int j = i / per_row, k = i - j * per_row;
        const int s = k / (TERMS * 64), term = (k >> 6) % TERMS, op = (k >> 4) & 3, ca = (k >> 2) & 3, p = k & 3;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (rowpair[j] >= 0 && 4 * s + ca < groups && term < AT)
            v = *reinterpret_cast<const uint4 *>(hid + (((int64_t)rowpair[j] * steps + s) * AT + term) * 512 + (k & 63) * 8);
        *reinterpret_cast<uint4 *>(ops + ((s * SETS + j / R) * 4 + op) * 1024 + (16 * p + 4 * ca + j % R + R * term) * 16) = v;
    }
}

// The same with token j in row j of one set, no token in rows >= T.
__device__ __forceinline__ void stage_tokens(char *ops, const char *x, int T, int groups, int tid, int nthreads) {
    const int per_row = (groups + 3) / 4 * 32;
    for (int i = tid; i < 4 * per_row; i += nthreads) {
        const int j = i / per_row, k = i - j * per_row;
        const int s = k >> 5, ca = (k >> 3) & 3, p = (k >> 1) & 3, g = k & 1;
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
        if (j < T && k < groups * 8) {
            const uint4 *v = reinterpret_cast<const uint4 *>(x + (int64_t)j * groups * 256 + k * 32);
            v0 = v[0], v1 = v[1];
        }
        uint32_t w[8];
        interleave16(v0, v1, w);
        char *at = ops + (s * 4 + 2 * g) * 1024 + (16 * p + 4 * ca + j) * 16;
        *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(at + 1024) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

struct EverySlot {
    __device__ __forceinline__ bool operator()(int, int) const { return true; }
};

// acc[t] += scale * (codes . a[t]) for one quad, in the slots (t, i) that takes() holds for.
template <int AT, int SETS, typename Takes = EverySlot>
__device__ __forceinline__ void quad(uint2 code, uint32_t scale_bits, const uint4 (&a)[SETS][4], float4v_t (&acc)[SETS],
                                     Takes takes = Takes()) {
    const uint64_t v = sign_nz_fields64<true>((uint64_t)code.x | ((uint64_t)code.y << 32));
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
    const float scale = f16_bits_to_float((uint16_t)scale_bits);
#pragma unroll
    for (int t = 0; t < SETS; ++t) {
        float4v_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) d = mfma16<AT>(a[t][i], b[i], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][i] = fmaf(takes(t, i) ? scale : 0.f, d[i], acc[t][i]);
    }
}

// The sums of a wave into sums[q][t][slot][r][c].  Every lane stores, a lane without a used
// sum into the spare words behind, at the same constant offsets from a base of its own: one
// address register, and no matrix instruction is moved under a partial EXEC mask.
template <int SETS, int Q>
__device__ __forceinline__ void store_sums(float *sums, int lane, const float4v_t (&acc)[Q][SETS]) {
    const int p = lane >> 4, col = lane & 15, r = col >> 2, c = col & 3;
    int at = p == c ? r * 4 + c : Q * SETS * 64 + col;
    asm volatile("" : "+v"(at));   // or the select is repeated for every store
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int t = 0; t < SETS; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) sums[at + (q * SETS + t) * 64 + v * 16] = acc[q][t][v];
}

// One output of a wave's sums.
template <int SETS>
__device__ __forceinline__ float sum_of(const float *sums, int t, int q, int slot, int r) {
    const float4 v = *reinterpret_cast<const float4 *>(sums + (q * SETS + t) * 64 + slot * 16 + r * 4);
    return (v.x + v.y) + (v.z + v.w);
}

// The same over the terms of hidden row i, the smallest first.
template <int AT, int SETS>
__device__ __forceinline__ float sum_of_terms(const float *sums, int i, int q, int r) {
    constexpr int R = rows_per_set(AT);
    float y = sum_of<SETS>(sums, i / R, q, i % R + R * (AT - 1), r);
#pragma unroll
    for (int m = AT - 2; m >= 0; --m) y += sum_of<SETS>(sums, i / R, q, i % R + R * m, r);
    return 2.f * y;   // the weights were +-2, the hidden values quarters
}

// Floats of a wave's sums.
template <int SETS, int Q>
__host__ __device__ constexpr int sums_floats() { return 2 * SETS * Q * 64; }

// LDS of a workgroup: operands, the waves' sums, then what the kernel adds.
template <int SETS>
__host__ __device__ constexpr int ops_bytes(int groups) { return (groups + 3) / 4 * SETS * 4096; }

// The compiler keeps the wave's LDS accesses on their sides.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int SETS, int Q>
__device__ __forceinline__ void clear(float4v_t (&acc)[Q][SETS]) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int t = 0; t < SETS; ++t) acc[q][t] = (float4v_t){0.f, 0.f, 0.f, 0.f};
}

// The wave's units u0, u0 + stride, ... < units of Q quads each, over all of K.  G steps' loads are
// in flight: each is refilled for the next G, or the next unit's first, as soon as it is used.
// ready() fills the operands, rows(u) gives a unit's rows, done(u, sums) is called by the wave.
template <int AT, int SETS, int Q, int G, typename Ready, typename RowsOf, typename Done>
__device__ __forceinline__ void product(Ready ready, const char *ops, float *sums, int u0, int stride, int units,
                                        int groups, int lane, RowsOf rows, Done done) {
    const int steps = (groups + 3) / 4;
    Step<Q> st[G];
    {
        const Rows w = rows(u0);
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const At at = place_of(j, groups, lane, u0 < units);
#pragma unroll
            for (int q = 0; q < Q; ++q) load_quad<Q>(st[j], w, at, groups, q);
        }
    }
    ready();   // the first weights are on their way
    for (int u = u0; u < units; u += stride) {
        float4v_t acc[Q][SETS];
        clear<SETS, Q>(acc);
        for (int s = 0;;) {
            const bool turn = s + G >= steps;   // the next loads are the next unit's
            const Rows w = rows(turn ? u + stride : u);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                uint4 a[SETS][4];
                const char *op = ops + min(s + j, steps - 1) * (SETS * 4096) + lane * 16;
#pragma unroll
                for (int t = 0; t < SETS; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[t][i] = *reinterpret_cast<const uint4 *>(op + (t * 4 + i) * 1024);
                const At at = place_of(turn ? j : s + G + j, groups, lane, !turn || u + stride < units);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    quad<AT, SETS>(st[j].code[q], st[j].scale[q], a, acc[q]);
                    load_quad<Q>(st[j], w, at, groups, q);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if ((s += G) >= steps) break;
        }
        // the wave's own LDS accesses are served in order: only the compiler has to keep it
        store_sums<SETS, Q>(sums, lane, acc);
        wave_order();
        done(u, sums);
        wave_order();
    }
}

// ---- kernels --------------------------------------------------------------------

// Waves of a workgroup of the two products.  At most 128 registers, so that a CU holds two of
// them (32 tokens, 64 experts of 2048 x 1024, 8 a token: up 36.5 -> 33.2 us, down 31.8 -> 29.2).
constexpr int kWaves = 8;
static_assert(kWaves > kMoeSmall, "waves that fetch while others route");

// hid[pair][f] = silu(g) * u, 2 Q values f a unit: quads [0, Q / 2) are gate rows, the rest the up
// rows of the same f.  SMALL: routes by itself while other waves fetch the tokens, the slots are the
// tokens, and the first workgroup leaves the ids behind for the down kernel.
template <int AT, int SETS, int Q, int G, bool SMALL>
__global__ __launch_bounds__(64 * kWaves, 4) void moe_up_kernel(const char *__restrict__ X, const void *__restrict__ logits,
                                                             int l_dtype, const uint8_t *__restrict__ GU,
                                                             const uint16_t *__restrict__ GUS, Plan plan, int T, int E,
                                                             int top_k, int renorm, int H, int F, int terms) {
    static_assert(Q % 2 == 0, "gate and up quads");
    constexpr int ROWS = SETS * rows_per_set(AT);
    static_assert(!SMALL || ROWS >= kMoeSmall, "a slot a token");
    extern __shared__ float4 lds4[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int groups = H >> 7;
    char *ops = reinterpret_cast<char *>(lds4);
    float *sums = reinterpret_cast<float *>(ops + ops_bytes<SETS>(groups));
    int64_t *off = reinterpret_cast<int64_t *>(sums + kWaves * sums_floats<SETS, Q>());
    int *rowpair = reinterpret_cast<int *>(off + ROWS);   // the pair of a row of the tiles, -1: none
    float *rowweight = reinterpret_cast<float *>(rowpair + ROWS);
    int *ids = rowpair + 2 * ROWS, *chosen = ids + kMoeSmall * kMoeMaxTopK;   // SMALL
    uint32_t *bits = reinterpret_cast<uint32_t *>(chosen + 1);
    float *weights = reinterpret_cast<float *>(bits + kMoeMaxExperts / 32);
    int e, count = ROWS, start = 0;
    if constexpr (SMALL) {
        const int P = T * top_k, words = (E + 31) / 32;
        if (wave < T) {   // T <= 4
            int id;
            float w;
            route_any(logits, l_dtype, wave, E, top_k, renorm != 0, lane, id, w);
            if (lane < top_k) {
                ids[wave * top_k + lane] = id;
                weights[wave * top_k + lane] = w;
                if (blockIdx.x == 0 && blockIdx.y == 0) plan.ids[wave * top_k + lane] = id;
            }
        } else {
            if (wave == kWaves - 1 && lane < words) bits[lane] = 0;
            if constexpr (SMALL) stage_tokens(ops, X, T, groups, tid - 64 * T, 64 * (kWaves - T));
        }
        __syncthreads();
        if (wave == 0) {
            for (int i = lane; i < P; i += 64)
                if (ids[i] >= 0) atomicOr(&bits[ids[i] >> 5], 1u << (ids[i] & 31));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
            const int x = nth_bit(bits, words, blockIdx.y);
            if (lane == 0) *chosen = x;
            for (int t = 0; t < T; ++t) {
                const uint64_t m = __ballot(lane < top_k && ids[t * top_k + min(lane, top_k - 1)] == x);
                const int pr = m != 0 ? t * top_k + __ffsll((unsigned long long)m) - 1 : -1;
                if (lane == 0) rowpair[t] = pr, rowweight[t] = weights[max(pr, 0)];
            }
            if (lane >= T && lane < ROWS) rowpair[lane] = -1;
        }
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(*chosen);
        if (e < 0) return;
    } else {
        start = uniform(plan.start[blockIdx.y]);
        count = uniform(plan.start[blockIdx.y + 1]) - start;
        if (count <= 0) return;
        e = uniform(plan.experts[blockIdx.y]);
    }
    const int units = (F + 2 * Q - 1) / (2 * Q);
    int base = 0;
    auto go = [&](auto sets) __attribute__((always_inline)) {
        constexpr int S = decltype(sets)::value, ROWS = S * rows_per_set(AT);
        product<AT, S, Q, G>(
            [&]() __attribute__((always_inline)) {
                if constexpr (!SMALL) {
                    if (base > 0) __syncthreads();   // the operands of the chunk before are read
                    if (tid < ROWS) {
                        const int pr = base + tid < count ? plan.pairs[start + base + tid] : -1;
                        off[tid] = pr >= 0 ? (int64_t)(pr / top_k) * H * 2 : -1;
                        rowpair[tid] = pr;
                        rowweight[tid] = pr >= 0 ? plan.weights[pr] : 0.f;
                    }
                    __syncthreads();
                    stage<S>(ops, X, off, groups, tid, 64 * kWaves);
                    __syncthreads();
                }
            },
            ops, sums + wave * sums_floats<SETS, Q>(), blockIdx.x * kWaves + wave, gridDim.x * kWaves, units, groups, lane,
            [&](int u) __attribute__((always_inline)) {
                const int f0 = u * 2 * Q;
                const int64_t g0 = (int64_t)e * 2 * F + f0;
                return rows_of(GU, GUS, g0, g0 + F, min(2 * Q, F - f0), min(2 * Q, F - f0), groups);
            },
            [&](int u, const float *sm) __attribute__((always_inline)) {
#pragma unroll
                for (int o0 = 0; o0 < ROWS * 2 * Q; o0 += 64) {
                    const int o = o0 + lane, ff = o % (2 * Q), i = min(o / (2 * Q), ROWS - 1), f = u * 2 * Q + ff;
                    // the weights were +-2
                    const float g = 0.5f * sum_of<S>(sm, i / 4, ff / 4, i % 4, ff % 4);
                    const float y = 0.5f * sum_of<S>(sm, i / 4, ff / 4 + Q / 2, i % 4, ff % 4);
                    const int pr = rowpair[i];
                    const float h = 0.25f * (g / (1.f + expf(-g)) * y * rowweight[i]);
                    const __bf16 t1 = (__bf16)h;
                    const float h1 = __builtin_isinf(h) ? 0.f : h - (float)t1;   // infinity has no rest
                    const __bf16 t2 = (__bf16)h1;
                    if (o < ROWS * 2 * Q && pr >= 0 && f < F) {
                        uint16_t *at = plan.hid + (int64_t)pr * hid_words(F, terms) + hidden_at(f, terms);
                        at[0] = __builtin_bit_cast(uint16_t, t1);
                        at[512] = __builtin_bit_cast(uint16_t, t2);
                        if (terms == 3) at[1024] = __builtin_bit_cast(uint16_t, (__bf16)(h1 - (float)t2));
                    }
                }
            });
        base += ROWS;
    };
    while (base < count) {   // one set will do for a few tokens (32 tokens: 33 -> 30 us, down 29 -> 28)
        if (SETS > 1 && count - base <= rows_per_set(AT)) go(std::integral_constant<int, 1>());
        else go(std::integral_constant<int, SETS>());
    }
}

// part[pair][n] = (Wd h)[n], 4 Q values n a unit.
template <int AT, int SETS, int Q, int G>
__global__ __launch_bounds__(64 * kWaves, 4) void moe_down_kernel(const uint8_t *__restrict__ D,
                                                               const uint16_t *__restrict__ DS, Plan plan, int H, int F) {
    extern __shared__ float4 lds4[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int groups = F >> 7;
    char *ops = reinterpret_cast<char *>(lds4);
    float *sums = reinterpret_cast<float *>(ops + ops_bytes<SETS>(groups));
    int *rowpair = reinterpret_cast<int *>(sums + kWaves * sums_floats<SETS, Q>());
    const int start = uniform(plan.start[blockIdx.y]), count = uniform(plan.start[blockIdx.y + 1]) - start;
    if (count <= 0) return;
    const int e = uniform(plan.experts[blockIdx.y]);
    const int units = (H + 4 * Q - 1) / (4 * Q);
    int base = 0;
    auto go = [&](auto sets) __attribute__((always_inline)) {
        constexpr int S = decltype(sets)::value, ROWS = S * rows_per_set(AT);
        product<AT, S, Q, G>(
            [&]() __attribute__((always_inline)) {
                if (base > 0) __syncthreads();   // the operands of the chunk before are read
                if (tid < ROWS) rowpair[tid] = base + tid < count ? plan.pairs[start + base + tid] : -1;
                __syncthreads();
                stage_hidden<AT, S>(ops, plan.hid, rowpair, groups, tid, 64 * kWaves);
                __syncthreads();
            },
            ops, sums + wave * sums_floats<SETS, Q>(), blockIdx.x * kWaves + wave, gridDim.x * kWaves, units, groups, lane,
            [&](int u) __attribute__((always_inline)) {
                const int n0 = u * 4 * Q;
                const int64_t r0 = (int64_t)e * H + n0;
                return rows_of(D, DS, r0, r0 + 2 * Q, min(2 * Q, H - n0), min(2 * Q, H - n0 - 2 * Q), groups);
            },
            [&](int u, const float *sm) __attribute__((always_inline)) {
#pragma unroll
                for (int o0 = 0; o0 < ROWS * 4 * Q; o0 += 64) {
                    const int o = o0 + lane, nn = o % (4 * Q), i = min(o / (4 * Q), ROWS - 1), n = u * 4 * Q + nn;
                    const float y = sum_of_terms<AT, S>(sm, i, nn / 4, nn % 4);
                    const int pr = rowpair[i];
                    if (o < ROWS * 4 * Q && pr >= 0 && n < H) plan.part[(int64_t)pr * H + n] = y;
                }
            });
        base += ROWS;
    };
    while (base < count) {
        if (SETS > 1 && count - base <= rows_per_set(AT)) go(std::integral_constant<int, 1>());
        else go(std::integral_constant<int, SETS>());
    }
}

// y[t][n] = the sum of the token's parts, in the order of its choices, 4 values a thread.
__global__ __launch_bounds__(256) void moe_sum_kernel(Plan plan, void *__restrict__ Y, int y_dtype, int top_k, int H) {
    const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (n >= H) return;
    const float *part = plan.part + (int64_t)t * top_k * H + n;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < top_k; j += 4) {
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4 *>(part + (int64_t)min(j + i, top_k - 1) * H);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // a choice that there is not has nothing in its part
            if (j + i >= top_k || plan.ids[t * top_k + j + i] < 0) continue;
            y.x += v[i].x, y.y += v[i].y, y.z += v[i].z, y.w += v[i].w;
        }
    }
    const int64_t at = (int64_t)t * H + n;
    const float o[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (y_dtype == 2) store_out<2>(Y, at + i, o[i]);
        else if (y_dtype == 1) store_out<1>(Y, at + i, o[i]);
        else store_out<0>(Y, at + i, o[i]);
    }
}

// Few tokens: a workgroup goes through every taken expert for its rows of Y.  Its waves take the
// (expert, step) units in turn; the slots of the tiles are the tokens.  One that did not take the
// expert at hand has zeros there, and zeros in place of the expert's scales: they need not be finite.
template <int AT, int SETS, int Q>
__global__ __launch_bounds__(512) void moe_down_small_kernel(const uint8_t *__restrict__ D,
                                                            const uint16_t *__restrict__ DS, Plan plan,
                                                            void *__restrict__ Y, int y_dtype, int T, int E, int top_k,
                                                            int H, int F, int nw) {
    constexpr int R = rows_per_set(AT);
    static_assert(SETS * R <= kMoeSmall, "tokens");
    extern __shared__ float4 lds4[];
    float *red = reinterpret_cast<float *>(lds4);
    int *ids = reinterpret_cast<int *>(red + nw * sums_floats<SETS, Q>());
    uint32_t *bits = reinterpret_cast<uint32_t *>(ids + kMoeSmall * kMoeMaxTopK);
    int *experts = reinterpret_cast<int *>(bits + kMoeMaxExperts / 32);   // [P], then their number
    int *pair = experts + kMoeSmall * kMoeMaxTopK + 1;                    // [P][T]: token's pair of an expert, -1: none
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int P = T * top_k, words = (E + 31) / 32;
    for (int i = tid; i < P; i += 64 * nw) ids[i] = plan.ids[i];
    for (int i = tid; i < words; i += 64 * nw) bits[i] = 0;
    for (int i = tid; i < P * T; i += 64 * nw) pair[i] = -1;
    __syncthreads();
    if (wave == 0) {
        for (int i = lane; i < P; i += 64)
            if (ids[i] >= 0) atomicOr(&bits[ids[i] >> 5], 1u << (ids[i] & 31));
        wave_order();
        int n = 0;   // the set bits, in order
        for (int w0 = 0; w0 < words; w0 += 2) {
            const uint32_t word = w0 + (lane >> 5) < words ? bits[w0 + (lane >> 5)] : 0u;
            const bool set = (word >> (lane & 31)) & 1u;
            const uint64_t m = __ballot(set);
            if (set) experts[n + __popcll(m & ((1ull << lane) - 1))] = 32 * w0 + lane;
            n += __popcll(m);
        }
        if (lane == 0) experts[kMoeSmall * kMoeMaxTopK] = n;
        for (int i = lane; i < P; i += 64) {   // the expert's place: the set bits before its own
            const int e = ids[i];
            if (e < 0) continue;
            int at = __popc(bits[e >> 5] & ((1u << (e & 31)) - 1));
            for (int w = 0; w < e >> 5; ++w) at += __popc(bits[w]);
            pair[at * T + i / top_k] = i;
        }
    }
    __syncthreads();
    const int taken = uniform(experts[kMoeSmall * kMoeMaxTopK]);
    const int groups = F >> 7, n0 = blockIdx.x * 4 * Q, steps = (groups + 3) / 4, units = taken * steps;
    const int ca = (lane & 15) >> 2, slot = lane & 3, per_pair = (int)hid_words(F, AT) * 2;
    const __amdgpu_buffer_rsrc_t rx = buffer_of(plan.hid, P * per_pair);
    const int lane_at = slot / R * 1024 + (ca * 4 + (lane >> 4)) * 16;   // in a step's terms, 1 KB each

    uint4 a[SETS][4];
    uint64_t took[SETS];   // bit of a slot's lane: its token took the unit's expert
    Step<Q> st;
    Rows w;
    At at;
    // Unit u: its rows' place, and the loads of its activations.
    auto fetch = [&](int u) __attribute__((always_inline)) {
        const bool live = u < units;
        const int i = live ? u / steps : 0, s = live ? u - i * steps : 0, e = uniform(experts[i]);
#pragma unroll
        for (int t = 0; t < SETS; ++t) {
            const int tok = R * t + slot % R, pr = live && slot / R < AT && tok < T ? pair[i * T + min(tok, T - 1)] : -1;
            took[t] = __ballot(pr >= 0);
            const int off = pr >= 0 && 4 * s + ca < groups ? pr * per_pair + s * (AT * 1024) + lane_at : OUT_OF_RANGE;
#pragma unroll
            for (int k = 0; k < 4; ++k) a[t][k] = load16(rx, off + k * 256);
        }
        const int64_t r0 = (int64_t)e * H + n0;
        w = rows_of(D, DS, r0, r0 + 2 * Q, min(2 * Q, H - n0), min(2 * Q, H - n0 - 2 * Q), groups);
        at = place_of(s, groups, lane, live);
    };
    float4v_t acc[Q][SETS];
    clear<SETS, Q>(acc);
    int u = wave;
    if (u < units) {
        fetch(u);
#pragma unroll
        for (int q = 0; q < Q; ++q) load_quad<Q>(st, w, at, groups, q);
        for (;;) {
            uint4 now[SETS][4];
            uint64_t takers[SETS];
#pragma unroll
            for (int t = 0; t < SETS; ++t) {
                takers[t] = took[t];
#pragma unroll
                for (int k = 0; k < 4; ++k) now[t][k] = a[t][k];
            }
            fetch(u + nw);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                quad<AT, SETS>(st.code[q], st.scale[q], now, acc[q], [&](int t, int i) { return (takers[t] >> i & 1) != 0; });
                load_quad<Q>(st, w, at, groups, q);
                __builtin_amdgcn_sched_barrier(0);
            }
            u += nw;
            if (u >= units) break;
        }
    }
    store_sums<SETS, Q>(red + wave * sums_floats<SETS, Q>(), lane, acc);
    __syncthreads();
    for (int o = tid >> 2; o < T * 4 * Q; o += 16 * nw) {   // the 4 lanes of a DPP quad share an output
        const int nn = o % (4 * Q), i = o / (4 * Q);
        float y = 0.f;
        for (int w = tid & 3; w < nw; w += 4) {
            const float *sm = red + w * sums_floats<SETS, Q>();
            y += sum_of_terms<AT, SETS>(sm, i, nn / 4, nn % 4);
        }
        y += __builtin_bit_cast(float, dpp<0xB1>(__builtin_bit_cast(uint32_t, y)));
        y += __builtin_bit_cast(float, dpp<0x4E>(__builtin_bit_cast(uint32_t, y)));
        if ((tid & 3) != 0 || n0 + nn >= H) continue;
        const int64_t at = (int64_t)i * H + n0 + nn;
        if (y_dtype == 2) store_out<2>(Y, at, y);
        else if (y_dtype == 1) store_out<1>(Y, at, y);
        else store_out<0>(Y, at, y);
    }
}

// ---- launches -------------------------------------------------------------------

constexpr size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

Plan plan_of(void *ws, int64_t P, int64_t H, int64_t F) {
    char *w = static_cast<char *>(ws);
    auto take = [&](size_t n) {
        char *at = w;
        w += align256(n);
        return at;
    };
    Plan p;
    p.ids = reinterpret_cast<int *>(take((size_t)P * 4));
    p.weights = reinterpret_cast<float *>(take((size_t)P * 4));
    p.experts = reinterpret_cast<int *>(take((size_t)P * 4));
    p.start = reinterpret_cast<int *>(take((size_t)(P + 1) * 4));
    p.pairs = reinterpret_cast<int *>(take((size_t)P * 4));
    p.hid = reinterpret_cast<uint16_t *>(take((size_t)P * hid_words(F, 3) * 2));
    p.part = reinterpret_cast<float *>(w);
    return p;
}

// Workgroups for `slots` experts' `units`: about two a CU, each wave with as many units as the others.
int workgroups(int64_t units, int slots) {
    const int64_t most = std::max<int64_t>(1, 512 / slots), waves = std::min((units + kWaves - 1) / kWaves, most) * kWaves;
    const int64_t each = (units + waves - 1) / waves;
    return (int)(((units + each - 1) / each + kWaves - 1) / kWaves);
}

constexpr size_t kLds = 160 * 1024;

int hidden_terms(const MoeArgs &a) { return a.y_dtype == 2 ? 3 : 2; }

template <int AT, int SETS, int Q, int G, bool SMALL>
hipError_t launch_up(const MoeArgs &a, const Plan &plan, int slots) {
    const size_t lds = ops_bytes<SETS>((int)(a.H / 128)) + kWaves * sums_floats<SETS, Q>() * 4 +
                       SETS * rows_per_set(AT) * 16 + (SMALL ? kMoeSmall * kMoeMaxTopK * 8 + 4 + kMoeMaxExperts / 8 : 0);
    if constexpr (SETS > 1)
        if (lds > kLds) return launch_up<AT, SETS / 2, Q, G, SMALL>(a, plan, slots);
    const dim3 g((unsigned)workgroups((a.F + 2 * Q - 1) / (2 * Q), slots), (unsigned)slots), b(64 * kWaves);
    constexpr auto kern = &moe_up_kernel<AT, SETS, Q, G, SMALL>;
    const hipError_t e = raise_lds_limit<kern>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, g, b, lds, a.stream, static_cast<const char *>(a.X), a.logits, a.l_dtype, a.GU, a.GUS, plan,
                       (int)a.T, (int)a.E, (int)a.top_k, a.renormalize, (int)a.H, (int)a.F, hidden_terms(a));
    return hipGetLastError();
}

template <int AT, int SETS, int Q, int G>
hipError_t launch_down(const MoeArgs &a, const Plan &plan, int slots) {
    const size_t lds = ops_bytes<SETS>((int)(a.F / 128)) + kWaves * sums_floats<SETS, Q>() * 4 + SETS * rows_per_set(AT) * 4;
    if constexpr (SETS > 1)
        if (lds > kLds) return launch_down<AT, SETS / 2, Q, G>(a, plan, slots);
    const dim3 g((unsigned)workgroups((a.H + 4 * Q - 1) / (4 * Q), slots), (unsigned)slots), b(64 * kWaves);
    constexpr auto kern = &moe_down_kernel<AT, SETS, Q, G>;
    const hipError_t e = raise_lds_limit<kern>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, g, b, lds, a.stream, a.D, a.DS, plan, (int)a.H, (int)a.F);
    return hipGetLastError();
}

template <int AT, int SETS, int Q>
hipError_t launch_down_small(const MoeArgs &a, const Plan &plan) {
    const int64_t units = a.T * a.top_k * ((a.F + 511) / 512);   // at most
    const int nw = (int)(units < 8 ? units : 8);
    const dim3 g((unsigned)((a.H + 4 * Q - 1) / (4 * Q))), b(64 * nw);
    const size_t lds = (size_t)nw * sums_floats<SETS, Q>() * 4 + kMoeSmall * kMoeMaxTopK * 4 * (2 + kMoeSmall) +
                       kMoeMaxExperts / 8 + 4;
    constexpr auto kern = &moe_down_small_kernel<AT, SETS, Q>;
    const hipError_t e = raise_lds_limit<kern>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, g, b, lds, a.stream, a.D, a.DS, plan, a.Y, a.y_dtype, (int)a.T, (int)a.E, (int)a.top_k,
                       (int)a.H, (int)a.F, nw);
    return hipGetLastError();
}

// Rows of a workgroup of the small down kernel: one workgroup a CU where they allow it, else few
// rounds of them (four tokens, H = 5120: 16, 24, 32 rows 13.9, 9.4, 10.9 us; H = 2048: 16 rows 2 us
// more than 8).  Four sets leave registers for 16 rows.
template <int AT, int SETS>
hipError_t down_small(const MoeArgs &a, const Plan &plan) {
    constexpr int MOST = SETS > 2 ? 4 : 8;
    int best = 0, least = 0;
    for (int q = 2; q <= MOST; q += 2) {
        const int cost = (int)(((a.H + 4 * q - 1) / (4 * q) + 255) / 256) * (q + 1);
        if (best == 0 || cost < least) least = cost, best = q;
    }
    if (best == 2) return launch_down_small<AT, SETS, 2>(a, plan);
    if constexpr (MOST > 4) {
        if (best == 6) return launch_down_small<AT, SETS, 6>(a, plan);
        if (best == 8) return launch_down_small<AT, SETS, 8>(a, plan);
    }
    return launch_down_small<AT, SETS, 4>(a, plan);
}

// Steps of K that come in twos rather than in fours.  The up kernel takes them so, with twice the rows
// a wave, only if that leaves every SIMD two waves (one token, 2 experts of 5120 x 2048: 21.7 us for
// the layer with them, 18.6 without; four tokens, 8 experts: 32.8 and 34.8).
bool few_steps(int64_t K) { return (K + 511) / 512 % 4 == 1 || (K + 511) / 512 % 4 == 2; }

template <int SETS, bool SMALL>
hipError_t up(const MoeArgs &a, const Plan &plan, int slots) {
    if (few_steps(a.H) && a.F / 8 * slots >= 2048)
        return a.x_dtype == 0 ? launch_up<0, SETS, 4, 2, SMALL>(a, plan, slots) : launch_up<1, SETS, 4, 2, SMALL>(a, plan, slots);
    return a.x_dtype == 0 ? launch_up<0, SETS, 2, 4, SMALL>(a, plan, slots) : launch_up<1, SETS, 2, 4, SMALL>(a, plan, slots);
}

template <int AT>
hipError_t launch_chunk(const MoeArgs &a) {
    const int P = (int)(a.T * a.top_k);
    const Plan plan = plan_of(a.ws, P, a.H, a.F);
    const int slots = (int)(a.E < P ? a.E : P);
    hipError_t e;
    if (a.T <= kMoeSmall) {
        e = up<1, true>(a, plan, slots);
        if (e != hipSuccess) return e;
        constexpr int R = rows_per_set(AT);
        if (a.T <= R) return down_small<AT, 1>(a, plan);
        if constexpr (2 * R < kMoeSmall)
            if (a.T > 2 * R) return down_small<AT, 4>(a, plan);
        return down_small<AT, 2>(a, plan);
    }
    hipLaunchKernelGGL(moe_plan_kernel, dim3(1), dim3(1024), 0, a.stream, a.logits, a.l_dtype, (int)a.T, (int)a.E,
                       (int)a.top_k, a.renormalize, slots, plan);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    // A second set of slots once the experts have more than two tokens in the mean.
    e = P > 2 * slots ? up<2, false>(a, plan, slots) : up<1, false>(a, plan, slots);
    if (e != hipSuccess) return e;
    e = few_steps(a.F) ? launch_down<AT, 2, 4, 2>(a, plan, slots) : launch_down<AT, 2, 2, 4>(a, plan, slots);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_sum_kernel, dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.T), dim3(256), 0, a.stream, plan,
                       a.Y, a.y_dtype, (int)a.top_k, (int)a.H);
    return hipGetLastError();
}

}  // namespace

size_t moe_workspace(int64_t T, int64_t top_k, int64_t H, int64_t F) {
    const int64_t P = (T < kMoeChunk ? T : kMoeChunk) * top_k;
    return 4 * align256((size_t)P * 4) + align256((size_t)(P + 1) * 4) + align256((size_t)P * hid_words(F, 3) * 2) +
           align256((size_t)P * H * 4);
}

hipError_t launch_moe(const MoeArgs &a0) {
    MoeArgs a = a0;
    const int64_t lsize = a.l_dtype == 2 ? 4 : 2, ysize = a.y_dtype == 2 ? 4 : 2;
    for (int64_t t = 0; t < a0.T; t += kMoeChunk) {
        a.T = a0.T - t < kMoeChunk ? a0.T - t : kMoeChunk;
        a.X = static_cast<const char *>(a0.X) + t * a.H * 2;
        a.logits = static_cast<const char *>(a0.logits) + t * a.E * lsize;
        a.Y = static_cast<char *>(a0.Y) + t * a.H * ysize;
        const hipError_t e = hidden_terms(a) == 3 ? launch_chunk<3>(a) : launch_chunk<2>(a);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tern
