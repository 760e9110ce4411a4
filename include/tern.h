/*
 * tern.h -- C ABI of libtern.so, the ternary-weight matmul for AMD MI355X (gfx950).
 *
 * The operation (2kiu.com/news/5082861, "putting a ternary embedding model
 * into vLLM"):
 *   - weights W[N,K] take values in {-1, 0, +1}; each is a 2-bit code
 *     00 -> 0, 01 -> +1, 10 -> -1, 11 -> reserved, read as 0            (§3.1)
 *   - four codes per byte, little-endian: weight 4j+i of a row sits in
 *     bits 2i..2i+1 of byte j of that row; packed[N, K/4] uint8         (§2.2, §3.1)
 *   - every `group` = 128 consecutive weights of a row along K share one
 *     fp16 scale; scales[N, K/128]                                      (§1.1, §3.1)
 *   - Y[M,N] = X[M,K] . (T (*) S)^T, X fp16 or bf16, fp32 accumulation  (§4.2)
 *   - callers flatten activations to a contiguous 2-D [tokens, K]      (§4.4)
 *
 * Conventions shared by every entry point:
 *   - Every pointer is a DEVICE pointer the caller allocated and owns.  The
 *     library allocates no device memory, uses no scratch buffer but the
 *     workspace that a caller hands to it, and never frees or retains a
 *     caller buffer.  Its only state across calls is a
 *     per-process record, per device and kernel instantiation, that the
 *     kernel's dynamic-LDS limit has been raised (hipFuncSetAttribute, done
 *     once on first use); no call's result depends on an earlier call.
 *   - Every tensor is dense, row-major and contiguous.  Pointers to X, W, T
 *     and packed bytes must be 16-byte aligned (TERN_ERR_ALIGN otherwise);
 *     scales need 2-byte and Y its element alignment.
 *   - Calls are asynchronous on `stream` (NULL = the device's default
 *     stream) and never synchronize the host.
 *   - Arguments are validated before anything is launched.  A non-OK status
 *     means nothing was launched and no output byte was written, except
 *     TERN_ERR_HIP, which reports a failed launch.
 *   - Sizes of zero are valid: nothing is launched (tern_matmul with K = 0
 *     and M, N > 0 writes Y = 0, the empty sum).  A pointer may be NULL only
 *     when the buffer it stands for has zero elements.
 *   - The library never exits the process and never throws across the ABI.
 */
#ifndef TERN_H
#define TERN_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TERN_OK = 0,
    TERN_ERR_NULL = 1,        /* a required pointer is NULL */
    TERN_ERR_SHAPE = 2,       /* negative size, K % 4 != 0, or a size beyond the limits below */
    TERN_ERR_GROUP = 3,       /* K is not a multiple of `group`, or group <= 0 */
    TERN_ERR_DTYPE = 4,       /* x or y dtype outside the supported set */
    TERN_ERR_ALIGN = 5,       /* a pointer lacks the alignment stated above */
    TERN_ERR_UNSUPPORTED = 6, /* a valid request this build does not implement (group != 128, forced path that cannot run) */
    TERN_ERR_HIP = 7          /* the HIP runtime reported an error at launch */
} tern_status;

typedef enum { TERN_F16 = 0, TERN_BF16 = 1, TERN_F32 = 2 } tern_dtype;

/* Which kernel family computes tern_matmul_path's result. */
typedef enum {
    TERN_PATH_AUTO = 0, /* choose by shape (what tern_matmul does): for M <= 4, GEMV_FP4 with
                           bf16 X (K <= 32768), else with fp16 X GEMV_MFMA for M = 3, 4 where
                           it fits and GEMV for M <= 2 or where GEMV_MFMA does not fit;
                           GEMV_B16 for 5 <= M <= 16 with N >= 16384 and K <= 8192;
                           MFMA for every other shape */
    TERN_PATH_GEMV = 1, /* VALU sign-select decode kernel; M <= TERN_GEMV_MAX_M */
    TERN_PATH_MFMA = 2, /* LDS-staged activations + in-register weight decode + MFMA; any M */
    TERN_PATH_GEMV_MFMA = 3, /* decode kernel whose sign-select sums run on the matrix cores
                                (v_mfma_f32_4x4x4_16b on +-2 / 0 operands); M <= 4, with
                                the activations X[M,K] staged whole in LDS */
    TERN_PATH_GEMV_FP4 = 4, /* decode kernel with the weights as 4-bit (e2m1 +-2 / 0) matrix-core
                               operands and each bf16 activation split exactly into two e4m3
                               terms with a power-of-two scale per 32 (v_mfma_scale_f32_
                               16x16x128_f8f6f4); bf16 X only, M <= 4, K <= 32768, and no
                               more weight rows than a launch of fewer than 2^32
                               threads holds (6 * 10^7 of them are not too many) */
    TERN_PATH_GEMV_B16 = 5  /* decode kernel for batches of up to 16 rows: +-2 / 0 weight
                               operands of v_mfma_f32_16x16x32 against activation fragments
                               held in registers, waves splitting K; M <= 16, K <= 2^20 */
} tern_path;

#define TERN_GROUP 128
#define TERN_GEMV_MAX_M 4
#define TERN_MX_BLOCK 32
/* Size limits: M, N <= 2^31 - 1 and K <= 2^30; M*N, M*K and N*K <= 2^62. */

/* Human-readable name of a status code (a static string; never NULL). */
const char *tern_status_string(tern_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int tern_version(void);

/*
 * tern_pack -- T[N,K] int8 -> packed[N,K/4] uint8.
 * Source: 2kiu.com/news/5082861 §3.1 (code map, four codes per byte, first
 * weight in the lowest two bits).  T holds -1, 0 or +1; any other value is
 * written as the reserved code 11, which every reader decodes as 0.
 * Requires K % 4 == 0 (TERN_ERR_SHAPE).  T and packed: 16-byte aligned.
 */
tern_status tern_pack(const int8_t *T, uint8_t *packed, int64_t N, int64_t K, hipStream_t stream);

/*
 * tern_unpack -- packed[N,K/4] uint8 -> T[N,K] int8 in {-1, 0, +1}.
 * Source: 2kiu.com/news/5082861 §3.1 (the unpack function that recovers the
 * integer matrix from the packed bytes).  Code 11 is written as 0.
 * Requires K % 4 == 0.  Both pointers 16-byte aligned.
 */
tern_status tern_unpack(const uint8_t *packed, int8_t *T, int64_t N, int64_t K, hipStream_t stream);

/*
 * tern_matmul -- Y[M,N] = X[M,K] . (T (*) S)^T with fp32 accumulation.
 * Source: 2kiu.com/news/5082861 §4.2 (the kernel contract x[M,K], w[N,K/4],
 * scale[N,K/128], out[M,N]) with §3.1 for the weight encoding.
 *   X        [M,K]      x_dtype TERN_F16 or TERN_BF16
 *   packed_W [N,K/4]    uint8, the encoding of tern_pack
 *   scales   [N,K/128]  fp16 bit patterns (little-endian), one per 128
 *                       consecutive weights of a row
 *   Y        [M,N]      y_dtype TERN_F32, TERN_BF16 or TERN_F16; overwritten
 *                       (never accumulated into); fp32 results are rounded
 *                       to nearest-even into bf16/fp16, overflow gives inf
 *   group    must be 128 (TERN_ERR_UNSUPPORTED otherwise) and divide K
 * Result accuracy: |Y - exact| <= 2e-3 * sum_k |X[m,k] * S[n,k/128]| + one
 * ulp of y_dtype, for finite inputs (every finite fp16 scale).
 */
tern_status tern_matmul(const void *X, tern_dtype x_dtype, const uint8_t *packed_W,
                        const uint16_t *scales, void *Y, tern_dtype y_dtype, int64_t M, int64_t N,
                        int64_t K, int32_t group, hipStream_t stream);

/*
 * tern_matmul_path -- tern_matmul with an explicit kernel choice.  Same
 * arguments, layouts and result contract as tern_matmul; `path` picks the
 * kernel family (for tests that compare the two, and for benchmarks).
 * TERN_PATH_GEMV, TERN_PATH_GEMV_MFMA or TERN_PATH_GEMV_FP4 with M >
 * TERN_GEMV_MAX_M, or with an activation block too large for on-chip staging,
 * TERN_PATH_GEMV_FP4 with fp16 activations, and TERN_PATH_GEMV_B16 with M > 16
 * or K > 2^20, return TERN_ERR_UNSUPPORTED.
 */
tern_status tern_matmul_path(const void *X, tern_dtype x_dtype, const uint8_t *packed_W,
                             const uint16_t *scales, void *Y, tern_dtype y_dtype, int64_t M,
                             int64_t N, int64_t K, int32_t group, tern_path path,
                             hipStream_t stream);

/*
 * tern_dequant -- W[N,K] = t * s, the dense 16-bit weight matrix.
 * Source: 2kiu.com/news/5082861 §4.1 (the first route: dequantise, then a
 * library GEMM; the pages measure their kernel against it in §4.3).  This
 * is the comparison route's first half, not part of tern_matmul.
 *   packed [N,K/4] uint8, scales [N,K/group] fp16 bits, W [N,K] in w_dtype
 *   (TERN_F16: exact; TERN_BF16: s rounded to bf16, nearest even).
 *   group must be 128 and divide K.  packed and W 16-byte aligned.
 */
tern_status tern_dequant(const uint8_t *packed, const uint16_t *scales, void *W, tern_dtype w_dtype,
                         int64_t N, int64_t K, int32_t group, hipStream_t stream);

/*
 * tern_block_map -- which 128-weight blocks hold a nonzero weight.
 * Source: 2kiu.com/news/5082861 §6 (next steps: skip blocks that are
 * entirely zero).  block_map[n, w] (uint32, row-major [N, ceil(K/4096)]) has
 * bit b set when block 32w + b of row n contains a code 01 or 10; blocks of
 * codes 00 and 11 only are clear, and so are the unused high bits of a row's
 * last word.  packed 16-byte aligned, block_map 4-byte aligned; group must
 * be 128.  Computed once per weight matrix, not per product.
 */
tern_status tern_block_map(const uint8_t *packed, uint32_t *block_map, int64_t N, int64_t K, int32_t group,
                           hipStream_t stream);

/*
 * tern_matmul_blockmap -- tern_matmul that skips the unmarked blocks.
 * Source: 2kiu.com/news/5082861 §6 (zero-block skipping), §4.2 otherwise.
 * Same arguments, layouts, result contract and errors as tern_matmul, plus
 * block_map in the layout of tern_block_map (4-byte aligned; NULL only when
 * M, N or K is 0).  Blocks whose bit is clear are not read (no code bytes,
 * no scale) and not computed, so the map must mark every block with a
 * nonzero weight; marking more blocks is harmless.  The skipping kernel is
 * the decode path for M <= 2 (where the GEMV is the faster kernel); other
 * calls are tern_matmul (the map is not read).
 */
tern_status tern_matmul_blockmap(const void *X, tern_dtype x_dtype, const uint8_t *packed_W,
                                 const uint16_t *scales, const uint32_t *block_map, void *Y, tern_dtype y_dtype,
                                 int64_t M, int64_t N, int64_t K, int32_t group, hipStream_t stream);

/*
 * tern_quantize_scales -- int8 scale codes for tern_matmul_s8.
 * Source: 2kiu.com/news/5082861 §6 (next steps: compress the fp16 block
 * scale further to INT8).  The pages do not fix the scheme; this library's
 * reading is a symmetric code per output row with one fp32 factor:
 *   row_factor[n]  = max_g |S[n,g]| / 127            (fp32 division)
 *   scales_q[n,g]  = round-to-nearest-even(S[n,g] / row_factor[n]),
 *                    clamped to [-127, 127]; 0 for a row whose scales are 0
 * so the effective scale is scales_q[n,g] * row_factor[n] (relative error
 * up to 1/254 of the row's largest scale).  Both divisions are IEEE fp32.
 *   scales [N,K/group] fp16 bits (2-byte aligned), scales_q [N,K/group]
 *   int8, row_factor [N] fp32 (4-byte aligned).  group must be 128.
 */
tern_status tern_quantize_scales(const uint16_t *scales, int8_t *scales_q, float *row_factor, int64_t N,
                                 int64_t K, int32_t group, hipStream_t stream);

/*
 * tern_matmul_s8 -- tern_matmul_path with int8 block scales:
 *   Y[m,n] = sum_g (scales_q[n,g] * row_factor[n]) * sum_{k in g} t[n,k] X[m,k]
 * Source: 2kiu.com/news/5082861 §6 (INT8 scales, halving the scale traffic:
 * 1 byte per 128 weights instead of 2), with §4.2 for everything else.
 * Arguments, layouts, paths and errors as tern_matmul_path, with the fp16
 * scales replaced by scales_q [N,K/128] int8 and row_factor [N] fp32
 * (4-byte aligned; NULL only when M, N or K is 0).  Each path runs the
 * kernels of tern_matmul_path, reading the int8 codes in place of the fp16
 * scales.  Accuracy: the tern_matmul bound with
 * S[n,g] = scales_q[n,g] * row_factor[n].
 */
tern_status tern_matmul_s8(const void *X, tern_dtype x_dtype, const uint8_t *packed_W, const int8_t *scales_q,
                           const float *row_factor, void *Y, tern_dtype y_dtype, int64_t M, int64_t N,
                           int64_t K, int32_t group, tern_path path, hipStream_t stream);

/*
 * Microscaled 4-bit floats (the OCP MX format with e2m1 elements), for the
 * layers that a mixed-precision ternary model keeps at more than two bits.
 * A matrix [R,K], K % 32 == 0 (TERN_ERR_GROUP otherwise), is held as
 *   codes [R,K/2] uint8: two 4-bit codes a byte, the even element in the low
 *       nibble; a code is a sign bit and one of the magnitudes 0, 0.5, 1,
 *       1.5, 2, 3, 4, 6;
 *   exps [R,K/32] uint8: one per 32 consecutive elements of a row; the scale
 *       is 2^(exps - 127), and 255 makes the block NaN.
 * codes and the dense matrix: 16-byte aligned; exps: any alignment.
 */

/*
 * tern_mx_quantize -- X[M,K] (TERN_F16, TERN_BF16 or TERN_F32) -> codes, exps.
 * A block with the largest magnitude a gets the scale 2^E, E = max(floor(
 * log2 a) - 2, -127); each element is rounded to the nearest magnitude of
 * element / 2^E, ties to the even code, and to 6 if it lies above.  A zero
 * block gets the byte 0.  A block with an infinity or a NaN gets the byte 255
 * and zero codes, and reads back as NaN.
 */
tern_status tern_mx_quantize(const void *X, tern_dtype x_dtype, uint8_t *codes, uint8_t *exps, int64_t M, int64_t K,
                             hipStream_t stream);

/*
 * tern_mx_dequant -- codes, exps -> W[M,K] in w_dtype.  Exact in TERN_F32 and
 * TERN_BF16; in TERN_F16 rounded to nearest even where the value leaves the
 * type's range.
 */
tern_status tern_mx_dequant(const uint8_t *codes, const uint8_t *exps, void *W, tern_dtype w_dtype, int64_t M,
                            int64_t K, hipStream_t stream);

/*
 * tern_mx_matmul -- Y[M,N] = X[M,K] . W^T, W[N,K] held as codes and exps,
 * X in TERN_F16 or TERN_BF16, sums in fp32, Y in any of the three types,
 * rounded once (nearest even).  Any M, K <= 2^24.  X 16-byte aligned, Y to its
 * element.
 * The products are exact.  An infinity in X gives infinities, or NaN where its
 * weight is zero; a NaN gives NaN.  Either reaches its row of Y only, one in a
 * row of W (a block with exponent 255, or values beyond the fp32 range) that
 * column only.
 */
tern_status tern_mx_matmul(const void *X, tern_dtype x_dtype, const uint8_t *codes, const uint8_t *exps, void *Y,
                           tern_dtype y_dtype, int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * tern_mx_matmul_mx -- the same product with X[M,K] held as x_codes and
 * x_exps too (for instance from tern_mx_quantize).  K <= 2^24.
 */
tern_status tern_mx_matmul_mx(const uint8_t *x_codes, const uint8_t *x_exps, const uint8_t *codes,
                              const uint8_t *exps, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                              hipStream_t stream);

/*
 * tern_moe -- a mixture-of-experts layer with ternary experts, for the few
 * tokens of a decode step:
 *   y[t] = sum over e in S(t) of w[t,e] * Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t]))
 * S(t): the top_k experts by logit (ties to the lowest index; an expert whose
 * logit is -inf is never taken, so a token whose logits are all -inf, such as
 * padding, gets y = 0).  w: softmax of the logits, over S(t) if renormalize
 * is not 0, else over all experts.  A NaN counts as the largest logit; a row
 * with a NaN or +inf has NaN weights.
 *   X [T,H] TERN_F16 or TERN_BF16, logits [T,E] and Y [T,H] of any type
 *   gate_up [E,2F,H/4] tern_pack codes, rows 0..F-1 of an expert Wg and
 *       F..2F-1 Wu; gate_up_scales [E,2F,H/128] fp16
 *   down [E,H,F/4], down_scales [E,H,F/128]: Wd
 *   group must be 128 and divide H and F; 1 <= top_k <= min(E, 32) and
 *   E <= 1024 (TERN_ERR_UNSUPPORTED beyond those two limits); H, F <= 16384
 *   (TERN_ERR_SHAPE: the tokens of an expert stay in LDS).
 *   workspace: tern_moe_workspace bytes (TERN_ERR_SHAPE if fewer), 256-byte
 *       aligned, for this call alone until the stream has passed it.
 * All sums are fp32, and Y is rounded once.  A hidden value times its weight
 * w is fp32; where Y is TERN_F32 it enters the down product with all its bits,
 * where Y has 16 bits rounded to 2^-16 of itself, so that Y carries an error of
 * 2^-16 sum |w h Wd| beside its own rounding.  A 128-weight block's sum, before
 * its scale, has to stay below half the fp32 range.  Any T; tokens are
 * taken 64 at a time, each time reading the experts that they take.  The
 * result of a token does not depend on the other tokens of its call beyond
 * the order in which fp32 sums are formed, and repeated calls agree bit for
 * bit.
 */
size_t tern_moe_workspace(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t F);
tern_status tern_moe(const void *X, tern_dtype x_dtype, const void *logits, tern_dtype l_dtype,
                     const uint8_t *gate_up, const uint16_t *gate_up_scales, const uint8_t *down,
                     const uint16_t *down_scales, void *Y, tern_dtype y_dtype, int64_t T, int64_t E, int64_t top_k,
                     int64_t H, int64_t F, int32_t group, int32_t renormalize, void *workspace,
                     size_t workspace_bytes, hipStream_t stream);

/*
 * 8-bit activations.  A matrix [M,K] is held as
 *   codes [M,K] int8 and scales fp32, one per row ([M], q_group 0) or one per 128
 *   consecutive values of a row ([M,K/128], q_group 128, which must divide K:
 *   TERN_ERR_GROUP otherwise; any other q_group is TERN_ERR_UNSUPPORTED);
 *   the value is code * scale.
 * What is made here has a scale a / 127 for a row or block whose largest
 * magnitude is a, and codes 127 v / a rounded to nearest, ties to even, and cut
 * off at 127 (an a below 2^-126 is an fp32 of few bits, and may be less than |v|):
 * in [-127, 127], and always the same for the same values.  A block of zeros has
 * the scale 0.  One with an infinity or a NaN has the scale NaN and codes 0.
 */

/*
 * tern_rms_norm -- root-mean-square norm of the rows of X[M,K], with the
 * addition to a residual stream before it:
 *   h = X + residual, rounded to the stream's type and written to residual_out
 *       (without a residual h = X)
 *   Y = h / sqrt(mean of h^2 over the row + eps) * weight, formed in fp32 (three
 *       roundings, and what falls below 2^-126 on the way loses bits) and rounded
 *       to Y's type
 *   codes, scales: the same values as 8-bit activations.  The largest |h weight|
 *       of a row or block is taken as an fp32; beyond that range its scale is NaN.
 *   X, Y of any type; residual and residual_out in X's type or TERN_F32
 *       (TERN_ERR_DTYPE otherwise), both NULL for none; weight [K] of any type,
 *       NULL for ones.  Y or codes may be NULL, not both; scales goes with codes.
 *   residual_out may be the buffer of residual, or of X if the types are the
 *       same; other buffers do not overlap.
 *   K <= 65536 (TERN_ERR_SHAPE); eps >= 0 and finite (TERN_ERR_UNSUPPORTED).
 * Every pointer needs the alignment of its element only.  Squares are summed in
 * 64 bits.  A NaN or infinity reaches its own row only.
 */
tern_status tern_rms_norm(const void *X, tern_dtype x_dtype, const void *residual, tern_dtype r_dtype,
                          const void *weight, tern_dtype w_dtype, void *residual_out, void *Y, tern_dtype y_dtype,
                          int8_t *codes, float *scales, int32_t q_group, int64_t M, int64_t K, float eps,
                          hipStream_t stream);

/*
 * tern_q8_quantize -- codes and scales of X[M,K] of any type, with q_group 0 for
 * K <= 65536 (TERN_ERR_SHAPE).  tern_q8_dequant -- their values, products in fp32,
 * rounded to y_dtype.  Element alignment.
 */
tern_status tern_q8_quantize(const void *X, tern_dtype x_dtype, int8_t *codes, float *scales, int32_t q_group,
                             int64_t M, int64_t K, hipStream_t stream);
tern_status tern_q8_dequant(const int8_t *codes, const float *scales, int32_t q_group, void *Y, tern_dtype y_dtype,
                            int64_t M, int64_t K, hipStream_t stream);

/*
 * tern_matmul_q8 -- tern_matmul with 8-bit activations:
 *   Y[m,n] = sum over blocks g of 128 of x_scale[m,g] S[n,g] * sum over k in g of code[m,k] t[n,k]
 * The inner sums are exact integers; the rest is fp32, rounded once.  Any codes
 * from -128 to 127 and any scales.  packed_W, scales and group as tern_matmul;
 * x_codes 16-byte, x_scales 4-byte aligned; K <= 2^23, M and N <= 2^28, M N <=
 * 2^36.  A NaN or infinite scale reaches its own row or column of Y only.
 *   workspace: tern_matmul_q8_workspace bytes (TERN_ERR_SHAPE if fewer; for a large
 *       product some 1.5 K for each row of X, else none, never for 32 rows or
 *       fewer), 16-byte aligned, for this call alone until the stream has passed it.
 */
size_t tern_matmul_q8_workspace(int64_t M, int64_t N, int64_t K);
tern_status tern_matmul_q8(const int8_t *x_codes, const float *x_scales, int32_t q_group, const uint8_t *packed_W,
                           const uint16_t *scales, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                           int32_t group, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * tern_moe_route -- the experts of T tokens, and their weights, from a router's
 * logits [T,E] of any type:
 *   s = softmax of a token's logits, or sigmoid of each
 *   c = s + bias (fp32 [E]); with bias NULL s, experts in the order of their logits
 *   with groups > 1, groups of E / groups consecutive experts: only the experts of
 *       the keep_groups groups with the largest sums of their group_best (1 or 2)
 *       largest c are open.  An expert that is never taken does not count, so that
 *       a group may have a sum of one c; with group_best 1 and bias NULL, groups
 *       go by their largest logit, with 2 by sums of s
 *   ids [T,top_k] int32: the top_k open experts, largest c first
 *   weights [T,top_k] fp32: their s, divided by the sum of it over the taken ones
 *       if renormalize is not 0 (0 where that sum is 0), times scale
 * Ties go to the lowest index.  An expert whose logit or c is -inf is never taken:
 * where fewer than top_k can be, the rest of ids is -1 with weight 0.  A NaN c
 * counts as the largest; a softmax over a NaN or +inf has NaN weights.  c and the
 * weights are formed in 64 bits, and the weights rounded once.
 * groups divides E (TERN_ERR_GROUP); 1 <= keep_groups <= groups, group_best <= E /
 * groups, 1 <= top_k <= keep_groups * (E / groups) (TERN_ERR_SHAPE); E <= 1024,
 * top_k <= 32, groups <= 64 (TERN_ERR_UNSUPPORTED).  Element alignment.
 */
typedef enum { TERN_SCORE_SOFTMAX = 0, TERN_SCORE_SIGMOID = 1 } tern_score;
tern_status tern_moe_route(const void *logits, tern_dtype l_dtype, const float *bias, int32_t *ids, float *weights,
                           int64_t T, int64_t E, int64_t top_k, tern_score score, int64_t groups, int64_t keep_groups,
                           int32_t group_best, int32_t renormalize, float scale, hipStream_t stream);

/*
 * tern_moe_routed -- tern_moe with its experts and weights given, ids [T,top_k]
 * int32 and weights [T,top_k] fp32, as tern_moe_route leaves them:
 *   y[t] = sum over j of weights[t,j] * Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])), e = ids[t,j]
 * An id outside of [0, E) adds nothing; the same expert twice adds up.  Everything
 * else as tern_moe, the workspace too; top_k <= 32 may exceed E.
 */
tern_status tern_moe_routed(const void *X, tern_dtype x_dtype, const int32_t *ids, const float *weights,
                            const uint8_t *gate_up, const uint16_t *gate_up_scales, const uint8_t *down,
                            const uint16_t *down_scales, void *Y, tern_dtype y_dtype, int64_t T, int64_t E,
                            int64_t top_k, int64_t H, int64_t F, int32_t group, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);

/*
 * tern_stream_copy -- calibration, not part of the method: stream `bytes`
 * bytes of src with 16-byte loads (one instruction reads 1 KB of
 * consecutive bytes, every load of a thread issued before any is used) and,
 * when dst is not NULL, write them to dst.  With dst NULL it only reads.
 * It gives the plain-read (and copy) ceiling the decode kernels are timed
 * against, and a kernel of known traffic for scaling the HBM byte counters.
 * bytes % 16 == 0 and bytes <= 2^40 (TERN_ERR_SHAPE); src and dst 16-byte
 * aligned (TERN_ERR_ALIGN); src NULL with bytes > 0 is TERN_ERR_NULL;
 * bytes == 0 launches nothing.  Asynchronous on `stream`.
 */
tern_status tern_stream_copy(const void *src, void *dst, uint64_t bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TERN_H */
