// tern_api.hip -- the C ABI declared in include/tern.h: argument validation
// and kernel dispatch.  Validation never touches the GPU, so a rejected call
// launches nothing and writes nothing.
#include <hip/hip_runtime.h>

#include "../../include/tern.h"
#include "tern_kernels.h"
#include "tern_moe.h"
#include "tern_mx.h"
#include "tern_q8.h"
#include "tern_route.h"

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxK = int64_t(1) << 30;
// Products with microscaled weights: offsets inside the rows of one workgroup are 32-bit (72 rows
// of K / 2 bytes).
constexpr int64_t kMxMaxK = int64_t(1) << 24;
// Products with 8-bit activations: the same, 128 rows of K bytes; a grid has fewer than 2^32 threads,
// up to 8 for each row of W with few rows of X, and one for 32 outputs in tiles of 64 x 128 (the decode
// kernel of up to 4 rows has more of them a row, and leaves what is too much for a launch to these).
constexpr int64_t kQ8MaxK = int64_t(1) << 23, kQ8MaxDim = int64_t(1) << 28, kQ8MaxOut = int64_t(1) << 36;
constexpr int64_t kMaxProduct = int64_t(1) << 62;
constexpr size_t kGemvLdsLimit = 152 * 1024;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool product_ok(int64_t a, int64_t b) { return a == 0 || b <= kMaxProduct / a; }

tern_status check_pack_args(const void *T, const void *P, int64_t N, int64_t K) {
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxK || K % 4 != 0) return TERN_ERR_SHAPE;
    if (!product_ok(N, K)) return TERN_ERR_SHAPE;
    if (N == 0 || K == 0) return TERN_OK;
    if (T == nullptr || P == nullptr) return TERN_ERR_NULL;
    if (!aligned(T, 16) || !aligned(P, 16)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

size_t dtype_size(tern_dtype d) { return d == TERN_F32 ? 4 : 2; }

// S is the scale array (fp16 values, or int8 codes with s_align 1)
tern_status check_matmul_args(const void *X, tern_dtype x_dtype, const uint8_t *W, const void *S,
                              uintptr_t s_align, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                              int32_t group) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxK) return TERN_ERR_SHAPE;
    if (!product_ok(M, N) || !product_ok(M, K) || !product_ok(N, K)) return TERN_ERR_SHAPE;
    if (K % 4 != 0) return TERN_ERR_SHAPE;
    if (group <= 0 || K % group != 0) return TERN_ERR_GROUP;
    if (x_dtype != TERN_F16 && x_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (y_dtype != TERN_F16 && y_dtype != TERN_BF16 && y_dtype != TERN_F32) return TERN_ERR_DTYPE;
    if (group != TERN_GROUP) return TERN_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return TERN_OK;
    if (Y == nullptr) return TERN_ERR_NULL;
    if (!aligned(Y, dtype_size(y_dtype))) return TERN_ERR_ALIGN;
    if (K == 0) return TERN_OK;
    if (X == nullptr || W == nullptr || S == nullptr) return TERN_ERR_NULL;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(S, s_align)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

tern_status from_hip(hipError_t e) { return e == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

// Kernel arguments of a validated product: fp16 scales S, or int8 codes Q with
// row factors R (exactly one of the two is set).
tern::GemmArgs make_args(const void *X, tern_dtype x_dtype, const uint8_t *W, const uint16_t *S, const int8_t *Q,
                         const float *R, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                         hipStream_t stream) {
    tern::GemmArgs a;
    a.X = X;
    a.x_dtype = x_dtype == TERN_BF16 ? 1 : 0;
    a.W = W;
    a.S = S;
    a.Q = Q;
    a.R = R;
    a.Y = Y;
    a.y_dtype = y_dtype == TERN_F16 ? 0 : (y_dtype == TERN_BF16 ? 1 : 2);
    a.M = M;
    a.N = N;
    a.K = K;
    a.stream = stream;
    return a;
}

bool gemv_fits(int64_t M, int64_t K) {
    return M >= 1 && M <= TERN_GEMV_MAX_M && tern::gemv_lds_bytes(M, K) <= kGemvLdsLimit;
}

// The automatic choice: the VALU decode kernel for one or two activation
// rows; from three rows on, the MFMA kernel (16-row tiles: its time hardly
// changes up to M = 16) is faster.  Measured on the 5120 / 17408 decode
// shapes: M = 2 GEMV 4.6 / 12.5 / 13.6 us against MFMA 7.4 / 15.8 / 16.4;
// M = 3 GEMV 7.6 / 18.8 / 19.9 against MFMA 7.5 / 15.9 / 16.6.
constexpr int64_t kAutoGemvMaxM = 2;

// Up to M = 4 the decode kernel also wins where it takes its short-step form
// (N <= 5120, K <= 8192; bf16, graph-timed): 5120 -> 5120 at M = 3 / 4
// 5.3 / 6.1 us against MFMA 6.9 / 7.0, 5120 -> 1024 at M = 4 3.8 against
// 5.7, 6144 -> 5120 at M = 3 / 4 5.5 / 6.3 against 8.8 / 8.8.
bool auto_gemv(int64_t M, int64_t N, int64_t K) {
    return (M <= kAutoGemvMaxM && gemv_fits(M, K)) || tern::gemv_short(M, N, K);
}

// With bf16 activations the fp4 matrix-core decode kernel is the fastest of
// the decode kernels at every M <= 4 measured (graph-timed, weights rotated
// over 2 GB; M = 1: 5120 -> 5120 4.04 us against the VALU kernel's 4.16,
// 5120 -> 17408 7.34 against 8.28, 17408 -> 5120 8.51 against 9.08; M = 4:
// 5120 -> 17408 11.0 against 29.4 (VALU) and 13.4 (16-row MFMA tiles),
// 17408 -> 5120 12.7 against 23.9 and 15.9).  With fp16 activations the
// 4x4x4 matrix-core kernel takes M = 3, 4 (M = 4: 5120 -> 17408 11.3 us
// against 13.4, 5120 -> 5120 6.1 against the VALU kernel's 6.5).
//
// For 5 <= M <= 16 the 16-row decode kernel beats the MFMA tiles where
// there are many weight rows and K is not long (graph-timed, bf16, weights
// rotated over 2 GB; M = 16: 5120 -> 34816 23.0 us against 31.1, 8192 ->
// 28672 34.0 against 40.5, 5120 -> 17408 16.9 against 19.0; M = 8 / 5 at
// 5120 -> 17408 16.9 / 16.8 against 19.1 / 18.6).  With N <= 15360, or K =
// 17408 (17408 -> 5120: 19.7 against 18.8), the tiles are as fast or faster.
bool auto_b16(int64_t M, int64_t N, int64_t K) {
    return M >= 5 && M <= 16 && N >= 16384 && K <= 8192 && tern::gemv_b16_fits(M, N, K);
}

tern_path auto_path(const tern::GemmArgs &a) {
    if (a.M <= 4 && a.x_dtype == 1 && tern::gemv_fp4_fits(a.M, a.N, a.K, 1)) return TERN_PATH_GEMV_FP4;
    if (a.M >= 3 && a.M <= 4 && a.x_dtype == 0 && tern::gemv_mfma_fits(a.M, a.N, a.K)) return TERN_PATH_GEMV_MFMA;
    if (auto_b16(a.M, a.N, a.K)) return TERN_PATH_GEMV_B16;
    return auto_gemv(a.M, a.N, a.K) ? TERN_PATH_GEMV : TERN_PATH_MFMA;
}

// A forced path that cannot run this shape is TERN_ERR_UNSUPPORTED (checked
// before anything is launched).
tern_status check_path(tern_path path, tern_dtype x_dtype, int64_t M, int64_t N, int64_t K) {
    if (path != TERN_PATH_AUTO && path != TERN_PATH_GEMV && path != TERN_PATH_MFMA && path != TERN_PATH_GEMV_MFMA &&
        path != TERN_PATH_GEMV_FP4 && path != TERN_PATH_GEMV_B16)
        return TERN_ERR_UNSUPPORTED;
    if (M == 0 || N == 0 || K == 0) return TERN_OK;
    if (path == TERN_PATH_GEMV && !gemv_fits(M, K)) return TERN_ERR_UNSUPPORTED;
    if (path == TERN_PATH_GEMV_MFMA && !tern::gemv_mfma_fits(M, N, K)) return TERN_ERR_UNSUPPORTED;
    if (path == TERN_PATH_GEMV_FP4 && !tern::gemv_fp4_fits(M, N, K, x_dtype == TERN_BF16 ? 1 : 0))
        return TERN_ERR_UNSUPPORTED;
    if (path == TERN_PATH_GEMV_B16 && !tern::gemv_b16_fits(M, N, K)) return TERN_ERR_UNSUPPORTED;
    return TERN_OK;
}

hipError_t dispatch(const tern::GemmArgs &a, tern_path path) {
    switch (path) {
    case TERN_PATH_GEMV: return tern::launch_gemv(a);
    case TERN_PATH_MFMA: return tern::launch_gemm(a);
    case TERN_PATH_GEMV_MFMA: return tern::launch_gemv_mfma(a);
    case TERN_PATH_GEMV_FP4: return tern::launch_gemv_fp4(a);
    case TERN_PATH_GEMV_B16: return tern::launch_gemv_b16(a);
    default: {
        const tern_path p = auto_path(a);
        return p == TERN_PATH_AUTO ? hipErrorInvalidValue : dispatch(a, p);
    }
    }
}

int dtype_index(tern_dtype d) { return d == TERN_F16 ? 0 : (d == TERN_BF16 ? 1 : 2); }

bool known_dtype(tern_dtype d) { return d == TERN_F16 || d == TERN_BF16 || d == TERN_F32; }

// A microscaled matrix [rows, K] and, beside it, the dense one it comes from or goes to.
tern_status check_mx_args(const void *codes, const void *exps, const void *dense, tern_dtype dtype, int64_t rows,
                          int64_t K) {
    if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxK || !product_ok(rows, K)) return TERN_ERR_SHAPE;
    if (K % TERN_MX_BLOCK != 0) return TERN_ERR_GROUP;
    if (!known_dtype(dtype)) return TERN_ERR_DTYPE;
    if (rows == 0 || K == 0) return TERN_OK;
    if (codes == nullptr || exps == nullptr || dense == nullptr) return TERN_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(dense, 16)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

// Both products: XE is null where X holds 16-bit values.
tern_status check_mx_product(const void *X, const void *XE, bool mx, const void *W, const void *WE, const void *Y,
                             tern_dtype y_dtype, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMxMaxK) return TERN_ERR_SHAPE;
    if (!product_ok(M, N) || !product_ok(M, K) || !product_ok(N, K)) return TERN_ERR_SHAPE;
    if (K % TERN_MX_BLOCK != 0) return TERN_ERR_GROUP;
    if (!known_dtype(y_dtype)) return TERN_ERR_DTYPE;
    if (M == 0 || N == 0) return TERN_OK;
    if (Y == nullptr) return TERN_ERR_NULL;
    if (!aligned(Y, dtype_size(y_dtype))) return TERN_ERR_ALIGN;
    if (K == 0) return TERN_OK;
    if (X == nullptr || W == nullptr || WE == nullptr || (mx && XE == nullptr)) return TERN_ERR_NULL;
    if (!aligned(X, 16) || !aligned(W, 16)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

tern_status mx_product(const void *X, const uint8_t *XE, int x_dtype, const uint8_t *W, const uint8_t *WE, void *Y,
                       tern_dtype y_dtype, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
    const tern_status st = check_mx_product(X, XE, x_dtype == 2, W, WE, Y, y_dtype, M, N, K);
    if (st != TERN_OK || M == 0 || N == 0) return st;
    if (K == 0) return from_hip(tern::launch_fill_zero(Y, M * N * (int64_t)dtype_size(y_dtype), stream));
    tern::MxArgs a;
    a.X = X;
    a.XE = XE;
    a.x_dtype = x_dtype;
    a.W = W;
    a.WE = WE;
    a.Y = Y;
    a.y_dtype = dtype_index(y_dtype);
    a.M = M;
    a.N = N;
    a.K = K;
    a.stream = stream;
    return from_hip(tern::mx_gemm_wins(a) ? tern::launch_mx_gemm(a) : tern::launch_mx_gemv(a));
}

// 8-bit activations [M,K]: their sizes and q_group; then their pointers, where there are any.
tern_status check_q8_sizes(int32_t q_group, int64_t M, int64_t K) {
    if (M < 0 || K < 0 || M > kMaxDim || K > kMaxK || !product_ok(M, K)) return TERN_ERR_SHAPE;
    if (q_group != 0 && q_group != TERN_GROUP) return TERN_ERR_UNSUPPORTED;
    if (q_group != 0 && K % q_group != 0) return TERN_ERR_GROUP;
    return TERN_OK;
}

tern_status check_q8_pointers(const int8_t *codes, const float *scales) {
    if (codes == nullptr || scales == nullptr) return TERN_ERR_NULL;
    return aligned(scales, 4) ? TERN_OK : TERN_ERR_ALIGN;
}

bool q8_product_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && N >= 0 && K >= 0 && M <= kQ8MaxDim && N <= kQ8MaxDim && K <= kQ8MaxK && M * N <= kQ8MaxOut;
}

// Which kernel takes a product with 8-bit activations: the decode kernel of up to 4 rows; the one for
// few rows, always up to 32 where it reads the weights once; beyond that the one of three with the
// shortest time by their own estimates.  Measured, in us, few rows / tiles of 64 x 128 / of 128 x 384
// (estimates in brackets), N x K: 5120 x 5120, 128 rows 15.5 / 27.6 / 62.1 (16 / 28 / 68), 512 rows
// 51.7 / 39.6 / 65.3 (57 / 41 / 68); 17408 x 5120, 64 rows 36.9 / 28.2 / 66.7 (30 / 28 / 68), 512 rows
// 182 / 86.9 / 70.7 (195 / 81 / 68); 5120 x 17408, 128 rows 40.9 / 82.1 / 180 (49 / 86 / 188);
// 1024 x 1024, 1024 rows 7.9 / 9.4 / 25.7 (7 / 8 / 28), 4096 rows 25.6 / 14.3 / 30.5 (20 / 11 / 28).
enum class Q8Kernel { Decode, Rows, Blocks, Tiles };
Q8Kernel q8_kernel(int64_t M, int64_t N, int64_t K) {
    if (M <= TERN_GEMV_MAX_M && tern::gemv_fp4_fits(M, N, K, 3)) return Q8Kernel::Decode;
    const bool rows = tern::q8_rows_fits(M, N, K);
    if (rows && M <= 32) return Q8Kernel::Rows;
    if (M <= 32) return Q8Kernel::Blocks;   // no workspace for so few
    const double blocks = tern::q8_blocks_time(M, N, K), tiles = tern::q8_gemm_time(M, N, K);
    if (rows && tern::q8_rows_time(M, N, K) < (blocks < tiles ? blocks : tiles)) return Q8Kernel::Rows;
    return blocks < tiles ? Q8Kernel::Blocks : Q8Kernel::Tiles;
}
size_t q8_workspace(int64_t M, int64_t N, int64_t K) {
    return q8_kernel(M, N, K) == Q8Kernel::Tiles ? tern::q8_gemm_workspace(M, N, K) : 0;
}

bool moe_sizes_ok(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t F) {
    if (T < 0 || E < 0 || top_k < 0 || H < 0 || F < 0) return false;
    if (T > kMaxDim || E > kMaxDim || top_k > kMaxDim || H > tern::kMoeMaxWidth || F > tern::kMoeMaxWidth)
        return false;
    return product_ok(2 * E, H * F) && product_ok(T, H) && product_ok(T, E);   // weights, values, logits
}

// tern_moe and, with ids and weights in place of the logits, tern_moe_routed.
tern_status moe(const void *X, tern_dtype x_dtype, const void *logits, tern_dtype l_dtype, const int32_t *ids,
                const float *weights, bool routed, const uint8_t *gate_up, const uint16_t *gate_up_scales,
                const uint8_t *down, const uint16_t *down_scales, void *Y, tern_dtype y_dtype, int64_t T, int64_t E,
                int64_t top_k, int64_t H, int64_t F, int32_t group, int32_t renormalize, void *workspace,
                size_t workspace_bytes, hipStream_t stream) {
    if (!moe_sizes_ok(T, E, top_k, H, F) || top_k < 1 || (routed ? E < 1 : top_k > E))
        return TERN_ERR_SHAPE;
    if (group <= 0 || H % group != 0 || F % group != 0) return TERN_ERR_GROUP;
    if (x_dtype != TERN_F16 && x_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (!known_dtype(l_dtype) || !known_dtype(y_dtype)) return TERN_ERR_DTYPE;
    if (group != TERN_GROUP || E > tern::kMoeMaxExperts || top_k > tern::kMoeMaxTopK) return TERN_ERR_UNSUPPORTED;
    if (T == 0 || H == 0) return TERN_OK;
    if (Y == nullptr) return TERN_ERR_NULL;
    if (!aligned(Y, dtype_size(y_dtype))) return TERN_ERR_ALIGN;
    if (F == 0) return from_hip(tern::launch_fill_zero(Y, T * H * (int64_t)dtype_size(y_dtype), stream));
    if (routed ? ids == nullptr || weights == nullptr : logits == nullptr) return TERN_ERR_NULL;
    if (X == nullptr || gate_up == nullptr || gate_up_scales == nullptr || down == nullptr || down_scales == nullptr ||
        workspace == nullptr)
        return TERN_ERR_NULL;
    if (!aligned(logits, dtype_size(l_dtype)) || !aligned(ids, 4) || !aligned(weights, 4)) return TERN_ERR_ALIGN;
    if (!aligned(X, 16) || !aligned(gate_up, 16) || !aligned(down, 16) || !aligned(gate_up_scales, 2) ||
        !aligned(down_scales, 2) || !aligned(workspace, 256))
        return TERN_ERR_ALIGN;
    if (workspace_bytes < tern::moe_workspace(T, top_k, H, F)) return TERN_ERR_SHAPE;
    tern::MoeArgs a;
    a.X = X;
    a.x_dtype = dtype_index(x_dtype);
    a.logits = logits;
    a.l_dtype = dtype_index(l_dtype);
    a.ids = ids;
    a.weights = weights;
    a.GU = gate_up;
    a.GUS = gate_up_scales;
    a.D = down;
    a.DS = down_scales;
    a.Y = Y;
    a.y_dtype = dtype_index(y_dtype);
    a.T = T;
    a.E = E;
    a.top_k = top_k;
    a.H = H;
    a.F = F;
    a.renormalize = renormalize;
    a.ws = workspace;
    a.stream = stream;
    return from_hip(tern::launch_moe(a));
}

}  // namespace

extern "C" {

const char *tern_status_string(tern_status status) {
    switch (status) {
    case TERN_OK: return "TERN_OK";
    case TERN_ERR_NULL: return "TERN_ERR_NULL: a required pointer is NULL";
    case TERN_ERR_SHAPE: return "TERN_ERR_SHAPE: invalid size (negative, K % 4 != 0, or beyond limits)";
    case TERN_ERR_GROUP: return "TERN_ERR_GROUP: K is not a multiple of group, or group <= 0";
    case TERN_ERR_DTYPE: return "TERN_ERR_DTYPE: unsupported x or y dtype";
    case TERN_ERR_ALIGN: return "TERN_ERR_ALIGN: pointer misaligned";
    case TERN_ERR_UNSUPPORTED: return "TERN_ERR_UNSUPPORTED: request not implemented by this build";
    case TERN_ERR_HIP: return "TERN_ERR_HIP: HIP launch error";
    }
    return "TERN_ERR_UNKNOWN: not a tern_status value";
}

int tern_version(void) { return 100; }

tern_status tern_pack(const int8_t *T, uint8_t *packed, int64_t N, int64_t K, hipStream_t stream) {
    const tern_status st = check_pack_args(T, packed, N, K);
    if (st != TERN_OK || N == 0 || K == 0) return st;
    return from_hip(tern::launch_pack(T, packed, N * (K / 4), stream));
}

tern_status tern_unpack(const uint8_t *packed, int8_t *T, int64_t N, int64_t K, hipStream_t stream) {
    const tern_status st = check_pack_args(T, packed, N, K);
    if (st != TERN_OK || N == 0 || K == 0) return st;
    return from_hip(tern::launch_unpack(packed, T, N * (K / 4), stream));
}

tern_status tern_matmul_path(const void *X, tern_dtype x_dtype, const uint8_t *packed_W,
                             const uint16_t *scales, void *Y, tern_dtype y_dtype, int64_t M,
                             int64_t N, int64_t K, int32_t group, tern_path path,
                             hipStream_t stream) {
    const tern_status st = check_matmul_args(X, x_dtype, packed_W, scales, 2, Y, y_dtype, M, N, K, group);
    if (st != TERN_OK) return st;
    const tern_status pst = check_path(path, x_dtype, M, N, K);
    if (pst != TERN_OK) return pst;
    if (M == 0 || N == 0) return TERN_OK;
    if (K == 0) return from_hip(tern::launch_fill_zero(Y, M * N * (int64_t)dtype_size(y_dtype), stream));

    const tern::GemmArgs a = make_args(X, x_dtype, packed_W, scales, nullptr, nullptr, Y, y_dtype, M, N, K, stream);
    return from_hip(dispatch(a, path));
}

tern_status tern_matmul(const void *X, tern_dtype x_dtype, const uint8_t *packed_W, const uint16_t *scales,
                        void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K, int32_t group,
                        hipStream_t stream) {
    return tern_matmul_path(X, x_dtype, packed_W, scales, Y, y_dtype, M, N, K, group, TERN_PATH_AUTO,
                            stream);
}

tern_status tern_quantize_scales(const uint16_t *scales, int8_t *scales_q, float *row_factor, int64_t N,
                                 int64_t K, int32_t group, hipStream_t stream) {
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxK || !product_ok(N, K) || K % 4 != 0) return TERN_ERR_SHAPE;
    if (group <= 0 || K % group != 0) return TERN_ERR_GROUP;
    if (group != TERN_GROUP) return TERN_ERR_UNSUPPORTED;
    if (N == 0) return TERN_OK;
    if (row_factor == nullptr) return TERN_ERR_NULL;
    if (K > 0 && (scales == nullptr || scales_q == nullptr)) return TERN_ERR_NULL;
    if (!aligned(scales, 2) || !aligned(row_factor, 4)) return TERN_ERR_ALIGN;
    return from_hip(tern::launch_quantize_scales(scales, scales_q, row_factor, N, K / group, stream));
}

tern_status tern_matmul_s8(const void *X, tern_dtype x_dtype, const uint8_t *packed_W, const int8_t *scales_q,
                           const float *row_factor, void *Y, tern_dtype y_dtype, int64_t M, int64_t N,
                           int64_t K, int32_t group, tern_path path, hipStream_t stream) {
    const tern_status st = check_matmul_args(X, x_dtype, packed_W, scales_q, 1, Y, y_dtype, M, N, K, group);
    if (st != TERN_OK) return st;
    if (M > 0 && N > 0 && K > 0 && row_factor == nullptr) return TERN_ERR_NULL;
    if (!aligned(row_factor, 4)) return TERN_ERR_ALIGN;
    const tern_status pst = check_path(path, x_dtype, M, N, K);
    if (pst != TERN_OK) return pst;
    if (M == 0 || N == 0) return TERN_OK;
    if (K == 0) return from_hip(tern::launch_fill_zero(Y, M * N * (int64_t)dtype_size(y_dtype), stream));

    const tern::GemmArgs a =
        make_args(X, x_dtype, packed_W, nullptr, scales_q, row_factor, Y, y_dtype, M, N, K, stream);
    return from_hip(dispatch(a, path));
}

tern_status tern_block_map(const uint8_t *packed, uint32_t *block_map, int64_t N, int64_t K, int32_t group,
                           hipStream_t stream) {
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxK || !product_ok(N, K) || K % 4 != 0) return TERN_ERR_SHAPE;
    if (group <= 0 || K % group != 0) return TERN_ERR_GROUP;
    if (group != TERN_GROUP) return TERN_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return TERN_OK;
    if (packed == nullptr || block_map == nullptr) return TERN_ERR_NULL;
    if (!aligned(packed, 16) || !aligned(block_map, 4)) return TERN_ERR_ALIGN;
    return from_hip(tern::launch_block_map(packed, block_map, N, K, stream));
}

tern_status tern_matmul_blockmap(const void *X, tern_dtype x_dtype, const uint8_t *packed_W,
                                 const uint16_t *scales, const uint32_t *block_map, void *Y, tern_dtype y_dtype,
                                 int64_t M, int64_t N, int64_t K, int32_t group, hipStream_t stream) {
    const tern_status st = check_matmul_args(X, x_dtype, packed_W, scales, 2, Y, y_dtype, M, N, K, group);
    if (st != TERN_OK) return st;
    if (M > 0 && N > 0 && K > 0 && block_map == nullptr) return TERN_ERR_NULL;
    if (!aligned(block_map, 4)) return TERN_ERR_ALIGN;
    const bool skip = M >= 1 && M <= kAutoGemvMaxM && K > 0 && tern::gemv_skip_lds_bytes(M, K) <= kGemvLdsLimit;
    if (!skip) return tern_matmul_path(X, x_dtype, packed_W, scales, Y, y_dtype, M, N, K, group, TERN_PATH_AUTO,
                                       stream);
    if (N == 0) return TERN_OK;

    const tern::GemmArgs a = make_args(X, x_dtype, packed_W, scales, nullptr, nullptr, Y, y_dtype, M, N, K, stream);
    return from_hip(tern::launch_gemv_skip(a, block_map));
}

tern_status tern_dequant(const uint8_t *packed, const uint16_t *scales, void *W, tern_dtype w_dtype,
                         int64_t N, int64_t K, int32_t group, hipStream_t stream) {
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxK || !product_ok(N, K) || K % 4 != 0) return TERN_ERR_SHAPE;
    if (group <= 0 || K % group != 0) return TERN_ERR_GROUP;
    if (w_dtype != TERN_F16 && w_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (group != TERN_GROUP) return TERN_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return TERN_OK;
    if (packed == nullptr || scales == nullptr || W == nullptr) return TERN_ERR_NULL;
    if (!aligned(packed, 16) || !aligned(W, 16) || !aligned(scales, 2)) return TERN_ERR_ALIGN;
    return from_hip(tern::launch_dequant(packed, scales, W, w_dtype == TERN_BF16 ? 1 : 0, N, K, stream));
}

tern_status tern_mx_quantize(const void *X, tern_dtype x_dtype, uint8_t *codes, uint8_t *exps, int64_t M, int64_t K,
                             hipStream_t stream) {
    const tern_status st = check_mx_args(codes, exps, X, x_dtype, M, K);
    if (st != TERN_OK || M == 0 || K == 0) return st;
    return from_hip(tern::launch_mx_quantize(X, dtype_index(x_dtype), codes, exps, M * (K / TERN_MX_BLOCK), stream));
}

tern_status tern_mx_dequant(const uint8_t *codes, const uint8_t *exps, void *W, tern_dtype w_dtype, int64_t M,
                            int64_t K, hipStream_t stream) {
    const tern_status st = check_mx_args(codes, exps, W, w_dtype, M, K);
    if (st != TERN_OK || M == 0 || K == 0) return st;
    return from_hip(tern::launch_mx_dequant(codes, exps, W, dtype_index(w_dtype), M * (K / TERN_MX_BLOCK), stream));
}

tern_status tern_mx_matmul(const void *X, tern_dtype x_dtype, const uint8_t *codes, const uint8_t *exps, void *Y,
                           tern_dtype y_dtype, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
    if (x_dtype != TERN_F16 && x_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    return mx_product(X, nullptr, dtype_index(x_dtype), codes, exps, Y, y_dtype, M, N, K, stream);
}

tern_status tern_mx_matmul_mx(const uint8_t *x_codes, const uint8_t *x_exps, const uint8_t *codes,
                              const uint8_t *exps, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                              hipStream_t stream) {
    return mx_product(x_codes, x_exps, 2, codes, exps, Y, y_dtype, M, N, K, stream);
}

size_t tern_moe_workspace(int64_t T, int64_t E, int64_t top_k, int64_t H, int64_t F) {
    if (!moe_sizes_ok(T, E, top_k, H, F) || T == 0 || H == 0 || F == 0 || top_k > tern::kMoeMaxTopK) return 0;
    return tern::moe_workspace(T, top_k, H, F);
}

tern_status tern_moe(const void *X, tern_dtype x_dtype, const void *logits, tern_dtype l_dtype,
                     const uint8_t *gate_up, const uint16_t *gate_up_scales, const uint8_t *down,
                     const uint16_t *down_scales, void *Y, tern_dtype y_dtype, int64_t T, int64_t E, int64_t top_k,
                     int64_t H, int64_t F, int32_t group, int32_t renormalize, void *workspace,
                     size_t workspace_bytes, hipStream_t stream) {
    return moe(X, x_dtype, logits, l_dtype, nullptr, nullptr, false, gate_up, gate_up_scales, down, down_scales, Y,
               y_dtype, T, E, top_k, H, F, group, renormalize, workspace, workspace_bytes, stream);
}

tern_status tern_moe_routed(const void *X, tern_dtype x_dtype, const int32_t *ids, const float *weights,
                            const uint8_t *gate_up, const uint16_t *gate_up_scales, const uint8_t *down,
                            const uint16_t *down_scales, void *Y, tern_dtype y_dtype, int64_t T, int64_t E,
                            int64_t top_k, int64_t H, int64_t F, int32_t group, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    return moe(X, x_dtype, nullptr, TERN_F32, ids, weights, true, gate_up, gate_up_scales, down, down_scales, Y, y_dtype,
               T, E, top_k, H, F, group, 0, workspace, workspace_bytes, stream);
}

tern_status tern_moe_route(const void *logits, tern_dtype l_dtype, const float *bias, int32_t *ids, float *weights,
                           int64_t T, int64_t E, int64_t top_k, tern_score score, int64_t groups, int64_t keep_groups,
                           int32_t group_best, int32_t renormalize, float scale, hipStream_t stream) {
    if (T < 0 || E < 1 || T > kMaxDim || E > kMaxDim || !product_ok(T, E)) return TERN_ERR_SHAPE;
    if (groups < 1 || E % groups != 0) return TERN_ERR_GROUP;
    if (keep_groups < 1 || keep_groups > groups || group_best < 1 || group_best > 2) return TERN_ERR_SHAPE;
    if ((groups > 1 && group_best > E / groups) || top_k < 1 || top_k > keep_groups * (E / groups)) return TERN_ERR_SHAPE;
    if (!known_dtype(l_dtype)) return TERN_ERR_DTYPE;
    if (score != TERN_SCORE_SOFTMAX && score != TERN_SCORE_SIGMOID) return TERN_ERR_UNSUPPORTED;
    if (E > tern::kRouteMaxExperts || top_k > tern::kRouteMaxTopK || groups > tern::kRouteMaxGroups)
        return TERN_ERR_UNSUPPORTED;
    if (T == 0) return TERN_OK;
    if (logits == nullptr || ids == nullptr || weights == nullptr) return TERN_ERR_NULL;
    if (!aligned(logits, dtype_size(l_dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return TERN_ERR_ALIGN;
    tern::RouteArgs a;
    a.logits = logits;
    a.l_dtype = dtype_index(l_dtype);
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.E = (int)E;
    a.top_k = (int)top_k;
    a.sigmoid = score == TERN_SCORE_SIGMOID;
    a.groups = (int)groups;
    a.keep = (int)keep_groups;
    a.best = group_best;
    a.renormalize = renormalize;
    a.scale = scale;
    a.stream = stream;
    return from_hip(tern::launch_route(a));
}

tern_status tern_rms_norm(const void *X, tern_dtype x_dtype, const void *residual, tern_dtype r_dtype,
                          const void *weight, tern_dtype w_dtype, void *residual_out, void *Y, tern_dtype y_dtype,
                          int8_t *codes, float *scales, int32_t q_group, int64_t M, int64_t K, float eps,
                          hipStream_t stream) {
    const bool coded = codes != nullptr || scales != nullptr, added = residual != nullptr || residual_out != nullptr;
    tern_status st = check_q8_sizes(coded ? q_group : 0, M, K);
    if (st != TERN_OK) return st;
    if (K > tern::kNormMaxK) return TERN_ERR_SHAPE;
    if (!known_dtype(x_dtype) || (added && r_dtype != x_dtype && r_dtype != TERN_F32)) return TERN_ERR_DTYPE;
    if ((weight != nullptr && !known_dtype(w_dtype)) || (Y != nullptr && !known_dtype(y_dtype))) return TERN_ERR_DTYPE;
    if (!(eps >= 0.f && eps <= 3.402823466e38f)) return TERN_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return TERN_OK;
    if (X == nullptr || (Y == nullptr && !coded)) return TERN_ERR_NULL;
    if (added && (residual == nullptr || residual_out == nullptr)) return TERN_ERR_NULL;
    if (coded && (st = check_q8_pointers(codes, scales)) != TERN_OK) return st;
    if (!aligned(X, dtype_size(x_dtype)) || (Y != nullptr && !aligned(Y, dtype_size(y_dtype))) ||
        (weight != nullptr && !aligned(weight, dtype_size(w_dtype))) ||
        (added && (!aligned(residual, dtype_size(r_dtype)) || !aligned(residual_out, dtype_size(r_dtype)))))
        return TERN_ERR_ALIGN;
    tern::NormArgs a{};
    a.X = X;
    a.x_dtype = dtype_index(x_dtype);
    a.R = residual;
    a.r_dtype = added ? dtype_index(r_dtype) : 0;
    a.W = weight;
    a.w_dtype = weight != nullptr ? dtype_index(w_dtype) : 0;
    a.H = residual_out;
    a.Y = Y;
    a.y_dtype = Y != nullptr ? dtype_index(y_dtype) : 0;
    a.Q = codes;
    a.S = scales;
    a.grouped = coded && q_group != 0;
    a.normalize = 1;
    a.M = M;
    a.K = K;
    a.eps = eps;
    a.stream = stream;
    return from_hip(tern::launch_norm(a));
}

tern_status tern_q8_quantize(const void *X, tern_dtype x_dtype, int8_t *codes, float *scales, int32_t q_group,
                             int64_t M, int64_t K, hipStream_t stream) {
    tern_status st = check_q8_sizes(q_group, M, K);
    if (st != TERN_OK) return st;
    if (q_group == 0 && K > tern::kNormMaxK) return TERN_ERR_SHAPE;
    if (!known_dtype(x_dtype)) return TERN_ERR_DTYPE;
    if (M == 0 || K == 0) return TERN_OK;
    if (X == nullptr) return TERN_ERR_NULL;
    if ((st = check_q8_pointers(codes, scales)) != TERN_OK) return st;
    if (!aligned(X, dtype_size(x_dtype))) return TERN_ERR_ALIGN;
    tern::NormArgs a{};
    a.X = X;
    a.x_dtype = dtype_index(x_dtype);
    a.Q = codes;
    a.S = scales;
    a.M = q_group != 0 ? M * (K / q_group) : M;   // blocks are rows of their own
    a.K = q_group != 0 ? q_group : K;
    a.stream = stream;
    return from_hip(tern::launch_norm(a));
}

tern_status tern_q8_dequant(const int8_t *codes, const float *scales, int32_t q_group, void *Y, tern_dtype y_dtype,
                            int64_t M, int64_t K, hipStream_t stream) {
    tern_status st = check_q8_sizes(q_group, M, K);
    if (st != TERN_OK) return st;
    if (!known_dtype(y_dtype)) return TERN_ERR_DTYPE;
    if (M == 0 || K == 0) return TERN_OK;
    if (Y == nullptr) return TERN_ERR_NULL;
    if ((st = check_q8_pointers(codes, scales)) != TERN_OK) return st;
    if (!aligned(Y, dtype_size(y_dtype))) return TERN_ERR_ALIGN;
    const int64_t width = q_group != 0 ? q_group : K;
    return from_hip(tern::launch_q8_dequant(codes, scales, Y, dtype_index(y_dtype), M * (K / width), width, stream));
}

size_t tern_matmul_q8_workspace(int64_t M, int64_t N, int64_t K) {
    if (!q8_product_ok(M, N, K) || M == 0 || N == 0 || K == 0 || K % TERN_GROUP != 0) return 0;
    return q8_workspace(M, N, K);
}

tern_status tern_matmul_q8(const int8_t *x_codes, const float *x_scales, int32_t q_group, const uint8_t *packed_W,
                           const uint16_t *scales, void *Y, tern_dtype y_dtype, int64_t M, int64_t N, int64_t K,
                           int32_t group, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!q8_product_ok(M, N, K)) return TERN_ERR_SHAPE;
    if (group <= 0 || K % group != 0) return TERN_ERR_GROUP;
    if (!known_dtype(y_dtype)) return TERN_ERR_DTYPE;
    if (group != TERN_GROUP || (q_group != 0 && q_group != TERN_GROUP)) return TERN_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return TERN_OK;
    if (Y == nullptr) return TERN_ERR_NULL;
    if (!aligned(Y, dtype_size(y_dtype))) return TERN_ERR_ALIGN;
    if (K == 0) return from_hip(tern::launch_fill_zero(Y, M * N * (int64_t)dtype_size(y_dtype), stream));
    if (x_codes == nullptr || x_scales == nullptr || packed_W == nullptr || scales == nullptr) return TERN_ERR_NULL;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 4) || !aligned(packed_W, 16) || !aligned(scales, 2))
        return TERN_ERR_ALIGN;
    const Q8Kernel kernel = q8_kernel(M, N, K);
    const size_t need = kernel == Q8Kernel::Tiles ? tern::q8_gemm_workspace(M, N, K) : 0;
    if (need > 0 && workspace == nullptr) return TERN_ERR_NULL;
    if (!aligned(workspace, 16)) return TERN_ERR_ALIGN;
    if (workspace_bytes < need) return TERN_ERR_SHAPE;
    if (kernel == Q8Kernel::Decode) {
        tern::GemmArgs g = make_args(x_codes, TERN_BF16, packed_W, scales, nullptr, x_scales, Y, y_dtype, M, N, K, stream);
        g.x_dtype = 3;
        g.x_grouped = q_group != 0;
        return from_hip(tern::launch_gemv_fp4(g));
    }
    tern::Q8Args a;
    a.Q = x_codes;
    a.XS = x_scales;
    a.grouped = q_group != 0;
    a.W = packed_W;
    a.S = scales;
    a.Y = Y;
    a.y_dtype = dtype_index(y_dtype);
    a.M = M;
    a.N = N;
    a.K = K;
    a.terms = workspace;
    a.w_scales = a.x_scales = nullptr;
    a.stream = stream;
    return from_hip(kernel == Q8Kernel::Rows     ? tern::launch_q8_rows(a)
                    : kernel == Q8Kernel::Blocks ? tern::launch_q8_blocks(a)
                                                 : tern::launch_q8_gemm(a));
}

}  // extern "C"
