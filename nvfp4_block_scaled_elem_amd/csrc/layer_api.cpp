// C ABI of the layer operators (declared in include/nvfp4.h): argument checks on the host, scratch, launches.
//
// Kernels per call (all on the caller's stream):
//   nvfp4_rms_norm        : k_rms_norm, or k_rms_norm_long beyond 16384 columns
//   nvfp4_rms_norm_grad   : k_rms_norm_grad -> k_column_sum (beyond 16384 columns: k_rms_norm_grad_long ->
//                           k_rms_norm_dw_long -> k_column_sum)
//   nvfp4_mxfp8_quantize / nvfp4_mxfp8_dequantize : one kernel each
//   nvfp4_linear          : (k_lin_xfrag ->) k_lin_skinny, or (k_mx_dequantize ->) (k_lin_decode ->) tiles
//   nvfp4_linear_grad     : (k_lin_dz with an activation or dbias; -> k_column_sum with dbias) -> (k_lin_transpose ->) tiles
//     tiles: k_lin_tile (-> k_lin_reduce where K is split), once or, the last columns by themselves, twice. Without
//     k_lin_decode and k_lin_transpose the weights are decoded in k_lin_tile, whichever is estimated to take less.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "host.hpp"
#include "launch.hpp"

namespace {

using nvfp4::NormArgs;
using nvfp4::aligned;
using nvfp4::plain_dtype;
using nvfp4::status;
using nvfp4::width;
using nvfp4::with_scratch;

// Fewer than 2^32 threads per dimension of a grid: 2^23 rows of 256 threads, and 2^35 - 2^11 elements (rows counted in whole
// blocks of 32) by eight per thread in work-groups of 256.
constexpr int64_t kMaxElems = ((int64_t)1 << 35) - ((int64_t)1 << 11);
constexpr int64_t kMaxRows = (int64_t)1 << 23;

// NVFP4_OK for a [rows][cols] operand of rows >= 0 with `ld` elements between rows.
int check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0) return NVFP4_ERR_INVALID_ARG;
    if (rows > kMaxRows || cols > kMaxElems) return NVFP4_ERR_SHAPE;
    if (rows * ((cols + 31) / 32 * 32) > kMaxElems) return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}

}  // namespace

NVFP4_API int nvfp4_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                             int dtype, int weight_dtype, int64_t rows, int64_t cols, float eps, void *sum_out,
                             void *y, uint8_t *y_scales, int y_dtype, void *stream) {
    if (!plain_dtype(dtype) || !plain_dtype(weight_dtype)) return NVFP4_ERR_INVALID_ARG;
    if (!plain_dtype(y_dtype) && y_dtype != NVFP4_DTYPE_MXFP8) return NVFP4_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps < INFINITY)) return NVFP4_ERR_INVALID_ARG;
    const int c = check_shape(rows, cols);
    if (c != NVFP4_OK) return c;
    if (rows == 0) return NVFP4_OK;
    if (!x || !weight || !y || (residual != nullptr) != (sum_out != nullptr) ||
        (y_dtype == NVFP4_DTYPE_MXFP8) != (y_scales != nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if ((rows > 1 && ldx < cols) || (residual && rows > 1 && ldr < cols)) return NVFP4_ERR_INVALID_ARG;
    const unsigned a = width(dtype);
    if (!aligned(x, a) || !aligned(residual, a) || !aligned(sum_out, a) || !aligned(weight, width(weight_dtype)) ||
        !aligned(y, width(y_dtype)))
        return NVFP4_ERR_INVALID_ARG;
    NormArgs p = {};
    p.x = x, p.r = residual, p.w = weight, p.y = y, p.h = sum_out, p.ys = y_scales;
    p.rows = rows, p.cols = cols, p.ldx = ldx, p.ldr = residual ? ldr : 0, p.eps = eps;
    p.w_f32 = weight_dtype == NVFP4_DTYPE_F32;
    p.out = y_dtype == NVFP4_DTYPE_MXFP8 ? nvfp4::kOutMx : y_dtype == NVFP4_DTYPE_F32 ? nvfp4::kOutF32 : nvfp4::kOutBf16;
    return status(nvfp4::launch_rms_norm(p, dtype == NVFP4_DTYPE_F32, static_cast<hipStream_t>(stream)));
}

NVFP4_API size_t nvfp4_rms_norm_grad_workspace_bytes(int64_t rows, int64_t cols) {
    return check_shape(rows, cols) == NVFP4_OK ? nvfp4::rms_norm_grad_workspace(rows, cols) : 0;
}

NVFP4_API int nvfp4_rms_norm_grad(const void *dy, int64_t lddy, const void *h, int64_t ldh, const uint8_t *h_scales,
                                  int h_dtype, const void *weight, const void *dh, int64_t lddh, int dtype,
                                  int weight_dtype, int64_t rows, int64_t cols, float eps, void *dx, float *dweight,
                                  void *workspace, size_t workspace_bytes, void *stream) {
    if (!plain_dtype(dtype) || !plain_dtype(weight_dtype)) return NVFP4_ERR_INVALID_ARG;
    if (h_dtype != dtype && h_dtype != NVFP4_DTYPE_MXFP8) return NVFP4_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps < INFINITY)) return NVFP4_ERR_INVALID_ARG;
    const int c = check_shape(rows, cols);
    if (c != NVFP4_OK) return c;
    const bool mx = h_dtype == NVFP4_DTYPE_MXFP8;
    if (!dweight || !aligned(dweight, 4) || !aligned(workspace, 256)) return NVFP4_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!dy || !h || !weight || !dx || mx != (h_scales != nullptr)) return NVFP4_ERR_INVALID_ARG;
        if (rows > 1 && (lddy < cols || ldh < cols || (dh && lddh < cols))) return NVFP4_ERR_INVALID_ARG;
        const unsigned a = width(dtype);
        if (!aligned(dy, a) || !aligned(dh, a) || !aligned(dx, a) || !aligned(h, width(h_dtype)) ||
            !aligned(weight, width(weight_dtype)))
            return NVFP4_ERR_INVALID_ARG;
    }
    NormArgs p = {};
    p.x = h, p.r = dh, p.w = weight, p.dy = dy, p.xs = h_scales, p.y = dx;
    p.rows = rows, p.cols = cols, p.ldx = ldh, p.ldr = dh ? lddh : 0, p.lddy = lddy, p.eps = eps;
    p.w_f32 = weight_dtype == NVFP4_DTYPE_F32;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_scratch(workspace, workspace_bytes, nvfp4::rms_norm_grad_workspace(rows, cols), st, [&](void *ws) {
        return nvfp4::launch_rms_norm_grad(p, dtype == NVFP4_DTYPE_F32, mx, dweight, static_cast<float *>(ws), st);
    });
}

NVFP4_API int nvfp4_mxfp8_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int64_t cols, uint8_t *codes,
                                   uint8_t *scales, void *stream) {
    if (!plain_dtype(dtype)) return NVFP4_ERR_INVALID_ARG;
    const int c = check_shape(rows, cols);
    if (c != NVFP4_OK) return c;
    if (rows == 0) return NVFP4_OK;
    if (!x || !codes || !scales || (rows > 1 && ldx < cols) || !aligned(x, width(dtype))) return NVFP4_ERR_INVALID_ARG;
    return status(nvfp4::launch_mx_quantize(x, dtype == NVFP4_DTYPE_F32, rows, cols, ldx, codes, scales,
                                            static_cast<hipStream_t>(stream)));
}

NVFP4_API int nvfp4_mxfp8_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t rows,
                                     int64_t cols, void *y, int y_dtype, void *stream) {
    if (!plain_dtype(y_dtype)) return NVFP4_ERR_INVALID_ARG;
    const int c = check_shape(rows, cols);
    if (c != NVFP4_OK) return c;
    if (rows == 0) return NVFP4_OK;
    if (!codes || !scales || !y || (rows > 1 && ldc < cols) || !aligned(y, width(y_dtype))) return NVFP4_ERR_INVALID_ARG;
    return status(nvfp4::launch_mx_dequantize(codes, ldc, scales, rows, cols, y, y_dtype == NVFP4_DTYPE_F32,
                                              static_cast<hipStream_t>(stream)));
}

namespace {

constexpr int64_t kMaxLd = (int64_t)1 << 23;    // a product's X: 256 rows of it stay below 2^32 bytes
constexpr int64_t kMaxSide = (int64_t)1 << 21;  // K and N of a product: grids stay below 65536 along y

// The shapes of a product [M][K] x [N][K]^T, gated or not. The weights are held to the bound of every operand: the
// kernels' 32-bit offsets of scale bytes and their grids rest on it.
int check_product(int64_t M, int64_t K, int64_t N, int activation, int gated) {
    if (M < 0 || K <= 0 || N <= 0) return NVFP4_ERR_INVALID_ARG;
    if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_GELU) return NVFP4_ERR_INVALID_ARG;
    if (gated != 0 && (gated != 1 || activation == NVFP4_ACT_NONE)) return NVFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || (gated && N % 2 != 0) || K > kMaxSide || N > kMaxSide) return NVFP4_ERR_SHAPE;
    for (const int c : {check_shape(M, K), check_shape(M, N), check_shape(N, K)})
        if (c != NVFP4_OK) return c;
    return NVFP4_OK;
}

}  // namespace

NVFP4_API size_t nvfp4_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, int x_dtype, int gated, int z_dtype) {
    if (check_product(M, K, N, gated ? NVFP4_ACT_SILU : NVFP4_ACT_NONE, gated) != NVFP4_OK || M == 0) return 0;
    const nvfp4::LinPlan plan =
        nvfp4::plan_linear(M, K, N, x_dtype == NVFP4_DTYPE_MXFP8, gated != 0, z_dtype == NVFP4_DTYPE_MXFP8 ? nvfp4::kKeepMx : nvfp4::kKeepNone);
    return plan.x_bytes + plan.part_bytes + plan.frag_bytes;
}

NVFP4_API int nvfp4_linear(const nvfp4_linear_args_t *a) {
    if (!a) return NVFP4_ERR_INVALID_ARG;
    const int c = check_product(a->M, a->K, a->N, a->activation, a->gated);
    if (c != NVFP4_OK) return c;
    const int64_t F = a->gated ? a->N / 2 : a->N;
    const bool xmx = a->x_dtype == NVFP4_DTYPE_MXFP8, zmx = a->z_dtype == NVFP4_DTYPE_MXFP8;
    if ((!xmx && a->x_dtype != NVFP4_DTYPE_BF16) || !plain_dtype(a->y_dtype)) return NVFP4_ERR_INVALID_ARG;
    if (a->z && !zmx && a->z_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_INVALID_ARG;
    if ((a->bias && !plain_dtype(a->bias_dtype)) || (a->residual && !plain_dtype(a->residual_dtype)))
        return NVFP4_ERR_INVALID_ARG;
    if (a->z && zmx && a->gated && F % 32 != 0) return NVFP4_ERR_SHAPE;
    if (!aligned(a->workspace, 256)) return NVFP4_ERR_INVALID_ARG;
    if (a->M == 0) return NVFP4_OK;
    if (!a->x || !a->codes || !a->scales || !a->alpha || !a->y || xmx != (a->x_scales != nullptr) ||
        (a->z && zmx) != (a->z_scales != nullptr))
        return NVFP4_ERR_INVALID_ARG;
    if (a->M > 1 && (a->ldx < a->K || (a->residual && a->ldr < F))) return NVFP4_ERR_INVALID_ARG;
    if (a->M > 1 && a->ldx >= kMaxLd) return NVFP4_ERR_SHAPE;
    if (!aligned(a->x, width(a->x_dtype)) || !aligned(a->codes, 8) || !aligned(a->alpha, 4) ||
        !aligned(a->y, width(a->y_dtype)) || (a->bias && !aligned(a->bias, width(a->bias_dtype))) ||
        (a->residual && !aligned(a->residual, width(a->residual_dtype))) || (a->z && !aligned(a->z, width(a->z_dtype))))
        return NVFP4_ERR_INVALID_ARG;
    nvfp4::LinArgs p = {};
    p.x = a->x, p.xs = a->x_scales, p.x_mx = xmx, p.ldx = a->ldx;
    p.codes = a->codes, p.scales = a->scales, p.alpha = a->alpha;
    p.bias = a->bias, p.bias_f32 = a->bias_dtype == NVFP4_DTYPE_F32;
    p.res = a->residual, p.res_f32 = a->residual_dtype == NVFP4_DTYPE_F32, p.ldr = a->residual ? a->ldr : 0;
    p.y = a->y, p.y_f32 = a->y_dtype == NVFP4_DTYPE_F32;
    p.z = a->z, p.zs = a->z_scales, p.keep = !a->z ? nvfp4::kKeepNone : zmx ? nvfp4::kKeepMx : nvfp4::kKeepBf16;
    p.M = a->M, p.L = a->K, p.N = a->N, p.F = F, p.act = a->activation, p.gated = a->gated;
    if (a->M == 1) p.ldx = a->K;
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    const nvfp4::LinPlan plan = nvfp4::plan_linear(p.M, p.L, p.N, p.x_mx, p.gated, p.keep);
    return with_scratch(a->workspace, a->workspace_bytes, plan.x_bytes + plan.part_bytes + plan.frag_bytes, st,
                        [&](void *ws) { return nvfp4::launch_linear(p, ws, st); });
}

NVFP4_API size_t nvfp4_linear_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int gated, int with_dbias) {
    if (check_product(M, K, N, gated ? NVFP4_ACT_SILU : NVFP4_ACT_NONE, gated) != NVFP4_OK) return 0;
    return nvfp4::linear_grad_workspace(M, K, N, gated ? N / 2 : N, with_dbias != 0);
}

NVFP4_API int nvfp4_linear_grad(const nvfp4_linear_grad_args_t *a) {
    if (!a) return NVFP4_ERR_INVALID_ARG;
    const int c = check_product(a->M, a->K, a->N, a->activation, a->gated);
    if (c != NVFP4_OK) return c;
    const int64_t F = a->gated ? a->N / 2 : a->N;
    const bool act = a->activation != NVFP4_ACT_NONE, zmx = act && a->z_dtype == NVFP4_DTYPE_MXFP8;
    if (act && !zmx && a->z_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_INVALID_ARG;
    if (zmx && a->gated && F % 32 != 0) return NVFP4_ERR_SHAPE;
    if (!aligned(a->workspace, 256) || !aligned(a->dbias, 4)) return NVFP4_ERR_INVALID_ARG;
    if (a->M > 0) {
        if (!a->dy || !a->codes || !a->scales || !a->alpha || !a->dx || act != (a->z != nullptr) ||
            act != (a->dz != nullptr) || zmx != (a->z_scales != nullptr))
            return NVFP4_ERR_INVALID_ARG;
        if (a->M > 1 && (a->lddy < F || (act && a->ldz < a->N))) return NVFP4_ERR_INVALID_ARG;
        if (a->M > 1 && a->lddy >= kMaxLd) return NVFP4_ERR_SHAPE;
        if (!aligned(a->dy, 2) || !aligned(a->codes, 8) || !aligned(a->alpha, 4) || !aligned(a->dx, 2) ||
            !aligned(a->dz, 2) || (act && !aligned(a->z, width(a->z_dtype))))
            return NVFP4_ERR_INVALID_ARG;
    }
    nvfp4::LinGradArgs g = {};
    g.dy = static_cast<const uint16_t *>(a->dy), g.lddy = a->M > 1 ? a->lddy : F;
    g.z = a->z, g.zs = a->z_scales, g.z_mx = zmx, g.ldz = a->M > 1 ? a->ldz : a->N;
    g.dz = static_cast<uint16_t *>(a->dz);
    g.M = a->M, g.N = a->N, g.F = F, g.act = a->activation, g.gated = a->gated;
    hipStream_t st = static_cast<hipStream_t>(a->stream);
    const size_t need = nvfp4::linear_grad_workspace(a->M, a->K, a->N, F, a->dbias != nullptr);
    return with_scratch(a->workspace, a->workspace_bytes, need, st, [&](void *ws) {
        return nvfp4::launch_linear_grad(g, a->codes, a->scales, a->alpha, a->K, a->dx, a->dbias, ws, st);
    });
}
