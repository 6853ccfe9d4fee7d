/*
 * nvfp4.h - C ABI of the MI355X (gfx950) NVFP4 weight quantizer.
 *
 * What the calls compute:
 *   NVFP4 quantisation of a weight matrix W into FP4 (E2M1) codes Q, one FP8 (E4M3) scale Delta_i per
 *   block of 16 consecutive elements of a row, and one FP32 global scale alpha, so that
 *   W ~ Q * Delta_i * alpha. The four modes are the ones the two pages describe:
 *     NVFP4_MODE_MAX           the max rule of the SOAR page ("SOAR: Scale Optimization for Accurate
 *                              Reconstruction in NVFP4 Quantization", quantisation equations):
 *                              alpha = max|W| / (6*448), Delta_i = E4M3(max|W_i| / (6*alpha)).
 *     NVFP4_MODE_FOUR_OVER_SIX the FourOverSix choice of the write-up "SOAR 周冠军笔记 07 |
 *                              香草小张：NVFP4 量化改进与推测解码实践", section 02: per block, the M=4
 *                              scale E4M3(1.5*Delta_i) replaces Delta_i when its squared reconstruction
 *                              error is strictly smaller.
 *     NVFP4_MODE_CJSO          the SOAR page's closed-form joint scale optimisation: from the max rule,
 *                              `iters` rounds of {least-squares alpha, re-quantise, least-squares Delta_i
 *                              rounded to E4M3, re-quantise}.
 *     NVFP4_MODE_SOAR          CJSO followed by the SOAR page's decoupled search: per block, quantise with
 *                              Delta_q = Delta_c * f (f = 0.50, 0.51, ..., 1.50) and reconstruct with
 *                              Delta_d, one of the two E4M3 values around the unrounded CJSO scale; keep
 *                              the least squared error (202 candidates, CJSO's own point first, strict <).
 *   Arithmetic: scaled values are x = w * (1/(alpha*Delta)) in binary32, rounded to the nearest E2M1
 *   value with ties to the even code and |x| > 6 saturating to 6 (a value rounding to 0 gets code 0);
 *   every choice between candidates compares exact squared errors. The results are bit-identical to
 *   the CPU oracle that defines them.
 *
 * Layout (row-major, contiguous, caller-owned):
 *   W          [rows][cols] bf16 (nvfp4_quantize) or fp32 (nvfp4_quantize_f32), 16-byte aligned.
 *   codes_out  [rows][cols/2] bytes, 8-byte aligned: byte k of a row holds column 2k in its low nibble
 *              and column 2k+1 in its high nibble; a code is sign (bit 3) | index into
 *              {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
 *   scales_out [rows][cols/16] E4M3 bytes (sign bit 0; at most 0x7E = 448).
 *   alpha_out  one float. Dequantisation: w_hat = e2m1(code) * e4m3(scale) * alpha.
 *   All pointers are device pointers (hipMalloc'd or torch CUDA tensors); `stream` is a hipStream_t
 *   (NULL = the default stream).
 *
 * Calls are asynchronous: they validate their arguments on the host, enqueue kernels on `stream` and
 * return. Results are valid once the stream has reached that point. The library keeps no pointer after
 * the enqueued work ends and has no mutable global state: calls on different streams may overlap, and
 * calls that share output buffers must be ordered by the caller.
 *
 * Errors: negative return values are reported synchronously and nothing is enqueued, except
 * NVFP4_ERR_HIP (a launch or allocation failed; work enqueued before the failure may still run).
 * Data-dependent conditions are reported in band: a NaN or an infinity anywhere in W gives
 * alpha_out = NaN and all-zero codes and scales (and sets NVFP4_STATUS_NONFINITE in the stats); an
 * all-zero W gives alpha = 0 with all-zero codes and scales.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum nvfp4_mode {
    NVFP4_MODE_MAX = 0,
    NVFP4_MODE_FOUR_OVER_SIX = 1,
    NVFP4_MODE_CJSO = 2,
    NVFP4_MODE_SOAR = 3
};

/* MXFP8 is a form of activations (the layer operators below); no entry point of the quantiser takes it. */
enum nvfp4_dtype { NVFP4_DTYPE_BF16 = 0, NVFP4_DTYPE_F32 = 1, NVFP4_DTYPE_MXFP8 = 2 };

/* How the SOAR search picks each candidate's two E4M3 reconstruct scales Delta_d (SOAR page, decoupled
 * search: "the two E4M3 values nearest the current value"). CJSO: the pair around the unrounded CJSO
 * scale, for every candidate (the reading of the page the default search takes). QUANT: the pair
 * around the candidate's quantisation scale Delta_q. LSQ: the pair around the least-squares scale of
 * the candidate's own codes (the block-scale step applied to them; a candidate whose codes are all
 * zero keeps Delta_c). */
enum nvfp4_dd_rule { NVFP4_DD_CJSO = 0, NVFP4_DD_QUANT = 1, NVFP4_DD_LSQ = 2 };
#define NVFP4_SEARCH_MAX_COUNT 1024

enum nvfp4_error {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARG = -1, /* null or misaligned pointer, rows/cols <= 0, unknown mode or dtype,
                                   iters outside [0, 1000] */
    NVFP4_ERR_SHAPE = -2,       /* cols % 16 != 0, or more than 2^35 elements */
    NVFP4_ERR_WORKSPACE = -3,   /* caller workspace smaller than nvfp4_workspace_bytes() */
    NVFP4_ERR_HIP = -4,         /* a HIP call failed */
    NVFP4_ERR_TOO_LARGE = -5,   /* nvfp4_quantize_noalloc: the call needs more scratch than its fixed
                                   device array holds */
    NVFP4_ERR_UNSUPPORTED = -6  /* nvfp4_matmul / nvfp4_matmul_ex on a capturing stream with a shape
                                   that takes the 128 x 128 or 256 x 128 output tiles; a layer operator on
                                   a capturing stream that needs scratch and was given none */
};

/* In-band status bits, written to nvfp4_stats_t.status by the device. */
#define NVFP4_STATUS_NONFINITE 1u

/* Optional per-call statistics in device memory (written by the call). */
typedef struct nvfp4_stats {
    uint32_t status;    /* NVFP4_STATUS_* bits */
    uint32_t m4_blocks; /* FourOverSix: number of blocks that kept M=4 */
    uint32_t reserved[2];
} nvfp4_stats_t;

/* Quantise a bf16 matrix. `iters` is the number of CJSO rounds (modes 2 and 3; ignored otherwise,
 * 0 makes CJSO equal to MAX). A scratch workspace is taken from a stream-ordered pool and given
 * back on the same stream. */
int nvfp4_quantize(const void *W, int64_t rows, int64_t cols, int mode, int iters, uint8_t *codes_out,
                   uint8_t *scales_out, float *alpha_out, void *stream);

/* Same for an fp32 matrix. */
int nvfp4_quantize_f32(const float *W, int64_t rows, int64_t cols, int mode, int iters,
                       uint8_t *codes_out, uint8_t *scales_out, float *alpha_out, void *stream);

/* Full argument set. */
typedef struct nvfp4_args {
    const void *W;
    int dtype; /* enum nvfp4_dtype */
    int64_t rows, cols;
    int mode; /* enum nvfp4_mode */
    int iters;
    uint8_t *codes_out;
    uint8_t *scales_out;
    float *alpha_out;
    uint8_t *mchoice_out;     /* nullable: [rows][cols/16] bytes, 1 where FourOverSix kept M=4 (mode 1) */
    nvfp4_stats_t *stats_out; /* nullable, device memory */
    void *workspace;          /* nullable: device memory of workspace_bytes, 256-byte aligned; NULL =
                                 the library allocates on `stream` */
    size_t workspace_bytes;
    void *stream;             /* hipStream_t */
    void *const *stage_events; /* nullable: nvfp4_kernel_count(mode, iters) + 1 hipEvent_t handles; the
                                  call records stage_events[0] before its first kernel and
                                  stage_events[j + 1] after kernel j, so each kernel can be timed on
                                  `stream`; NULL entries are skipped (fewer records, smaller gaps) */
    int n_stage_events;
    unsigned flags; /* NVFP4_FLAG_* bits (0 for the defaults) */
    /* SOAR search grid (mode 3; all three 0 elsewhere and for the page's grid, f_k = (50 + k)/100 for
     * k = 0..100): multipliers f_k = the binary32 value nearest (search_num0 + k) / search_den for
     * k < search_count, with 1 <= search_den <= 2^24, search_num0 >= 1,
     * 1 <= search_count <= NVFP4_SEARCH_MAX_COUNT and search_num0 + search_count - 1 <= 16 * search_den
     * (multipliers at most 16). Any other setting is NVFP4_ERR_INVALID_ARG. */
    int search_num0, search_den, search_count;
    int dd_rule; /* enum nvfp4_dd_rule (mode 3; 0 elsewhere). QUANT and LSQ scan every multiplier. */
} nvfp4_args_t;

/* SOAR: visit all 202 candidates of every block. Without it the search evaluates, per reconstruct
 * scale, only the two or three quantise scales next to it, which is exact: the block error is
 * unimodal in the quantise scale around that window (the kernel source gives the argument), so the
 * outputs are identical either way. The flag exists to check that and to time the full search. */
#define NVFP4_FLAG_FULL_SEARCH 1u
/* CJSO and SOAR: start from FourOverSix's block scales (each block's M=6 or M=4 choice, FourOverSix
 * write-up, section 02) instead of the max rule; alpha still starts from the max rule. For SOAR with no
 * rounds, the unrounded scale whose E4M3 neighbours the search tries is max|w|/(6 alpha), or 1.5*Delta6
 * for a block that took M=4. Not accepted for modes 0 and 1. */
#define NVFP4_FLAG_INIT_4O6 2u

int nvfp4_quantize_ex(const nvfp4_args_t *args);

/* nvfp4_quantize_ex for callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation. It allocates nothing (no hipMalloc, hipMallocAsync or
 * hipFree, neither here nor in any library it calls): its scratch is a fixed device array inside the
 * library, of nvfp4_noalloc_scratch_bytes() = 16 MiB, that every GPU the library runs on holds until the
 * process ends. The array of the current device is used, so the current device must be the stream's.
 * Same arguments, outputs and errors as nvfp4_quantize_ex, except:
 *   - args->workspace must be NULL and args->workspace_bytes 0 (else NVFP4_ERR_INVALID_ARG);
 *   - NVFP4_ERR_TOO_LARGE when nvfp4_workspace_bytes(rows, cols, mode) exceeds the array: MAX,
 *     FourOverSix and CJSO need 35 KB whatever the size; SOAR needs 2 more bytes per 16-element block,
 *     which caps it at about 134 million elements;
 *   - the first call on a device looks up that device's address of the array (NVFP4_ERR_HIP if that
 *     fails).
 * All calls on one GPU share its array: two calls that may overlap on one GPU (other streams, other
 * threads) race and must be ordered by the caller. Nothing in the array needs clearing between calls. */
int nvfp4_quantize_noalloc(const nvfp4_args_t *args);

/* Size in bytes of the fixed device array nvfp4_quantize_noalloc uses. */
size_t nvfp4_noalloc_scratch_bytes(void);

/* Number of kernels one call of this mode enqueues (MAX and FourOverSix: 2; CJSO: iters + 2; SOAR:
 * iters + 3; the last SOAR kernel is the decoupled search), or -1 for an unknown mode or bad iters. */
int nvfp4_kernel_count(int mode, int iters);

/* Device scratch needed by one call with these arguments (0 for an invalid shape). */
size_t nvfp4_workspace_bytes(int64_t rows, int64_t cols, int mode);

/* Round n binary32 values to E2M1 codes (one code per output byte, same rule as the quantiser:
 * nearest, ties to the even code, saturating at 6, NaN -> 0, negative results that round to zero ->
 * code 0). x and codes are device pointers; n <= 2^35 (else NVFP4_ERR_SHAPE). */
int nvfp4_encode_e2m1(const float *x, int64_t n, uint8_t *codes, void *stream);

/* The binary32 reciprocal the decoupled search uses for its quantisation scales (the candidates
 * x = w * fl(1/s) of the SOAR page's decoupled search), element-wise: r[i] = fl(1/s[i]), the correctly
 * rounded reciprocal for every input (for 2^-125 <= s < 2^125 it is computed from the hardware's
 * approximate reciprocal and one residual correction; elsewhere by IEEE division). Exported so that the
 * equality with IEEE division can be checked on the device. s and r are device pointers (4-byte
 * aligned, may not overlap); n <= 2^35 (else NVFP4_ERR_SHAPE). */
int nvfp4_reciprocal_f32(const float *s, int64_t n, float *r, void *stream);

/* Dequantise codes/scales/alpha (device pointers, layout above; alpha is a device pointer to one
 * float) into out [rows][cols] as bf16 (out_dtype 0) or fp32 (out_dtype 1):
 * out = e2m1(code) * e4m3(scale) * alpha, rounded once to the output type (SOAR page, dequantisation
 * equation). */
int nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales, const float *alpha, int64_t rows,
                     int64_t cols, void *out, int out_dtype, void *stream);

/* Reconstruction statistics of an encoding of W (SOAR page, dequantisation: w is reconstructed as
 * e2m1(code) * e4m3(scale) * alpha). W is [rows][cols] of dtype (enum nvfp4_dtype); codes, scales and
 * alpha are laid out as the quantiser writes them (scale sign bits are ignored). All pointers are device
 * pointers. On completion of the stream work:
 *   sse_out[0]  = sum over elements of d^2, d = w - (q * alpha) * Delta formed in binary64 (exact up to the
 *                 rounding of that difference) and the squares summed as double-doubles, then rounded to
 *                 binary64 (mean squared error = sse / (rows * cols));
 *   hist_out[c] = number of elements whose 4-bit code is c, c = 0..15.
 * Scratch is taken from a stream-ordered pool and given back on the same stream. Errors: as
 * nvfp4_quantize (arguments are checked on the host; nothing is enqueued on error). */
int nvfp4_error_stats(const void *W, int dtype, int64_t rows, int64_t cols, const uint8_t *codes,
                      const uint8_t *scales, const float *alpha, double *sse_out,
                      unsigned long long *hist_out, void *stream);

/* W4A16 product with NVFP4 weights, the use the format exists for: Y[M][N] = X[M][K] * What[N][K]^T with
 * What = e2m1(code) * e4m3(scale) * alpha (SOAR page, dequantisation equation), for a weight matrix [N][K]
 * stored as the quantiser writes it (codes [N][K/2], scales [N][K/16], alpha one float). X is bf16
 * [M][K] row-major; Y is [M][N] of y_dtype (NVFP4_DTYPE_BF16 or _F32). All pointers are device pointers;
 * X, codes and Y 16-byte aligned; K % 16 == 0, N <= 2^25 and fewer than 2^24 output tiles of 256 x 128
 * (else NVFP4_ERR_SHAPE). Arithmetic: every q * Delta is a bf16 value,
 * so the products with X are exact; the sum over k is accumulated in fp32 (packed bf16 dot products when
 * M <= 4, M * K * 2 <= 128 KiB and K <= 16384; bf16 MFMA otherwise) in an order the caller does not
 * control, then multiplied by alpha and
 * rounded once to the output type. When the output tiles are too few to fill the GPU, K is split and the
 * slices' fp32 sums (slices * M * N * 4 bytes, at most 1 GiB) go through scratch taken from a
 * stream-ordered pool and given back on the same stream; the slices are added in a fixed order, so
 * results are reproducible. Enqueued on `stream`; argument errors are returned synchronously. */
int nvfp4_matmul(const void *X, int64_t M, int64_t K, const uint8_t *codes, const uint8_t *scales,
                 const float *alpha, int64_t N, void *Y, int y_dtype, void *stream);

/* nvfp4_matmul with caller-supplied scratch for the K split: `workspace` (device memory, 256-byte aligned,
 * nullable) of `workspace_bytes` >= nvfp4_matmul_workspace_bytes(M, K, N) bytes. With a workspace nothing
 * is allocated, so the call may be captured into a HIP graph as plain kernel nodes; the workspace must then
 * stay allocated while the graph may run. NULL behaves as nvfp4_matmul. NVFP4_ERR_WORKSPACE if it is too
 * small. Same arithmetic, layout and errors as nvfp4_matmul.
 * Stream capture: shapes whose plan takes the 128 x 128 or 256 x 128 output tiles (nvfp4_matmul_plan:
 * kernel 2, tile columns 128) are refused on a capturing stream with NVFP4_ERR_UNSUPPORTED (nothing is
 * enqueued): one graph-captured run of those forms ended in a device memory fault whose cause has not been
 * found. The GEMV, the skinny kernel and the 128 x 64 tiles (with or without the K split) may be
 * captured. Eager calls of every shape are unaffected. */
int nvfp4_matmul_ex(const void *X, int64_t M, int64_t K, const uint8_t *codes, const uint8_t *scales,
                    const float *alpha, int64_t N, void *Y, int y_dtype, void *workspace, size_t workspace_bytes,
                    void *stream);

/* Scratch bytes nvfp4_matmul_ex needs for these shapes: slices * M * N * 4 when K is split, else 0 (also 0
 * for shapes nvfp4_matmul rejects). */
size_t nvfp4_matmul_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* The launch nvfp4_matmul takes for these shapes, for tests and tuning (no device work): plan_out[10] gets
 * {kernel (0 GEMV, 1 skinny MFMA, 2 tiled MFMA), tile rows (tiled; the rows of X compiled for, skinny),
 * tile columns, tiles along N, tiles, K slices, K per slice, work-groups, reduction work-groups, scratch
 * bytes}. Returns NVFP4_ERR_INVALID_ARG for a null pointer, a dimension <= 0 or K % 16 != 0. */
int nvfp4_matmul_plan(int64_t M, int64_t K, int64_t N, int64_t *plan_out);

/* GPTQ with the FourOverSix block scales fixed first (FourOverSix write-up, section 03: every block's
 * scale and its M = 6 / M = 4 choice are settled before GPTQ's weight iterations, which then run inside
 * that frame; GPTQ as published by Frantar, Ashkboos, Hoefler and Alistarh, 2022).
 *
 * Steps:
 *   1. The frame. scales_out and alpha_out are exactly nvfp4_quantize's FourOverSix result for W.
 *   2. GPTQ's preparation of H [cols][cols], the second moment of the layer's inputs. Inputs with a zero
 *      diagonal are dead: their weights count as zero and their diagonal as one. Every diagonal entry then
 *      gains percdamp * mean(diagonal).
 *   3. The columns in order. Each is quantised to the nearest E2M1 value of w~ / s in binary64, where
 *      s = fl32(alpha * Delta) of its block (ties to the even code; s = 0 gives code 0). Its error is spread
 *      over the later columns as GPTQ specifies: given the columns already fixed, the later weights are the
 *      minimiser of the H-weighted error. All of this runs in binary64.
 *   codes_out gets the resulting codes.
 *
 * Arguments:
 *   W           [rows][cols], dtype bf16 or fp32, 16-byte aligned.
 *   H           device binary64, row-major, symmetric; only its upper triangle (H[i][j], i <= j) is read.
 *   percdamp    finite and >= 0 (GPTQ's usual value is 0.01).
 *   codes_out, scales_out, alpha_out
 *               as for nvfp4_quantize.
 *   workspace   nullable; 256-byte aligned, of nvfp4_gptq_workspace_bytes(rows, cols) bytes, about
 *               8 * (cols^2 + rows * cols) bytes. NULL = the library allocates on `stream` and gives the
 *               scratch back on `stream`.
 *
 * Limits: cols % 16 == 0, cols <= 32768, rows <= 65535 * 64 and rows * cols <= 2^32 (else
 *         NVFP4_ERR_SHAPE).
 *
 * Errors:
 *   - Arguments are checked on the host, as for nvfp4_quantize.
 *   - If the damped H is not positive definite in binary64 (a Cholesky pivot that is not positive and
 *     finite), alpha_out = NaN and every code is 0 when the stream work ends.
 *   - A NaN or infinity in W gives FourOverSix's in-band result (alpha NaN, all-zero codes and scales). */
int nvfp4_gptq(const void *W, int dtype, int64_t rows, int64_t cols, const double *H, double percdamp,
               uint8_t *codes_out, uint8_t *scales_out, float *alpha_out, void *workspace,
               size_t workspace_bytes, void *stream);

/* Device scratch one nvfp4_gptq call needs (0 for an invalid shape). */
size_t nvfp4_gptq_workspace_bytes(int64_t rows, int64_t cols);

/* ------------------------------------------------------------------------------------ layer operators
 *
 * What a layer computes around its NVFP4 products, forward and backward.
 *
 * All of them: device pointers, row-major; `ld*` is the number of elements from a row of an operand to the
 * next (>= its columns; not looked at for fewer than two rows), the outputs are contiguous. Pointers are
 * aligned to their element; rows need no more alignment than that (16-byte aligned rows are fastest). rows = 0
 * is allowed: nothing is written but the column sums (dweight, dbias), which are zeros. rows <= 2^23 and, with
 * columns rounded up to 32, rows * columns <= 2^35 - 2^11 for every operand, weights among them (else
 * NVFP4_ERR_SHAPE). Outputs may not overlap inputs unless a call says so. Sums and statistics are binary32, in
 * an order that does not depend on timing; each output is rounded once.
 * Nothing is allocated when `workspace` (256-byte aligned) is given or none is needed; without it scratch
 * is taken from a stream-ordered pool, except on a capturing stream (NVFP4_ERR_UNSUPPORTED). A call writes what
 * it reads of its workspace, so calls and captured graphs may share one if they run one after the other; calls
 * or replays that may overlap need one each.
 *
 * MXFP8 ([rows][cols] code bytes and [rows][ceil(cols/32)] scale bytes): blocks of 32 consecutive columns
 * (the last may be shorter); a code is E4M3, a scale byte b is 2^(b-127) (E8M0), and a value is their
 * product. The scale written is the smallest power of two, 2^-127 at least, with max|v| <= 448 * scale, so
 * nothing saturates and a value is within half an E4M3 step (from 1.9375 * 2^127 on that is 2^128, which reads as
 * an infinity). Zeros: b = 0. A block holding a NaN or an infinity:
 * b = 255, codes 0x7F, and all its values read as NaN. */

/* MXFP8 codes and scales of x (dtype bf16 or fp32, [rows][cols], any cols >= 1), as activations are kept in
 * between a forward and a backward pass; and the values back, rounded to bf16 or fp32 (both hold every value
 * below 2^128 whose scale is at least 2^-117). */
int nvfp4_mxfp8_quantize(const void *x, int64_t ldx, int dtype, int64_t rows, int64_t cols, uint8_t *codes,
                         uint8_t *scales, void *stream);
int nvfp4_mxfp8_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t rows, int64_t cols,
                           void *y, int y_dtype, void *stream);

/* Root-mean-square norm with the residual's addition: h = x + residual, y = h * (mean(h^2) + eps)^(-1/2) *
 * weight over each row of cols >= 1 columns. x, residual and sum_out have `dtype` (bf16 or fp32), weight [cols]
 * has weight_dtype. sum_out gets h rounded to dtype (y is computed from h unrounded) and may be `residual`
 * itself (contiguous); residual and sum_out are both given or both NULL (then h = x). y is bf16, fp32 or
 * MXFP8 (y_dtype; y_scales for MXFP8 alone, else NULL). eps >= 0. Squares are binary32: where a row's sum of them
 * overflows (|h| from 1.8e19 on), y is 0 (and the gradient's dx may be NaN), and where it vanishes beside eps = 0,
 * y is not finite. */
int nvfp4_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight, int dtype,
                   int weight_dtype, int64_t rows, int64_t cols, float eps, void *sum_out, void *y,
                   uint8_t *y_scales, int y_dtype, void *stream);

/* Gradient of nvfp4_rms_norm at h, given dy at y and (nullable) dh at h from its other uses:
 *   dx = q * (weight dy) - h q^3 mean(weight dy h) + dh with q = (mean(h^2) + eps)^(-1/2): the gradient at x
 *        and at the residual alike, of `dtype` (bf16 or fp32), as dy and dh;
 *   dweight [cols] fp32 = the sum over rows of dy h q.
 * h is of `dtype` (h_dtype equal to it, h_scales NULL) or MXFP8 (a checkpoint of it). Scratch:
 * nvfp4_rms_norm_grad_workspace_bytes. */
int nvfp4_rms_norm_grad(const void *dy, int64_t lddy, const void *h, int64_t ldh, const uint8_t *h_scales,
                        int h_dtype, const void *weight, const void *dh, int64_t lddh, int dtype,
                        int weight_dtype, int64_t rows, int64_t cols, float eps, void *dx, float *dweight,
                        void *workspace, size_t workspace_bytes, void *stream);
size_t nvfp4_rms_norm_grad_workspace_bytes(int64_t rows, int64_t cols);

/* What a product applies to z: nothing; silu(z) = z / (1 + e^-z); gelu(z) = z / (1 + e^-v) with v = 2 sqrt(2/pi) (z +
 * 0.044715 z^3), the tanh form. */
enum nvfp4_activation { NVFP4_ACT_NONE = 0, NVFP4_ACT_SILU = 1, NVFP4_ACT_GELU = 2 };

/* The product of nvfp4_matmul with the rest of a layer's projection in its epilogue:
 *   z [M][N] = alpha * (x Wq^T) + bias, Wq = e2m1(code) * e4m3(scale) of the weights [N][K] (scale bytes 0x00 .. 0x7E,
 *   as the quantiser writes them);
 *   y [M][N] = act(z) + residual, or, gated (with an activation, N even, F = N / 2),
 *   y [M][F] = act(z[:, :F]) * z[:, F:] + residual: rows 0 .. F-1 of the weights are the gate.
 * x is bf16 or MXFP8 [M][K]; bias [N] and residual (as y) bf16 or fp32, NULL for none; y bf16 or fp32; z, kept
 * for the gradient, bf16 or MXFP8 (z_scales), NULL if not (gated and MXFP8: F % 32 == 0). K % 16 == 0; K, N
 * <= 2^21, ldx < 2^23 (else NVFP4_ERR_SHAPE). codes 8-byte aligned. residual may be y itself (contiguous, of y's type).
 * Arithmetic: as nvfp4_matmul (exact products, fp32 sums), then fp32 and one rounding per output. Values of
 * an MXFP8 x below 2^-126 may count as zero. */
typedef struct nvfp4_linear_args {
    const void *x;
    int64_t ldx;
    const uint8_t *x_scales; /* MXFP8 x alone, else NULL */
    int x_dtype;             /* NVFP4_DTYPE_BF16 or _MXFP8 */
    int64_t M, K, N;
    const uint8_t *codes;
    const uint8_t *scales;
    const float *alpha;
    const void *bias;
    int bias_dtype;
    int activation; /* enum nvfp4_activation */
    int gated;      /* 0 or 1 */
    const void *residual;
    int64_t ldr;
    int residual_dtype;
    void *y;
    int y_dtype;
    void *z;
    uint8_t *z_scales; /* MXFP8 z alone, else NULL */
    int z_dtype;       /* NVFP4_DTYPE_BF16 or _MXFP8 */
    void *workspace;   /* nvfp4_linear_workspace_bytes */
    size_t workspace_bytes;
    void *stream;
} nvfp4_linear_args_t;

int nvfp4_linear(const nvfp4_linear_args_t *args);

/* Scratch of one nvfp4_linear call (x rearranged for 9 to 64 rows; fp32 sums where K is split over work-groups;
 * an MXFP8 x decoded beyond; the decoded weights for many rows; 0 for up to 8 rows unless z is MXFP8). z_dtype: the form
 * in which z is kept, NVFP4_DTYPE_BF16 also where it is not. */
size_t nvfp4_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, int x_dtype, int gated, int z_dtype);

/* Gradient of nvfp4_linear, given dy (bf16, as y) at y; the residual's gradient is dy itself, the weights are
 * frozen:
 *   dz [M][N] bf16 = dy act'(z), or gated (dy * up * act'(gate), dy * act(gate)) for z = (gate, up);
 *   dx [M][K] bf16 = alpha * (dz Wq), of dz as rounded (the products are exact, the sums fp32);
 *   dbias [N] fp32 = the sum over rows of dz unrounded (NULL: not formed).
 * act' of a NaN or an infinity in z is NaN. z is what nvfp4_linear kept, bf16 or MXFP8 (contiguous scales).
 * activation = none: z and dz are NULL and dz = dy. lddy < 2^23. Scratch: nvfp4_linear_grad_workspace_bytes (the weights
 * decoded where that is the faster way, the bias's partial sums, fp32 sums where N is split over work-groups). */
typedef struct nvfp4_linear_grad_args {
    const void *dy;
    int64_t lddy;
    const void *z;
    int64_t ldz;
    const uint8_t *z_scales; /* MXFP8 z alone, else NULL */
    int z_dtype;
    int64_t M, K, N;
    const uint8_t *codes;
    const uint8_t *scales;
    const float *alpha;
    int activation;
    int gated;
    void *dx;
    void *dz;
    float *dbias;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
} nvfp4_linear_grad_args_t;

int nvfp4_linear_grad(const nvfp4_linear_grad_args_t *args);
size_t nvfp4_linear_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int gated, int with_dbias);

/* ------------------------------------------------------- rotary positions, a cache in 8 bits, attention
 *
 * What a decoder layer computes between its products. Errors, streams, scratch and alignment as for the layer
 * operators above; tokens <= 2^23, heads <= 65535. */

/* Rotary positions: for each token t and head, with (a, b) = (x[j], x[j + R/2]), j < R/2,
 *   y[j] = a cos w - b sin w, y[j + R/2] = b cos w + a sin w, w = positions[axis(j)][t] * base^(-2j/R);
 * columns from R on are copied. R = 2 * (sections[0] + ... + sections[axes - 1]) <= dim, and axis(j) is the one in whose
 * section j lies (sections of consecutive pairs, 1 <= axes <= 4). inverse = 1 turns back (w negated): the gradient of
 * the call with inverse = 0, and the other way round. x and y are bf16 or fp32 (`dtype`) with `xs`, `ys` elements from
 * token to token and `xh`, `yh` from head to head (not looked at for one token or head); y may be x itself with the same
 * strides, and may not overlap it otherwise. positions: int32 or, with positions64 = 1, int64, `tokens` per axis. Angles
 * are binary64, sines and cosines binary32, y is rounded once. dim <= 256, base > 0 and finite. */
typedef struct nvfp4_rotary_args {
    const void *x;
    int64_t xs, xh;
    void *y;
    int64_t ys, yh;
    int dtype;
    int64_t tokens;
    int heads, dim;
    const void *positions;
    int positions64;
    int axes;
    int sections[4];
    double base;
    int inverse;
    void *stream;
} nvfp4_rotary_args_t;

int nvfp4_rotary(const nvfp4_rotary_args_t *args);

/* A paged cache of keys and values in 8 bits: `pages` pages of 64 tokens for each of kv_heads heads, dim columns (dim % 16
 * == 0, dim <= 256).
 *   k_codes  [pages][kv_heads][64][dim]   E4M3
 *   v_codes  [pages][kv_heads][dim][64]   E4M3, the tokens of a column side by side
 *   k_scales, v_scales [pages][kv_heads]  E8M0 (as MXFP8): one power of two per page and head
 * Token t of sequence s is slot t % 64 of page table[s][t / 64] (table: int32, `ldt` elements from sequence to
 * sequence, `width` blocks each). lengths [seqs]: tokens of each sequence, those of the call among them. starts
 * [seqs + 1]: the rows starts[s] .. starts[s + 1] - 1 of the call's operands are the last tokens of sequence s; NULL: row
 * s is the one new token of sequence s (tokens == seqs). Rows in front of starts[0] and behind starts[seqs] are of no
 * sequence: not read, and their outputs not written. Codes and outputs 16-byte aligned.
 * lengths, starts and table are device data and not checked on the host. A page outside the cache holds nothing: its
 * tokens are not written and not attended to; a length beyond 64 * width counts as that. The pages that a call
 * writes to must be of one sequence only, once; pages that are only read may be shared.
 *
 * Writing: per block of 64 tokens and head, for keys and values apart, the scale is the smallest power of two (2^-127 at
 * least) with max|x| <= 448 * scale over the block's new tokens, and not below the scale it has where it holds
 * earlier tokens of the sequence (slots in front of the new ones): their codes are then rounded to the new scale, which is
 * exact for codes that stay at or above 2^-6 in magnitude. Codes are the nearest, ties to even. Slots behind the
 * sequence's end stay as they are. A NaN or an infinity in a block, or a magnitude from 248 * 2^120 on (whose nearest code is
 * worth 2^128), gives scale byte 255 and codes 0x7F: all its tokens read as NaN, until a sequence begins in the block anew. */
typedef struct nvfp4_kv_cache {
    uint8_t *k_codes, *v_codes;
    uint8_t *k_scales, *v_scales;
    int64_t pages;
    int kv_heads, dim;
} nvfp4_kv_cache_t;

typedef struct nvfp4_sequences {
    const int32_t *table;
    int64_t ldt;
    const int32_t *lengths;
    const int32_t *starts; /* nullable */
    int seqs, width;
} nvfp4_sequences_t;

/* k, v: [tokens][kv_heads][dim] bf16 or fp32 with their strides (unit columns). */
int nvfp4_kv_append(const nvfp4_kv_cache_t *cache, const nvfp4_sequences_t *seqs, const void *k, int64_t k_token,
                    int64_t k_head, const void *v, int64_t v_token, int64_t v_head, int dtype, int64_t tokens,
                    void *stream);

/* Attention of q [tokens][heads][dim] (bf16, its strides; heads a multiple of kv_heads, head i on key/value head i /
 * (heads / kv_heads)) over the cache: out [tokens][heads][dim] bf16, contiguous (it may be q itself, and may not overlap it
 * otherwise),
 *   out = sum_t softmax_t(scale * q . k_t) v_t
 * over the tokens t that a row sees: with causal = 1 row i of a sequence's n rows sees its first length - n + i + 1
 * tokens, with causal = 0 all `length`. A row that sees none gives zeros; one that sees a token of a block with scale byte
 * 255, or any token where its q holds a NaN or an infinity, gives NaN. Products with q are exact, sums fp32, probabilities
 * are rounded to bf16 before they are multiplied with the values. Values of the cache below 2^-126 may count as zero, and
 * sums are held of up to 2^8 times the values: length * |v| has to stay below 2^119.
 * 1e-30 < |scale| < 1e30, and scale * q . k has to stay below 2^126 in magnitude (it is held in fp32);
 * tokens * (heads / kv_heads)^2 < 2^32. Scratch: nvfp4_attention_workspace_bytes. */
int nvfp4_attention(const nvfp4_kv_cache_t *cache, const nvfp4_sequences_t *seqs, const void *q, int64_t q_token,
                    int64_t q_head, int heads, int64_t tokens, float scale, int causal, void *out, void *workspace,
                    size_t workspace_bytes, void *stream);
size_t nvfp4_attention_workspace_bytes(int64_t tokens, int seqs, int width, int heads, int kv_heads, int dim);

/* A layer of experts with NVFP4 weights for a few tokens, whole: for token t with logits l[t][0 .. experts - 1]
 *   its top_k largest logits choose experts, equal ones by the lower index; an expert of logit -inf is never chosen,
 *   so a token may have fewer, or none (then y = residual, or zeros);
 *   w = softmax(l) over all experts, or the logistic function of l (NVFP4_SCORE_SIGMOID), of the chosen; with
 *   normalize = 1 divided by their sum over the chosen;
 *   h = act(z), z = alpha1_e (x Wq1_e^T), or, gated, act(z[:inner]) * z[inner:], rounded to bf16;
 *   y = residual + sum over the chosen of w alpha2_e (h Wq2_e^T), fp32 sums, rounded once to bf16.
 * A NaN among a token's logits is chosen first and makes NaN of its y. x [tokens][width] bf16; logits [tokens][experts] bf16
 * or fp32 with `ldl`; up: the experts' [inner, or gated 2 inner][width] weights one after the other, as the quantiser writes
 * them (codes, scales, and one alpha per expert); down: [width][inner]; residual (nullable) as y, with `ldr`, may be y
 * itself (contiguous) and may not overlap it otherwise. width, inner % 16 == 0 and <= 2^21, experts <= 512, top_k <=
 * min(32, experts), tokens * top_k <= 8192, ldx, ldl, ldr < 2^31, an expert's weights below 2^31 values (else
 * NVFP4_ERR_SHAPE). Codes 8-byte aligned. No expert's weights are read that no token chose. Scratch: nvfp4_moe_workspace_bytes. */
enum nvfp4_scoring { NVFP4_SCORE_SOFTMAX = 0, NVFP4_SCORE_SIGMOID = 1 };
typedef struct nvfp4_moe_args {
    const void *x;
    int64_t ldx;
    const void *logits;
    int64_t ldl;
    int logits_dtype; /* NVFP4_DTYPE_BF16 or _F32 */
    int64_t tokens, width, inner;
    int experts, top_k;
    const uint8_t *up_codes, *up_scales;
    const float *up_alpha;
    const uint8_t *down_codes, *down_scales;
    const float *down_alpha;
    int activation; /* enum nvfp4_activation */
    int gated;
    int scoring; /* enum nvfp4_scoring */
    int normalize;
    const void *residual;
    int64_t ldr;
    void *y;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
} nvfp4_moe_args_t;

int nvfp4_moe(const nvfp4_moe_args_t *args);
size_t nvfp4_moe_workspace_bytes(int64_t tokens, int64_t width, int64_t inner, int experts, int top_k);

/* Text of an nvfp4_error value. */
const char *nvfp4_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif
