/*
 * fp8q_ffn.h -- C ABI of libfp8q, second part: the operators of a
 * transformer's feed-forward block between the quantizers and GEMMs of fp8q.h.
 *
 *   fp8q_rmsnorm_quantize    residual addition, root-mean-square norm, codes
 *   fp8q_rmsnorm_backward    its backward pass
 *   fp8q_gemm_gated          gate and up projections, activation, product,
 *                            codes, in one kernel
 *   fp8q_gated_backward      its elementwise backward pass, as codes for the
 *                            data and weight gradient GEMMs
 *
 * One feed-forward block, forward:
 *   codes y  = fp8q_rmsnorm_quantize(x, residual)            keeps h, rstd
 *   codes H  = fp8q_gemm_gated(y, [Wg; Wu])                  keeps G | U
 *   out      = fp8_gemm_blockwise(H, Wd)
 * and backward from dOut (quantized in both directions by
 * fp8_quantize_blockwise_transpose):
 *   dH       = fp8_gemm_blockwise(dOut, Wd^T)
 *   codes    = fp8q_gated_backward(G | U, dH)
 *   dWd      = fp8_gemm_blockwise_ex(dOut^T, H^T, b_block_rows 1)
 *   dy       = fp8_gemm_blockwise(dG | dU, [Wg; Wu]^T)
 *   d[Wg;Wu] = fp8_gemm_blockwise_ex((dG | dU)^T, y^T, b_block_rows 1)
 *   dx, dw   = fp8q_rmsnorm_backward(dy, h, rstd)
 * Both weight gradients sum over the tokens in blocks of 128; for another number
 * of tokens dOut and y are padded with zero rows before they are transposed, as
 * fp8q_gated_backward pads its transposed codes.
 *
 * Conventions (device pointers, asynchronous calls on `stream`, contiguous
 * row-major tensors, 16-byte alignment of tensors and 4-byte alignment of
 * scales, argument checks before any launch, status codes), formats and scales
 * are those of fp8q.h: a scale is the multiplier s = MAX / max(amax, 1e-12f) of
 * its 1x128 block, the code fp8_rne_satfinite(fp32(v * s)).  Codes are formed
 * from fp32 values; NaN elements do not count toward an amax and become NaN
 * codes.  An output must not overlap an input or another output, except where
 * a call says so (FP8_ERR_ARG).  The first call of each function on a device
 * loads its kernels and sets them up: make it outside a stream capture.
 */
#ifndef FP8Q_FFN_H
#define FP8Q_FFN_H

#include <stdint.h>

#include "fp8q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the gated product. */
enum fp8q_act {
    FP8Q_ACT_SILU = 0,     /* g * sigmoid(g) */
    FP8Q_ACT_GELU_TANH = 1 /* 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
};

/*
 * Residual addition, root-mean-square norm and 1x128 quantization of a row in
 * one pass:
 *   h    = RN_dtype(x + residual), or x without a residual
 *   rstd = 1 / sqrt(mean(h^2) + eps)
 *   y    = (h * rstd) * weight                    (fp32)
 *   q, scales = 1x128 codes of y
 * The norm is taken of h as it is stored.  Sums are fp32: rows whose squares
 * overflow fp32 get rstd = 0.  An infinite element makes its row's rstd 0 and
 * its own y NaN.
 *
 *   x, residual  [rows, cols] of dtype (FP8_F32 or FP8_BF16); residual may be
 *                NULL
 *   weight       [cols] of w_dtype
 *   eps          > 0 and finite
 *   q, scales    [rows, cols] codes of fmt, [rows, ceil(cols / 128)] fp32
 *   h            [rows, cols] of dtype; required with a residual, not written
 *                without one.  May be x or residual (in place).
 *   y            [rows, cols] of dtype, RN_dtype(y), or NULL
 *   rstd         [rows] fp32, or NULL.  Not written for cols == 0, as nothing is:
 *                the mean of no elements has no value
 * Any cols.  Rows of whole 16-byte vectors, up to 16384 bf16 or 8192 fp32
 * elements, stay in registers; others take a slower kernel with the same
 * definition.  The sums' order depends on cols and dtype only: a row's results
 * repeat bit for bit, whatever the tensors' alignment and the other rows.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN (x, residual, weight, q,
 * h, y: 16 bytes; scales, rstd: 4), FP8_ERR_FORMAT, FP8_ERR_DTYPE, FP8_ERR_ARG
 * (eps; overlapping tensors), FP8_ERR_CUDA.
 */
int fp8q_rmsnorm_quantize(const void *x, int dtype, const void *residual, const void *weight, int w_dtype, int64_t rows,
                          int64_t cols, float eps, int fmt, uint8_t *q, float *scales, void *h, void *y, float *rstd,
                          void *stream);

/*
 * The backward pass of that norm (of y, before its quantization), with
 * n = h * rstd, a = dy * weight, c = sum(a * n) / cols:
 *   dx      = rstd * (a - n * c) + dh     the gradient of x and of residual
 *   dweight = sum over rows of dy * n
 *
 *   dy, h       [rows, cols] of dtype
 *   rstd        [rows] fp32, from the forward call
 *   weight      [cols] of w_dtype
 *   dh          [rows, cols] of dtype: the gradient that reaches h by the
 *               residual stream, or NULL
 *   dx          [rows, cols] of dtype; may be dy or dh (in place)
 *   dweight     [cols] fp32, or NULL (a frozen weight); zeros for rows == 0
 *   workspace   at least fp8q_rmsnorm_backward_workspace(rows, cols) bytes of
 *               device memory, 16-byte aligned, of any content; needed with
 *               dweight (few rows need none: 0 bytes, and it may be NULL).
 *               Calls that share it must not overlap on the device.
 * Any cols.  Rows of whole 16-byte vectors, up to 8192 elements, stay in
 * registers (93 to 97 % of the copy rate).  Other widths up to 8192 are read
 * element by element, at about 30 %; wider rows, of any width, are read twice, at
 * 20 to 36 %.
 * The sums' order depends on the shape and the device only: results repeat
 * bit for bit.
 * Errors: as above, with FP8_ERR_ARG also for a workspace that is too small.
 */
int fp8q_rmsnorm_backward(const void *dy, const void *h, int dtype, const float *rstd, const void *weight, int w_dtype,
                          const void *dh, int64_t rows, int64_t cols, void *dx, float *dweight, void *workspace,
                          int64_t workspace_bytes, void *stream);

/* Bytes of workspace for the current device, or FP8_ERR_SHAPE. */
int64_t fp8q_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * Gate and up projections of a gated feed-forward block, its activation and
 * the product, in one kernel on the tensor cores:
 *   [G | U] = A B^T, with the block scales applied as in fp8_gemm_blockwise
 *   H = act(G) * U                                 (fp32)
 *   q, scales = 1x128 codes of H
 *
 *   a, a_fmt, sa  [M, K] codes with 1x128 scales [M, K/128]
 *   b, b_fmt, sb  [2F, K] codes, the F gate rows first, then the F up rows, with
 *                 128x128 scales [2F/128, K/128]
 *   q, scales     [M, F] codes of fmt and [M, F/128] scales; both NULL to get
 *                 only gu
 *   gu, gu_dtype  [M, 2F] G | U rounded to gu_dtype, or NULL.  H is formed from
 *                 the unrounded sums.
 * F % 128 == 0 and K % 128 == 0 (else FP8_ERR_SHAPE); any M.  K == 0 gives the
 * result of empty sums.  M, F, K < 2^30.  Few tokens (M <= 64, or so few that
 * the tokens' and columns' tiles leave half the SMs free) take a kernel that
 * splits K over a cluster of CTAs; its sums are joined in a fixed order, so
 * results repeat bit for bit in either kernel.  For K < 512 a token's results are
 * the same whatever the number of tokens; beyond, the order of its sums over K
 * depends on it.
 * Errors: FP8_ERR_NULL (no output at all; q without scales), FP8_ERR_SHAPE,
 * FP8_ERR_ALIGN (a, b, q, gu: 16 bytes; scales: 4), FP8_ERR_FORMAT,
 * FP8_ERR_DTYPE, FP8_ERR_ARG (unknown act; overlapping tensors), FP8_ERR_CUDA.
 */
int fp8q_gemm_gated(const uint8_t *a, const float *sa, int a_fmt, const uint8_t *b, const float *sb, int b_fmt,
                    int64_t M, int64_t F, int64_t K, int act, int fmt, uint8_t *q, float *scales, void *gu,
                    int gu_dtype, void *stream);

/*
 * The backward pass of H = act(G) * U, quantized for the GEMMs that follow:
 *   dG = dH * U * act'(G),  dU = dH * act(G),  H = act(G) * U    (fp32)
 *
 *   gu, dh        [M, 2F] G | U and [M, F] dH, of dtype
 *   q, scales     1x128 codes of [dG | dU]: [M, 2F] and [M, 2F/128].  A of the
 *                 data gradient [dG | dU] [Wg; Wu].
 *   qt, scales_t  1x128 codes of [dG | dU]^T: [2F, Mt] and [2F, Mt/128], or
 *                 both NULL.  A of the weight gradient.
 *   ht, ht_scales 1x128 codes of H^T: [F, Mt] and [F, Mt/128], or both NULL.
 *                 B (1x128) of the down projection's weight gradient.
 * Mt = ceil(M / 128) * 128: tokens from M on get zero codes and do not count
 * toward an amax, so the GEMMs over the tokens (K = Mt) add nothing for them.
 * F % 128 == 0 (else FP8_ERR_SHAPE), any M.
 * Errors: FP8_ERR_NULL (also one of a pair without the other), FP8_ERR_SHAPE,
 * FP8_ERR_ALIGN (gu, dh, q, qt, ht: 16 bytes; scales: 4), FP8_ERR_FORMAT,
 * FP8_ERR_DTYPE, FP8_ERR_ARG (unknown act; overlapping tensors), FP8_ERR_CUDA.
 */
int fp8q_gated_backward(const void *gu, const void *dh, int dtype, int64_t M, int64_t F, int act, int fmt, uint8_t *q,
                        float *scales, uint8_t *qt, float *scales_t, uint8_t *ht, float *ht_scales, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_FFN_H */
