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
 * and of its routed form, a block of experts:
 *   fp8q_moe_sort            (token, expert) pairs sorted by expert
 *   fp8q_moe_dispatch, fp8q_moe_dispatch_codes
 *                            tokens to the rows of their experts, as codes
 *   fp8q_moe_combine, fp8q_moe_combine_backward
 *                            the rows back to their tokens, with the router's
 *                            weights, and the gradients
 *   fp8q_gemm_gated_grouped, fp8q_gemm_grouped, fp8q_gemm_grouped_wgrad
 *                            the experts' products
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

/*
 * ---- A block of experts ---------------------------------------------------
 *
 * The router gives every token top_k experts and their weights; expert e works
 * on the tokens that chose it, which are laid out as rows, one expert's after
 * another's.  The layout is the sort's:
 *   offsets [num_experts + 1]  expert e has rows offsets[e] .. offsets[e+1] - 1
 *   pos [tokens, top_k]        the row of a pair, or -1 (the pair has none)
 *   src [rows]                 the pair t * top_k + k of a row, or -1 (no pair)
 * all int32, on the device: no call needs to know on the host how many rows an
 * expert has.  `rows` is the number of rows that tensors have room for; those
 * from offsets[num_experts] on are not read as results nor written.  (The two
 * calls that read rows by pos, fp8q_moe_combine and the weights' gradient of
 * fp8q_moe_combine_backward, hold pos to 0 .. rows - 1 instead.)
 *
 * Pairs may be dropped after the sort by setting their pos to -1: their rows are
 * then rows without a pair in every call, zeros among the rows that are written.
 * src stays as the sort made it; no two pairs share a row.
 *
 * Forward:
 *   route    = fp8q_moe_sort(experts)
 *   codes X  = fp8q_moe_dispatch(y) or fp8q_moe_dispatch_codes(codes of y)
 *   codes H  = fp8q_gemm_gated_grouped(X, [Wg; Wu] of every expert)  keeps G | U
 *   rows     = fp8q_gemm_grouped(H, Wd of every expert)
 *   out      = fp8q_moe_combine(rows, weights, residual)
 * and backward (align 128, so that the blocks of 128 rows over which the
 * weights' gradients are scaled are one expert's):
 *   codes dR, dweights = fp8q_moe_combine_backward(dOut, rows, weights)
 *   dH       = fp8q_gemm_grouped(dR, Wd^T)
 *   codes    = fp8q_gated_backward(G | U, dH)          on the rows, as it is
 *   dWd      = fp8q_gemm_grouped_wgrad(dR^T, H^T)
 *   dX       = fp8q_gemm_grouped(dG | dU, [Wg; Wu]^T)
 *   d[Wg;Wu] = fp8q_gemm_grouped_wgrad((dG | dU)^T, X^T)
 *   dy       = fp8q_moe_combine(dX) without weights
 *
 * num_experts 1 .. 1024, tokens * top_k <= 2^30.  Indices that no sort makes
 * (outside their range) are taken as -1; offsets are held inside 0 .. rows.
 */

/*
 * Sort of the pairs by expert, stable: an expert's rows come in the order of
 * the pairs t * top_k + k.  Expert e gets counts[e] rows, and its first one at a
 * multiple of align; the rows up to the next expert have no pair.
 *
 *   experts     [tokens, top_k] int32; an id outside 0 .. num_experts - 1 gives
 *               the pair no row.  A token may name an expert twice.
 *   align       a power of two, 1 .. 128: 1 packs the rows, 128 is what the
 *               transposed codes and the weights' gradients need
 *   rows        of src, at least fp8q_moe_rows(...), which holds any routing
 *               (else FP8_ERR_SHAPE)
 *   offsets, pos, src   as above; every element is written
 *   counts      [num_experts] int32: the pairs of each expert, or NULL
 *   workspace   at least fp8q_moe_sort_workspace(...) bytes of device memory,
 *               16-byte aligned, of any content; up to 4096 pairs need none (0
 *               bytes, it may be NULL).  Calls that share it must not overlap on
 *               the device.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN (workspace: 16 bytes; the
 * others: 4), FP8_ERR_ARG (align; a workspace that is too small; overlapping
 * tensors), FP8_ERR_CUDA.
 */
int fp8q_moe_sort(const int32_t *experts, int64_t tokens, int64_t top_k, int num_experts, int align, int64_t rows,
                  int32_t *offsets, int32_t *pos, int32_t *src, int32_t *counts, void *workspace,
                  int64_t workspace_bytes, void *stream);

/* Rows that hold any routing of tokens * top_k pairs (a multiple of align), or
 * FP8_ERR_SHAPE, FP8_ERR_ARG. */
int64_t fp8q_moe_rows(int64_t tokens, int64_t top_k, int num_experts, int align);

/* Bytes of workspace, or FP8_ERR_SHAPE. */
int64_t fp8q_moe_sort_workspace(int64_t tokens, int64_t top_k, int num_experts);

/*
 * Tokens to their rows, quantized: row r is token src[r] / top_k of x as 1x128
 * codes, zeros (with the scale of a zero block) where src[r] is -1 or the pos of
 * its pair is not r.
 *
 *   x            [tokens, cols] of dtype
 *   q, scales    [rows, cols] codes of fmt and [rows, cols / 128] scales
 *   qt, scales_t the same rows transposed, as 1x128 codes of their own:
 *                [cols, rows] and [cols, rows / 128], or both NULL.  rows is then a
 *                multiple of 128.  Blocks of 128 rows from offsets[num_experts] on
 *                are not written; rows from there on count as zeros in the block
 *                that they share.
 * cols % 128 == 0 (else FP8_ERR_SHAPE).  Its gradient is fp8q_moe_combine of the
 * rows' gradient, without weights.
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN (x, q, qt: 16 bytes; the
 * others: 4), FP8_ERR_FORMAT, FP8_ERR_DTYPE, FP8_ERR_ARG (overlapping tensors),
 * FP8_ERR_CUDA.
 */
int fp8q_moe_dispatch(const void *x, int dtype, int64_t cols, const int32_t *offsets, int num_experts,
                      const int32_t *pos, const int32_t *src, int64_t tokens, int64_t top_k, int64_t rows, int fmt,
                      uint8_t *q, float *scales, uint8_t *qt, float *scales_t, void *stream);

/*
 * The same of tokens that are codes already (fp8q_rmsnorm_quantize's): xq
 * [tokens, cols] of fmt and xs [tokens, cols / 128] are copied to the rows.
 */
int fp8q_moe_dispatch_codes(const uint8_t *xq, const float *xs, int fmt, int64_t cols, const int32_t *offsets,
                            int num_experts, const int32_t *pos, const int32_t *src, int64_t tokens, int64_t top_k,
                            int64_t rows, uint8_t *q, float *scales, void *stream);

/*
 * Rows back to their tokens:
 *   y[t] = RN_dtype(residual[t] + sum over k of weights[t][k] * x[pos[t][k]])
 * in fp32, k ascending; pairs without a row add nothing, whatever their weight.
 *
 *   x            [rows, cols] of dtype
 *   pos, weights [tokens, top_k]; weights fp32, or NULL for ones
 *   residual, y  [tokens, cols] of dtype; residual may be NULL
 * cols % 128 == 0 (else FP8_ERR_SHAPE).  Errors as for fp8q_moe_dispatch.
 */
int fp8q_moe_combine(const void *x, int dtype, int64_t rows, int64_t cols, const int32_t *pos, const float *weights,
                     const void *residual, int64_t tokens, int64_t top_k, void *y, void *stream);

/*
 * Its backward pass (the residual's gradient is dy):
 *   row r of token t, pair (t, k):  weights[t][k] * dy[t]  (fp32) as codes, zeros
 *                                   on rows without a pair
 *   dweights[t][k] = <dy[t], x[pos[t][k]]>  (fp32), 0 for pairs without a row
 *
 *   dy, x        [tokens, cols] and [rows, cols] of dtype; x may be NULL without
 *                dweights
 *   q, scales, qt, scales_t   as fp8q_moe_dispatch writes them; q and scales may
 *                be NULL (then qt and scales_t are), and weights with them
 *   dweights     [tokens, top_k] fp32, or NULL
 * dweights' sums are taken in an order that depends on cols and dtype only.
 * Errors as for fp8q_moe_dispatch.
 */
int fp8q_moe_combine_backward(const void *dy, const void *x, int dtype, int64_t cols, const int32_t *offsets,
                              int num_experts, const int32_t *pos, const int32_t *src, int64_t tokens, int64_t top_k,
                              int64_t rows, const float *weights, int fmt, uint8_t *q, float *scales, uint8_t *qt,
                              float *scales_t, float *dweights, void *stream);

/*
 * Every expert's product, rows offsets[e] .. offsets[e+1] - 1 of A with weights e:
 *   c[m] = A[m] B[e]^T, with the block scales applied as in fp8_gemm_blockwise
 *
 *   a, a_fmt, sa  [rows, K] codes with 1x128 scales [rows, K/128]
 *   b, b_fmt, sb  [num_experts, N, K] codes with 128x128 scales
 *                 [num_experts, N/128, K/128]
 *   c, c_dtype    [rows, N]
 * N % 128 == 0 and K % 128 == 0 (else FP8_ERR_SHAPE), num_experts * N < 2^31; any
 * offsets, aligned or not.  K == 0 gives empty sums.  Few rows an expert (up to 24
 * on average of rows / min(num_experts, rows), or no more tiles of 32 rows x 256
 * columns than the device has SMs) take a kernel that splits K over a cluster of
 * CTAs and joins its sums in a fixed order: results repeat bit for bit in either
 * kernel.  For K < 512 a row's results do not depend on the other rows; beyond, the
 * order of its sums over K depends on rows, num_experts and N.  Both choices go by
 * rows, the room, because the host does not know the rows in use: where most of the
 * room stays empty, tensors cut to size can be faster (32 experts of 4096 x 4096
 * gated, 498 rows: 111 us with room for 4096, 90 without).
 * Errors: FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN (a, b, c: 16 bytes; the
 * others: 4), FP8_ERR_FORMAT, FP8_ERR_DTYPE, FP8_ERR_ARG (overlapping tensors),
 * FP8_ERR_CUDA.
 */
int fp8q_gemm_grouped(const uint8_t *a, const float *sa, int a_fmt, const uint8_t *b, const float *sb, int b_fmt,
                      const int32_t *offsets, int num_experts, int64_t rows, int64_t N, int64_t K, void *c,
                      int c_dtype, void *stream);

/*
 * The same with the gated product of fp8q_gemm_gated: b [num_experts, 2F, K],
 * each expert's F gate rows first, sb [num_experts, 2F/128, K/128];
 *   [G | U] = A[m] B[e]^T,  H = act(G) * U,  q, scales = 1x128 codes of H
 *   q, scales     [rows, F] codes of fmt and [rows, F/128] scales; both NULL to get
 *                 only gu
 *   gu, gu_dtype  [rows, 2F] G | U rounded to gu_dtype, or NULL
 * F % 128 == 0 and K % 128 == 0.  Errors as above, and FP8_ERR_ARG for an unknown
 * act.
 */
int fp8q_gemm_gated_grouped(const uint8_t *a, const float *sa, int a_fmt, const uint8_t *b, const float *sb, int b_fmt,
                            const int32_t *offsets, int num_experts, int64_t rows, int64_t F, int64_t K, int act,
                            int fmt, uint8_t *q, float *scales, void *gu, int gu_dtype, void *stream);

/*
 * The gradient of every expert's weights, a product over its rows:
 *   dw[e] = A^T[:, rows of e] (B^T[:, rows of e])^T
 * with the scales applied as fp8_gemm_blockwise_ex does with b_block_rows 1.
 *
 *   at, a_fmt, sat  [N, rows] codes with 1x128 scales [N, rows/128]
 *   bt, b_fmt, sbt  [K, rows] codes with 1x128 scales [K, rows/128]
 *   offsets         multiples of 128 (a sort with align 128); others are rounded
 *                   down to one
 *   dw, dw_dtype    [num_experts, N, K]; zeros for an expert without rows
 * N, K and rows multiples of 128 (else FP8_ERR_SHAPE).  Errors as for
 * fp8q_gemm_grouped.
 */
int fp8q_gemm_grouped_wgrad(const uint8_t *at, const float *sat, int a_fmt, const uint8_t *bt, const float *sbt,
                            int b_fmt, const int32_t *offsets, int num_experts, int64_t rows, int64_t N, int64_t K,
                            void *dw, int dw_dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_FFN_H */
