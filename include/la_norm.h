/*
 * la_norm.h -- C ABI of the root-mean-square norm between two mixing layers (GB300, sm_103a):
 * residual addition, norm, optional 8-bit output with scales, and the gradients.
 *
 * For every row t of C columns, in FP32:
 *
 *     s_t = x_t + residual_t              (x_t without a residual)
 *     n_t = s_t / sqrt(mean_c(s_t[c]^2) + eps)
 *     y_t = n_t * weight
 *
 * The row that the next residual addition needs, residual_out = s rounded to `dtype`, is written
 * beside y; the norm is taken of the sum before that rounding.
 *
 * 8-bit output (la_rms_norm_fwd_fp8): y is stored as e4m3 values q with FP32 scales such that
 * y ~ q * scale, one scale per row (group = 0) or per 128 columns (group = 128; the last group
 * of a row may be shorter):
 *     top = max(max|y|, 2^-40),      scale = top / 448,      q = y * (448 / top) rounded to
 *                                            nearest even, clamped to +-448
 * each quotient and product rounded to FP32.  So q is y / scale but for 3 * 2^-24 of it, which
 * decides where y / scale lies that near to the middle between two e4m3 numbers.
 * A NaN in y is stored as NaN and does not enter its group's maximum.
 *
 * Layouts: x, residual, residual_out, y, dy, dres, dx [rows, C], innermost contiguous, each with
 * its row stride in elements (ld*, >= C); weight, dweight fp32 [C]; scales fp32 [rows, groups]
 * contiguous, groups = 1 or ceil(C / 128).  Pointers need the alignment of their element type
 * only (16-byte rows run faster).  1 <= C <= 16384; any rows >= 0.
 * Outputs may share no element with an input or with each other (LA_ERR_INVALID_ARGUMENT), except
 * residual_out, which may be the residual itself (same pointer and stride).
 *
 * dev_error (nullable device int): LA_DEV_ERR_TIMEOUT reports that a copy within a kernel passed
 * its time limit (the outputs are then incomplete).
 * Calls enqueue on `stream`, allocate nothing, never synchronise and may be captured in a CUDA
 * graph.  Results are bitwise repeatable.
 */
#ifndef LA_NORM_H
#define LA_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "la_gated.h"
#include "la_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* residual nullable; residual_out nullable, needs a residual. */
la_status la_rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps, void* y,
                          void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy, int64_t ldres_out, int rows,
                          int C, la_dtype dtype, int* dev_error, void* stream);

/* y is e4m3 [rows, C]; group 0 (a scale per row) or 128. */
la_status la_rms_norm_fwd_fp8(const void* x, const void* residual, const float* weight, float eps, void* y,
                              float* scales, void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy,
                              int64_t ldres_out, int rows, int C, int group, la_dtype dtype, int* dev_error,
                              void* stream);

/* Bytes of device workspace la_rms_norm_bwd needs.  Host only. */
la_status la_rms_norm_bwd_workspace(int rows, int C, size_t* bytes);

/*
 * la_rms_norm_bwd -- gradients of y = n(s) * weight for s (the forward's residual_out, or x
 * without a residual), with rstd = 1 / sqrt(mean(s^2) + eps):
 *
 *     dx      = rstd (weight dy - n mean_c(weight dy n)) + dres     (also dL/dresidual)
 *     dweight = sum over rows of dy n
 *
 * dres (nullable) is the gradient that reaches residual_out from later layers.  dweight sums the
 * rows in a fixed order and is written (0) when there are none.  workspace as in la_gated.h.
 */
la_status la_rms_norm_bwd(const void* s, const float* weight, float eps, const void* dy, const void* dres, void* dx,
                          float* dweight, int64_t lds, int64_t lddy, int64_t lddres, int64_t lddx, int rows, int C,
                          la_dtype dtype, void* workspace, size_t workspace_bytes, int* dev_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_NORM_H */
