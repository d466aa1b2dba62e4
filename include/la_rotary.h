/*
 * la_rotary.h -- C ABI of the norm and position rotation of queries and keys (GB300, sm_103a), the
 * pass in front of a linear-attention (la_prefill.h) or softmax-attention (la_attention.h) layer.
 *
 * For every token t and every query and key head, with x the head's D elements, in FP32:
 *
 *     n   = x / sqrt(mean_d(x[d]^2) + eps),   y = n * weight        (q_weight or k_weight)
 *     out = y with the R/2 pairs of its first R elements rotated: for pair i, by the angle
 *           a = positions[t] * inv_freq[i],
 *               out[lo] = y[lo] cos a - y[hi] sin a
 *               out[hi] = y[lo] sin a + y[hi] cos a
 *           (lo, hi) = (i, i + R/2), or (2i, 2i + 1) with `interleaved`.  Elements from R on are y.
 *
 * The angle is the exact product of the position and the FP32 frequency, taken modulo one turn in
 * 64-bit fixed point before the sine and cosine, so far positions lose no digits.  Frequencies must
 * be finite.
 *
 * Layouts: q, q_out [tokens, H, D], k, k_out [tokens, HK, D] in `dtype`, innermost contiguous, each
 * with a stride between tokens (ld*) and between heads (hs*) in elements, so that column ranges of
 * one projection's output, and head-major tensors, work in place.  Either the heads of a token lie
 * within its stride (hs >= D, ld >= (H - 1) hs + D) or the tokens of a head within the head's.
 * q_weight, k_weight fp32 [D], nullable (ones); positions int32 [tokens]; inv_freq fp32 [R/2]
 * (both nullable when R == 0).  D is 64, 128 or 256; 0 <= R <= D, even; any tokens >= 0.
 * Pointers need the alignment of their element type only (16-byte rows and R a multiple of 16,
 * FP32 8, run faster).  q_out may be q itself and k_out k itself (same pointer and strides);
 * beyond that outputs may share no element with an input or with each other (ranges between a
 * token's first and last head count whole): LA_ERR_INVALID_ARGUMENT.
 *
 * Calls enqueue on `stream`, allocate nothing, never synchronise and may be captured in a CUDA
 * graph.  Results are bitwise repeatable.
 */
#ifndef LA_ROTARY_H
#define LA_ROTARY_H

#include <stddef.h>
#include <stdint.h>

#include "la_gated.h"
#include "la_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

la_status la_qk_norm_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight, float eps,
                              const int32_t* positions, const float* inv_freq, void* q_out, void* k_out, int64_t ldq,
                              int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldqo, int64_t hsqo, int64_t ldko,
                              int64_t hsko, int tokens, int H, int HK, int D, int R, int interleaved, la_dtype dtype,
                              void* stream);

/* Bytes of device workspace la_qk_norm_rope_bwd needs.  Host only. */
la_status la_qk_norm_rope_bwd_workspace(int tokens, int H, int HK, int D, size_t* bytes);

/*
 * la_qk_norm_rope_bwd -- gradients for the forward's inputs q and k, given dq_out and dk_out
 * (gradients of its outputs): with g the gradient rotated back by the same angle,
 *
 *     dx      = rstd (weight g - n mean_d(weight g n)),   rstd = 1 / sqrt(mean_d(x^2) + eps)
 *     dweight = sum over tokens and heads of g n
 *
 * dq, dk have the layouts of q, k and may be dq_out, dk_out themselves.  dq_weight, dk_weight fp32
 * [D], nullable (not computed); they sum in a fixed order and are written (0) when there are no
 * tokens.  workspace: 256-byte aligned, as la_qk_norm_rope_bwd_workspace says.
 */
la_status la_qk_norm_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight, float eps,
                              const int32_t* positions, const float* inv_freq, const void* dq_out, const void* dk_out,
                              void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t ldq, int64_t hsq,
                              int64_t ldk, int64_t hsk, int64_t lddqo, int64_t hsdqo, int64_t lddko, int64_t hsdko,
                              int64_t lddq, int64_t hsdq, int64_t lddk, int64_t hsdk, int tokens, int H, int HK, int D,
                              int R, int interleaved, la_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_ROTARY_H */
