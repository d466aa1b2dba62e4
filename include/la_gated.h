/*
 * la_gated.h -- C ABI of the gated linear recurrence (GB300, sm_103a): scan over sequences,
 * its gradients, and the speculative-decoding trio (decode, verify, commit).
 *
 * Where la_prefill.h's recurrence decays a matrix state by a fixed lambda per head, this one
 * decays a vector state by a lambda that each token chooses per channel.  For every sequence n
 * with slot(n) >= 0 and channel c, with sig(z) = 1 / (1 + exp(-z)):
 *
 *     u_t    = slopes[c] sig(r_t)         lambda_t = exp(-u_t)      beta_t = sqrt(1 - lambda_t^2)
 *     h_t    = lambda_t h_{t-1} + beta_t sig(g_t) x_t               h_{-1} = h0[slot(n)][c] (or 0)
 *     o_t    = h_t                                                  h_final[slot(n)][c] = h_{L-1}
 *
 * r holds the decay gates' logits, g the input gates'; slopes >= 0 is expected (negative slopes
 * give unspecified values).  A gate logit of -inf is a closed gate: r = -inf keeps the state
 * unchanged and adds nothing (lambda = 1, beta = 0), g = -inf adds nothing for a finite x.
 * (sig(z) under FP32's smallest normal number, z < -87.3, counts as 0.)
 * A NaN reaches every output that depends on it, and no other sequence, request or channel.
 * States and arithmetic are FP32; o is rounded once.
 *
 * Layouts (innermost dimension contiguous):
 *   x, r, g, o and their gradients   [B*T, C] of `dtype`, each with its own row stride (ld*, in
 *                                    elements, >= C): column ranges of one projection's
 *                                    [B*T, 3 C] output, and of its gradient, are read and
 *                                    written in place
 *   slopes, dslopes                  fp32 [C]
 *   h0, h_final, dh_final, dh0       fp32 [P, C]   nullable
 *   state_indices, cu_seqlens        as in la_prefill.h (nullable; negative index = padded
 *                                    sequence: its rows of the outputs and every state slot are
 *                                    left untouched, its rows of the inputs do not matter)
 * Rows past cu_seqlens[N] (and before cu_seqlens[0]) belong to no sequence and are left as they
 * are.  Pointers need the alignment of their element type only (16-byte rows run faster).
 *
 * Sequences may share a slot that is only read; where states are written (h_final, dh0, decode,
 * commit) a slot that two sequences name is left with an unspecified state.
 *
 * Device-side checks: an index >= pool_size sets LA_DEV_ERR_BAD_INDEX and skips that sequence;
 * cu_seqlens that is not non-decreasing inside [0, T] sets LA_DEV_ERR_BAD_SEQLENS and skips the
 * whole call.  LA_DEV_ERR_TIMEOUT reports that a wait between the blocks of a scan passed its
 * limit (the outputs are then incomplete).
 *
 * Every call enqueues its kernels on `stream`, allocates nothing, never synchronises with the
 * host and may be captured in a CUDA graph.  Results are bitwise repeatable.
 * Outputs may share no element with an input or with another output (LA_ERR_INVALID_ARGUMENT;
 * interleaved column ranges of one buffer share none), except h_final, which may be h0.
 */
#ifndef LA_GATED_H
#define LA_GATED_H

#include <stddef.h>
#include <stdint.h>

#include "la_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the activations (la_gated.h, la_norm.h). */
typedef enum {
  LA_DTYPE_BF16 = 0,
  LA_DTYPE_FP32 = 1
} la_dtype;

/*
 * Bytes of device workspace la_gated_scan_fwd (backward = 0) or la_gated_scan_bwd (backward = 1)
 * needs for these sizes (packed = 1 when cu_seqlens will be given).  Host only; 0 when none.
 */
la_status la_gated_scan_workspace(int B, int T, int N, int C, int packed, la_dtype dtype, int backward,
                                  size_t* bytes);

/*
 * la_gated_scan_fwd -- the recurrence over every sequence.
 *
 * B, T, N, pool_size and the two modes (fixed length, packed) as la_prefill_fwd; C >= 1 channels.
 * workspace: device memory of at least la_gated_scan_workspace(...) bytes, 256-byte aligned, its
 * contents on entry do not matter; calls that share one must not overlap on the GPU.
 */
la_status la_gated_scan_fwd(const void* x, const void* r, const void* g, const float* slopes, const float* h0,
                            const int32_t* state_indices, const int32_t* cu_seqlens, void* o, float* h_final,
                            int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo, int B, int T, int N, int C,
                            int pool_size, la_dtype dtype, void* workspace, size_t workspace_bytes, int* dev_error,
                            void* stream);

/*
 * la_gated_scan_bwd -- gradients of la_gated_scan_fwd for dout = dL/do and dh_final =
 * dL/dh_final (nullable: 0), with G_t = dL/dh_t:
 *
 *     G_t  = dout_t + lambda_{t+1} G_{t+1}    G_{L-1} = dout_{L-1} + dh_final[slot]
 *     dx_t = G_t beta_t sig(g_t)              dg_t = dx_t x_t (1 - sig(g_t))
 *     du_t = G_t (sig(g_t) x_t lambda_t^2 / beta_t - lambda_t h_{t-1})
 *     dr_t = du_t u_t (1 - sig(r_t))          dslopes[c] = sum over all tokens of du_t sig(r_t)
 *     dh0[slot] = lambda_0 G_0                (dh_final[slot] for an empty sequence)
 *
 * o is the forward's output, which holds h_{t-1} for every token but the first (that one's is
 * h0's).  The term lambda^2 / beta is taken as 0 where u_t = 0 (or beta_t^2 is under FP32's smallest
 * normal number).  dslopes sums the sequences that run, in a fixed order, and is written (0) when there
 * are none; rows of padded sequences and unselected slots are not written.  dh0 nullable (not
 * computed).  The gradients' row strides are lddx, lddr, lddg.
 */
la_status la_gated_scan_bwd(const void* x, const void* r, const void* g, const float* slopes, const float* h0,
                            const void* o, const void* dout, const float* dh_final, const int32_t* state_indices,
                            const int32_t* cu_seqlens, void* dx, void* dr, void* dg, float* dslopes, float* dh0,
                            int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo, int64_t lddout, int64_t lddx,
                            int64_t lddr, int64_t lddg, int B, int T, int N, int C, int pool_size, la_dtype dtype,
                            void* workspace, size_t workspace_bytes, int* dev_error, void* stream);

/*
 * Speculative decoding over T >= 1 tokens per request (rows b T .. b T + T - 1), on the pooled
 * states state [P, C] fp32 at each request's slot (state_indices as in la_decode.h):
 *   la_gated_decode  outputs of all T tokens; the states advance over them (in place)
 *   la_gated_verify  the same outputs (bitwise); the states are left untouched
 *   la_gated_commit  the states advance over the first accepted_len[b] tokens (clamped to
 *                    [0, T]; 0 = untouched); no outputs.  With accepted_len == T the states are
 *                    bitwise those la_gated_decode leaves.
 */
la_status la_gated_decode(const void* x, const void* r, const void* g, const float* slopes, float* state,
                          const int32_t* state_indices, void* o, int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo,
                          int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error, void* stream);

la_status la_gated_verify(const void* x, const void* r, const void* g, const float* slopes, const float* state,
                          const int32_t* state_indices, void* o, int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo,
                          int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error, void* stream);

la_status la_gated_commit(const void* x, const void* r, const void* g, const float* slopes, float* state,
                          const int32_t* state_indices, const int32_t* accepted_len, int64_t ldx, int64_t ldr,
                          int64_t ldg, int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_GATED_H */
