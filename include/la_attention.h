/*
 * la_attention.h -- C ABI of softmax attention (GB300, sm_103a) for the layers of a hybrid model
 * that look back at every token, beside its linear-attention layers: whole prompts and their
 * gradients, drafted tokens over a key/value cache, and the writes into that cache.
 *
 * For a query row of head h, with key/value head hk = h / (H / HK) and the keys j that it sees,
 *
 *     p_j = exp(scale q.k_j - lse),   lse = log sum_j exp(scale q.k_j),   o = sum_j p_j v_j
 *
 * Scores, softmax statistics and outputs are held in FP32; the probabilities (and, in the
 * gradients, dS) are rounded to BF16 as operands of the products with v (dO, q and k).  A row that
 * sees no key gives o = 0 (lse = -inf).  scale: finite, any sign, at most 2e38 in size.
 *
 * Layouts: q, o, dout, dq BF16 [tokens, H, D]; k, v, dk, dv BF16 [tokens, HK, D]; innermost
 * contiguous, each with a stride between tokens (ld*) and between heads (hs*) in elements, both
 * multiples of 8, and 16-byte aligned; the heads of a token lie within its stride or the tokens of
 * a head within the head's (as in la_rotary.h).  H % HK == 0; D is 64 or 128.
 *
 * dev_error (nullable device int): LA_DEV_ERR_* bits as in la_prefill.h.
 * Outputs may share no element with an input or with each other (ranges between a token's first
 * and last head count whole): LA_ERR_INVALID_ARGUMENT.  Calls enqueue on `stream`, allocate
 * nothing, never synchronise and may be captured in a CUDA graph.  Results are bitwise repeatable: the
 * same call gives the same bits.  Which parts of a sum la_attn_verify and the dk and dv of
 * la_attn_prefill_bwd join depends on the whole batch's lengths, so there a request's bits may differ
 * beside other requests; la_attn_prefill_fwd and dq give a sequence the same bits in any batch.
 * A workspace is written before it is read: its contents on entry do not matter, and calls that
 * may run at the same time need one each.
 */
#ifndef LA_ATTENTION_H
#define LA_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "la_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * la_attn_prefill_fwd -- causal attention over whole sequences: token t of a sequence sees its
 * tokens 0 .. t.  cu_seqlens int32 [N + 1] (nullable) as in la_prefill.h: without it N == B
 * sequences of T tokens; with it B == 1, T is the number of tokens and sequence n spans
 * [cu_seqlens[n], cu_seqlens[n + 1]).  A sequence whose bounds do not fit is skipped
 * (LA_DEV_ERR_BAD_SEQLENS).  Rows of no sequence are neither written nor let into any result.
 * lse (nullable) fp32 [H, tokens], natural logarithm, as the gradients need it.
 */
la_status la_attn_prefill_fwd(const void* q, const void* k, const void* v, float scale, const int32_t* cu_seqlens,
                              void* o, float* lse, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv,
                              int64_t hsv, int64_t ldo, int64_t hso, int B, int T, int N, int H, int HK, int D,
                              int* dev_error, void* stream);

/* Bytes of device workspace la_attn_prefill_bwd needs for B * T tokens.  Host only. */
la_status la_attn_prefill_bwd_workspace(int B, int T, int H, int HK, int D, size_t* bytes);

/*
 * la_attn_prefill_bwd -- gradients of la_attn_prefill_fwd for q, k, v, given its o and lse and
 * dout = dL/do.  dk and dv sum over the H / HK query heads that share them, in FP32, before one
 * rounding.  A value that is not finite may reach any gradient of its own sequence.  workspace: 256-byte
 * aligned.
 */
la_status la_attn_prefill_bwd(const void* q, const void* k, const void* v, float scale, const void* o,
                              const float* lse, const void* dout, const int32_t* cu_seqlens, void* dq, void* dk,
                              void* dv, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv, int64_t hsv,
                              int64_t ldo, int64_t hso, int64_t lddo, int64_t hsdo, int64_t lddq, int64_t hsdq,
                              int64_t lddk, int64_t hsdk, int64_t lddv, int64_t hsdv, int B, int T, int N, int H,
                              int HK, int D, void* workspace, size_t workspace_bytes, int* dev_error, void* stream);

/*
 * The cache of la_attn_verify and la_attn_commit: k_cache, v_cache BF16 [pages, page_size, HK, D],
 * innermost contiguous, with strides between pages, tokens and heads (kp, kt, kh; vp, vt, vh), all
 * multiples of 8 elements, 16-byte aligned (so pages may be token-major or head-major, and keys and
 * values may share pages).  With page_table int32 [B, table_width] (row stride ld_table),
 * token i of request b is row i % page_size of page page_table[b][i / page_size]; page_size is then
 * a multiple of 16 and entries behind the request's last page are not read.  Without it
 * (page_table null) request b has page b whole (pages >= B, any page_size).
 * cache_lens int32 [B]: tokens in the cache per request; a negative length marks a padded request:
 * nothing is read or written for it.  A length beyond the pages skips the request
 * (LA_DEV_ERR_BAD_SEQLENS).  A page number outside [0, pages) (LA_DEV_ERR_BAD_INDEX) leaves the
 * outputs of its request in la_attn_verify, and that page's tokens in la_attn_commit, unwritten.
 * What lies in the cache behind a request's tokens reaches no result.
 */

/* Bytes of device workspace la_attn_verify needs.  Host only. */
la_status la_attn_verify_workspace(int B, int T, int H, int HK, int D, size_t* bytes);

/*
 * la_attn_verify -- the outputs of T drafted tokens of each of B requests (T = 1: decode).  q, o
 * [B*T, H, D] and the drafted tokens' own k, v [B*T, HK, D] are token-major by request; the cache
 * is left untouched.  A drafted token sees the request's whole cache and, of the drafted tokens,
 * those whose bits are set in mask[b][t] (int64 [B, T], nullable; bit u = drafted token u; T <= 64;
 * bits from T on are ignored); without a mask it sees drafted tokens 0 .. t (T <= 262144).
 * workspace: 256-byte aligned.  H / HK <= 128.
 */
la_status la_attn_verify(const void* q, const void* k, const void* v, float scale, const void* k_cache,
                         const void* v_cache, const int32_t* cache_lens, const int32_t* page_table,
                         const int64_t* mask, void* o, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv,
                         int64_t hsv, int64_t ldo, int64_t hso, int64_t kp, int64_t kt, int64_t kh, int64_t vp,
                         int64_t vt, int64_t vh, int64_t ld_table, int B, int T, int H, int HK, int D, int pages,
                         int page_size, int table_width, void* workspace, size_t workspace_bytes, int* dev_error,
                         void* stream);

/*
 * la_attn_commit -- write tokens' keys and values k, v [tokens, HK, D] into the cache behind each
 * request's cache_lens tokens (cache_lens itself is the caller's to advance).
 *   cu_seqlens null: request b has tokens b*T .. b*T + T - 1 and commits accepted_len[b] of them
 *     (clamped to [0, T]; null: all T): its tokens path[b][0], path[b][1], ... (int32 [B, T]; null:
 *     the first ones).  A path entry outside [0, T) skips that token (LA_DEV_ERR_BAD_INDEX).
 *   cu_seqlens int32 [B + 1]: request b commits tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (T is
 *     the number of tokens; accepted_len and path null); bounds that do not fit skip the request.
 * Two requests must not write the same row of a page.
 */
la_status la_attn_commit(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* cache_lens,
                         const int32_t* cu_seqlens, const int32_t* accepted_len, const int32_t* path,
                         const int32_t* page_table, int64_t ldk, int64_t hsk, int64_t ldv, int64_t hsv, int64_t kp,
                         int64_t kt, int64_t kh, int64_t vp, int64_t vt, int64_t vh, int64_t ld_table, int B, int T,
                         int HK, int D, int pages, int page_size, int table_width, int* dev_error, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_ATTENTION_H */
