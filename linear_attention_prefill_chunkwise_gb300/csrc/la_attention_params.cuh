// la_attention_params.cuh -- what the attention kernels (include/la_attention.h) are told, and the
// steps they share: bounds of sequences and rows of the cache.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace laa {

using bf16 = __nv_bfloat16;

// One tensor of heads: element (t, h, d) lies at p[t * ld + h * hs + d].
template <typename E>
struct Heads {
  E* p;
  int64_t ld, hs;
  __device__ __forceinline__ E* row(int64_t t, int h) const { return p + t * ld + h * hs; }
};

constexpr int kErrSeqlens = 1, kErrIndex = 2, kErrTimeout = 4;  // LA_DEV_ERR_*

struct PrefillParams {
  Heads<const bf16> v, o_in, dout;  // (q and k come by tensor maps)
  Heads<bf16> o, dq, dk, dv;
  float* lse;           // [H, tokens]
  const float* lse_in;  // gradients
  float* delta;         // [H, tokens] rowsum(dO o), gradients' workspace
  float* part;          // [splits][dk, dv][HK][tokens][D] sums over parts of a group's heads; null: one part
  uint8_t* marks;       // [HK, tokens] whether a row has such sums
  const int32_t* cu_seqlens;
  int* dev_error;
  float scale;
  int tokens, T, N, H, HK, splits;
};

struct CacheParams {
  Heads<const bf16> k, v;  // la_attn_verify: q, k and the cache come by tensor maps
  Heads<bf16> o;
  bf16 *k_out, *v_out;  // la_attn_commit, with the strides that follow
  int64_t kp, kt, kh, vp, vt, vh, ld_table;
  const int32_t *cache_lens, *page_table, *cu_seqlens, *accepted_len, *path;
  const int64_t* mask;
  void* part;  // workspace
  int* dev_error;
  float scale;
  int B, T, HK, D, pages, page_size, table_width;
};

// Rows [lo, hi) of sequence n; an empty range (and the error bit) where its bounds do not fit.
__device__ __forceinline__ bool sequence_rows(const PrefillParams& p, int n, int& lo, int& hi) {
  if (!p.cu_seqlens) {
    lo = n * p.T;
    hi = lo + p.T;
    return true;
  }
  lo = __ldg(p.cu_seqlens + n);
  hi = __ldg(p.cu_seqlens + n + 1);
  if (lo < 0 || hi < lo || hi > p.tokens) {
    lo = hi = 0;
    return false;
  }
  return true;
}

// Tokens that the cache can hold for a request.
__device__ __forceinline__ int64_t capacity(const CacheParams& p) {
  return p.page_table ? static_cast<int64_t>(p.table_width) * p.page_size : p.page_size;
}

}  // namespace laa
