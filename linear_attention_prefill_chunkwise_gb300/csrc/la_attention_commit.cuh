// la_attention_commit.cuh -- the writes of keys and values into the cache (include/la_attention.h).
//
// A block takes kTokens tokens of one request: the request's bounds and its pages are looked up by
// the block's first threads, then the tokens' heads move 16 bytes at a time.  Each row is read once
// and written once; the call is bound by those bytes (16 prompts of up to 4096 tokens, 8 heads of 128: 45 us,
// 0.85 of the copy rate), a small one by its launch and three reads that wait for each other (7 us).
#pragma once

#include "la_attention_params.cuh"
#include "sm103_ptx.cuh"

namespace laa {

constexpr int kCommitTokens = 16, kCommitThreads = 256;

static __global__ void __launch_bounds__(kCommitThreads) commit_kernel(const CacheParams p) {
  __shared__ int64_t src[kCommitTokens], page[kCommitTokens];
  __shared__ int slot[kCommitTokens];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int b = blockIdx.x;
  const int len = __ldg(p.cache_lens + b);
  if (len < 0) return;
  int64_t first;
  int n;
  if (p.cu_seqlens) {
    const int lo = __ldg(p.cu_seqlens + b), hi = __ldg(p.cu_seqlens + b + 1);
    if (lo < 0 || hi < lo || hi > p.T) {
      if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, kErrSeqlens);
      return;
    }
    first = lo;
    n = hi - lo;
  } else {
    first = static_cast<int64_t>(b) * p.T;
    n = p.accepted_len ? min(max(__ldg(p.accepted_len + b), 0), p.T) : p.T;
  }
  if (n == 0) return;
  if (len + static_cast<int64_t>(n) > capacity(p)) {
    if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, kErrSeqlens);
    return;
  }
  const int vecs = p.D / 8, per_token = p.HK * vecs;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.y) * kCommitTokens; i0 < n;
       i0 += static_cast<int64_t>(gridDim.y) * kCommitTokens) {
    const int count = static_cast<int>(min(static_cast<int64_t>(kCommitTokens), n - i0));
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < count) {
      const int i = static_cast<int>(i0) + threadIdx.x, at = len + i;
      int64_t from = i;
      bool bad = false;
      if (p.path) {
        from = __ldg(p.path + first + i);
        bad = from < 0 || from >= p.T;
      }
      int64_t pg = b;
      int sl = at;
      if (p.page_table) {
        pg = __ldg(p.page_table + b * p.ld_table + at / p.page_size);
        sl = at % p.page_size;
        bad = bad || pg < 0 || pg >= p.pages;
      }
      if (bad && p.dev_error) atomicOr(p.dev_error, kErrIndex);
      src[threadIdx.x] = bad ? -1 : first + from;
      page[threadIdx.x] = pg;
      slot[threadIdx.x] = sl;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < count * per_token; x += kCommitThreads) {
      const int i = x / per_token, r = x - i * per_token, h = r / vecs, d = (r - h * vecs) * 8;
      if (src[i] < 0) continue;
      const uint4 kx = *reinterpret_cast<const uint4*>(p.k.row(src[i], h) + d);
      const uint4 vx = *reinterpret_cast<const uint4*>(p.v.row(src[i], h) + d);
      *reinterpret_cast<uint4*>(p.k_out + page[i] * p.kp + slot[i] * p.kt + h * p.kh + d) = kx;
      *reinterpret_cast<uint4*>(p.v_out + page[i] * p.vp + slot[i] * p.vt + h * p.vh + d) = vx;
    }
  }
}

}  // namespace laa
