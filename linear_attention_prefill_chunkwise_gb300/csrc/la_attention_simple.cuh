// la_attention_simple.cuh -- the attention kernels (include/la_attention.h) in their simplest form: a
// warp per row (or key) and head, lanes along D, one key at a time with a running maximum and sum.
#pragma once

#include "la_attention_params.cuh"
#include "sm103_ptx.cuh"

namespace laa {

template <int D>
struct Row {
  float v[D / 32];
};
template <int D>
__device__ __forceinline__ Row<D> load_row(const bf16* p, int lane) {
  Row<D> r;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) r.v[i] = __bfloat162float(p[lane + 32 * i]);
  return r;
}
template <int D>
__device__ __forceinline__ void store_row(bf16* p, int lane, const Row<D>& r) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p[lane + 32 * i] = __float2bfloat16_rn(r.v[i]);
}
template <int D>
__device__ __forceinline__ float dot(const Row<D>& a, const Row<D>& b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) s = fmaf(a.v[i], b.v[i], s);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}
template <int D>
__device__ __forceinline__ void axpy(Row<D>& y, float a, const Row<D>& x) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) y.v[i] = fmaf(a, x.v[i], y.v[i]);
}

// Running softmax of one row.
template <int D>
struct Running {
  float top = -INFINITY, sum = 0.f;
  Row<D> acc = {};
  __device__ __forceinline__ void add(float z, const Row<D>& v) {
    const float m = fmaxf(top, z);
    if (m == -INFINITY) return;
    const float old = expf(top - m), e = expf(z - m);
    sum = sum * old + e;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc.v[i] *= old;
    axpy<D>(acc, e, v);
    top = m;
  }
  __device__ __forceinline__ Row<D> result() const {
    Row<D> r = acc;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) r.v[i] = sum > 0.f ? r.v[i] / sum : 0.f;
    return r;
  }
};

// The sequence of a row, by its bounds; false for a row of none.
__device__ __forceinline__ bool row_bounds(const PrefillParams& p, int row, int& lo, int& hi) {
  if (!p.cu_seqlens) {
    lo = row / p.T * p.T;
    hi = lo + p.T;
    return true;
  }
  if (row == 0 && threadIdx.x == 0 && blockIdx.y == 0 && p.dev_error)
    for (int n = 0; n < p.N; ++n)
      if (!sequence_rows(p, n, lo, hi)) atomicOr(p.dev_error, kErrSeqlens);
  for (int n = 0; n < p.N; ++n)
    if (sequence_rows(p, n, lo, hi) && row >= lo && row < hi) return true;
  return false;
}

template <int D>
__global__ void simple_fwd_kernel(const PrefillParams p) {
  const int row = blockIdx.x * 4 + threadIdx.x / 32, h = blockIdx.y, lane = threadIdx.x % 32;
  int lo, hi;
  if (row >= p.tokens || !row_bounds(p, row, lo, hi)) return;
  const int hk = h / (p.H / p.HK);
  const Row<D> q = load_row<D>(p.q.row(row, h), lane);
  Running<D> r;
  for (int j = lo; j <= row; ++j)
    r.add(p.scale * dot<D>(q, load_row<D>(p.k.row(j, hk), lane)), load_row<D>(p.v.row(j, hk), lane));
  store_row<D>(p.o.row(row, h), lane, r.result());
  if (p.lse && lane == 0) p.lse[static_cast<int64_t>(h) * p.tokens + row] = r.top + logf(r.sum);
}

template <int D>
__global__ void simple_dq_kernel(const PrefillParams p) {
  const int row = blockIdx.x * 4 + threadIdx.x / 32, h = blockIdx.y, lane = threadIdx.x % 32;
  int lo, hi;
  if (row >= p.tokens || !row_bounds(p, row, lo, hi)) return;
  const int hk = h / (p.H / p.HK);
  const int64_t at = static_cast<int64_t>(h) * p.tokens + row;
  const Row<D> q = load_row<D>(p.q.row(row, h), lane), g = load_row<D>(p.dout.row(row, h), lane);
  const float delta = dot<D>(g, load_row<D>(p.o_in.row(row, h), lane)), lse = p.lse_in[at];
  if (lane == 0) p.delta[at] = delta;
  Row<D> dq = {};
  for (int j = lo; j <= row; ++j) {
    const Row<D> k = load_row<D>(p.k.row(j, hk), lane);
    const float pj = expf(p.scale * dot<D>(q, k) - lse);
    axpy<D>(dq, p.scale * pj * (dot<D>(g, load_row<D>(p.v.row(j, hk), lane)) - delta), k);
  }
  store_row<D>(p.dq.row(row, h), lane, dq);
}

template <int D>
__global__ void simple_dkdv_kernel(const PrefillParams p) {
  const int j = blockIdx.x * 4 + threadIdx.x / 32, hk = blockIdx.y, lane = threadIdx.x % 32;
  int lo, hi;
  if (j >= p.tokens || !row_bounds(p, j, lo, hi)) return;
  const int G = p.H / p.HK;
  const Row<D> k = load_row<D>(p.k.row(j, hk), lane), v = load_row<D>(p.v.row(j, hk), lane);
  Row<D> dk = {}, dv = {};
  for (int h = hk * G; h < (hk + 1) * G; ++h)
    for (int t = j; t < hi; ++t) {
      const int64_t at = static_cast<int64_t>(h) * p.tokens + t;
      const Row<D> q = load_row<D>(p.q.row(t, h), lane), g = load_row<D>(p.dout.row(t, h), lane);
      const float pj = expf(p.scale * dot<D>(q, k) - p.lse_in[at]);
      axpy<D>(dv, pj, g);
      axpy<D>(dk, p.scale * pj * (dot<D>(g, v) - p.delta[at]), q);
    }
  store_row<D>(p.dk.row(j, hk), lane, dk);
  store_row<D>(p.dv.row(j, hk), lane, dv);
}

// Offset of cached token i of request b in elements, for strides (page, token).
__device__ __forceinline__ int64_t cached(const CacheParams& p, int b, int i, int64_t page, int64_t token) {
  const int n = p.page_table ? p.page_table[b * p.ld_table + i / p.page_size] : b;
  return n * page + (p.page_table ? i % p.page_size : i) * token;
}

// Whether a request runs; reports why not.
__device__ __forceinline__ bool request_fits(const CacheParams& p, int b, int rows, int len, int lane) {
  if (len < 0) return false;
  int err = 0;
  if (len + static_cast<int64_t>(rows) > capacity(p)) err = kErrSeqlens;
  if (!err && p.page_table)
    for (int i = lane; i * static_cast<int64_t>(p.page_size) < len + static_cast<int64_t>(rows); i += 32) {
      const int n = p.page_table[b * p.ld_table + i];
      if (n < 0 || n >= p.pages) err = kErrIndex;
    }
  err = __reduce_or_sync(0xFFFFFFFFu, err);
  if (err && lane == 0 && p.dev_error) atomicOr(p.dev_error, err);
  return err == 0;
}

template <int D>
__global__ void simple_verify_kernel(const CacheParams p) {
  const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, b = row / p.T, t = row % p.T;
  const int len = p.cache_lens[b], hk = h / (p.H / p.HK);
  if (!request_fits(p, b, 0, len, lane)) return;
  const Row<D> q = load_row<D>(p.q.row(row, h), lane);
  Running<D> r;
  for (int i = 0; i < len; ++i)
    r.add(p.scale * dot<D>(q, load_row<D>(p.k_cache + cached(p, b, i, p.kp, p.kt) + hk * p.kh, lane)),
          load_row<D>(p.v_cache + cached(p, b, i, p.vp, p.vt) + hk * p.vh, lane));
  for (int u = 0; u < p.T; ++u) {
    if (p.mask ? !(p.mask[row] >> u & 1) : u > t) continue;
    const int64_t at = static_cast<int64_t>(b) * p.T + u;
    r.add(p.scale * dot<D>(q, load_row<D>(p.k.row(at, hk), lane)), load_row<D>(p.v.row(at, hk), lane));
  }
  store_row<D>(p.o.row(row, h), lane, r.result());
}

}  // namespace laa
