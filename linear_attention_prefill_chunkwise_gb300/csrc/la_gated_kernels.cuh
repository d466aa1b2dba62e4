// la_gated_kernels.cuh -- kernels of the gated linear recurrence (include/la_gated.h).
//
// One thread per (sequence, channel) walks the sequence's tokens in order (in reverse order for
// the gradients); neighbouring threads hold neighbouring channels, so every load and store of a
// warp is one contiguous row piece.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "la_gated_math.cuh"
#include "sm103_ptx.cuh"

namespace lag {

constexpr unsigned kErrBadSeqlens = 1u, kErrBadIndex = 2u;
constexpr int kThreads = 128;

template <typename E>
struct Params {
  const E *x, *r, *g;
  const E *o_in, *dout;  // backward
  E *o, *dx, *dr, *dg;
  int64_t ldx, ldr, ldg, ldo, lddout, lddx, lddr, lddg;
  const float* slopes;
  const float* start;  // [P, C] states the walk begins with (h0; dh_final) or null
  const float* h0;     // backward: [P, C] or null
  float* finish;       // [P, C] states it ends with (h_final; dh0) or null
  float* dslopes;
  float* part;         // backward: [N, C] sums of each sequence's terms of dslopes
  const int32_t* state_indices;
  const int32_t* cu_seqlens;
  const int32_t* accepted_len;
  const int* bad;      // set by check_seqlens_kernel (packed mode)
  int* dev_error;
  int T, N, C, pool_size;
};

// cu_seqlens non-decreasing inside [0, T]?
__global__ void check_seqlens_kernel(const int32_t* cu, int N, int T, int* bad, int* dev_error) {
  int wrong = 0;
  for (int n = threadIdx.x; n < N; n += blockDim.x) wrong |= cu[n] < 0 || cu[n] > cu[n + 1] || cu[n + 1] > T;
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) {
    *bad = wrong;
    if (wrong && dev_error) atomicOr(reinterpret_cast<unsigned*>(dev_error), kErrBadSeqlens);
  }
}

struct Unit {
  int n, c, slot;
  int64_t first, rows;
};

template <typename E>
__device__ __forceinline__ bool unit_of(const Params<E>& p, Unit* q) {
  const int tiles = (p.C + kThreads - 1) / kThreads;
  q->n = static_cast<int>(blockIdx.x / tiles);
  q->c = static_cast<int>(blockIdx.x % tiles) * kThreads + static_cast<int>(threadIdx.x);
  q->slot = p.state_indices ? p.state_indices[q->n] : q->n;
  if (q->slot >= p.pool_size) {
    if (threadIdx.x == 0 && p.dev_error) atomicOr(reinterpret_cast<unsigned*>(p.dev_error), kErrBadIndex);
    q->slot = -1;
  }
  if (p.cu_seqlens) {
    q->first = p.cu_seqlens[q->n];
    q->rows = p.cu_seqlens[q->n + 1] - q->first;
  } else {
    q->first = static_cast<int64_t>(q->n) * p.T;
    q->rows = p.T;
  }
  return q->c < p.C && !(p.bad && *p.bad);
}

template <typename E, bool kDecode>
__global__ void __launch_bounds__(kThreads) gated_fwd_kernel(const Params<E> p) {
  constexpr bool kPrecise = sizeof(E) == 4;
  Unit q;
  if (!unit_of(p, &q) || q.slot < 0) return;
  const float slope = p.slopes[q.c];
  const size_t at = static_cast<size_t>(q.slot) * p.C + q.c;
  float h = p.start ? p.start[at] : 0.f;
  int64_t keep = q.rows;
  if constexpr (kDecode) {
    if (p.accepted_len) {
      const int a = p.accepted_len[q.n];
      keep = a < 0 ? 0 : a > q.rows ? q.rows : a;
      q.rows = keep;
    }
  }
  for (int64_t t = q.first; t < q.first + q.rows; ++t) {
    const float x = to_f32(p.x[t * p.ldx + q.c]);
    const Decay d = decay_of<kPrecise>(slope * sigmoid<kPrecise>(to_f32(p.r[t * p.ldr + q.c])));
    h = fmaf(d.lambda, h, d.beta * sigmoid<kPrecise>(to_f32(p.g[t * p.ldg + q.c])) * x);
    if (p.o) p.o[t * p.ldo + q.c] = from_f32<E>(h);
  }
  if (p.finish && !(kDecode && q.rows == 0)) p.finish[at] = h;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) gated_bwd_kernel(const Params<E> p) {
  constexpr bool kPrecise = sizeof(E) == 4;
  Unit q;
  if (!unit_of(p, &q)) return;
  float sum = 0.f;
  if (q.slot >= 0) {
    const float slope = p.slopes[q.c];
    const size_t at = static_cast<size_t>(q.slot) * p.C + q.c;
    float w = p.start ? p.start[at] : 0.f;  // lambda_{t+1} G_{t+1}
    for (int64_t t = q.first + q.rows - 1; t >= q.first; --t) {
      const float r = to_f32(p.r[t * p.ldr + q.c]);
      const float G = to_f32(p.dout[t * p.lddout + q.c]) + w;
      const float before = t > q.first ? to_f32(p.o_in[(t - 1) * p.ldo + q.c]) : p.h0 ? p.h0[at] : 0.f;
      const Grads d = grads_of<kPrecise>(to_f32(p.x[t * p.ldx + q.c]), r, to_f32(p.g[t * p.ldg + q.c]), slope, G,
                                         before);
      w = decay_of<kPrecise>(slope * sigmoid<kPrecise>(r)).lambda * G;
      p.dx[t * p.lddx + q.c] = from_f32<E>(d.dx);
      p.dr[t * p.lddr + q.c] = from_f32<E>(d.dr);
      p.dg[t * p.lddg + q.c] = from_f32<E>(d.dg);
      sum += d.ds;
    }
    if (p.finish) p.finish[at] = w;
  }
  p.part[static_cast<size_t>(q.n) * p.C + q.c] = sum;
}

// out[c] = sum over rows of part[rows][C], in row order.
__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float* part, int rows, int C, const int* bad,
                                                              float* out) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= C || (bad && *bad)) return;
  float s = 0.f;
  for (int i = 0; i < rows; ++i) s += part[static_cast<size_t>(i) * C + c];
  out[c] = s;
}

}  // namespace lag
