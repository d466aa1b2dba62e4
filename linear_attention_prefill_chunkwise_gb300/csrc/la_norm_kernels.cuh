// la_norm_kernels.cuh -- kernels of the root-mean-square norm (include/la_norm.h): one block per
// row, three passes over it (sum of squares, largest |y| for the 8-bit output, output).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "la_gated_math.cuh"

namespace lan {

using lag::from_f32;
using lag::to_f32;

constexpr int kThreads = 256;
constexpr int kBlocks = 608;  // blocks (rows of partial sums) of the gradient kernel: 4 per SM
constexpr int kGroup = 128;   // columns per scale of the grouped 8-bit output

template <typename E>
struct FwdParams {
  const E *x, *res;
  E *y, *res_out;
  uint8_t* y8;
  float* scales;
  const float* weight;
  int64_t ldx, ldres, ldy, ldres_out;
  float eps;
  int rows, C, group;
};

template <typename E>
struct BwdParams {
  const E *s, *dy, *dres;
  E* dx;
  const float* weight;
  float *part, *dweight;
  int64_t lds, lddy, lddres, lddx;
  float eps;
  int rows, C;
};

// Sum (or maximum) over the block, returned to every thread.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* smem) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = smem[0];
  for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i) t = kMax ? fmaxf(t, smem[i]) : t + smem[i];
  return t;
}

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

template <typename E, bool kFp8>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const FwdParams<E> p) {
  __shared__ float red[kThreads / 32];
  const int64_t row = blockIdx.x;
  const E* x = p.x + row * p.ldx;
  const E* res = p.res ? p.res + row * p.ldres : nullptr;
  auto sum_at = [&](int c) { return res ? to_f32(x[c]) + to_f32(res[c]) : to_f32(x[c]); };
  float ss = 0.f;
  for (int c = threadIdx.x; c < p.C; c += kThreads) {
    const float s = sum_at(c);
    ss = fmaf(s, s, ss);
  }
  const float rstd = rsqrtf(block_reduce<false>(ss, red) / static_cast<float>(p.C) + p.eps);
  if constexpr (kFp8) {
    const int width = p.group ? p.group : p.C;
    const int groups = (p.C + width - 1) / width;
    for (int k = 0; k < groups; ++k) {
      const int end = min(p.C, (k + 1) * width);
      float m = 0.f;
      for (int c = k * width + threadIdx.x; c < end; c += kThreads) m = fmaxf(m, fabsf(sum_at(c) * rstd * p.weight[c]));
      m = fmaxf(block_reduce<true>(m, red), 0x1p-40f);
      if (threadIdx.x == 0) p.scales[row * groups + k] = m / 448.f;
      const float inv = 448.f / m;
      for (int c = k * width + threadIdx.x; c < end; c += kThreads)
        p.y8[row * p.ldy + c] = to_e4m3(sum_at(c) * rstd * p.weight[c] * inv);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.C; c += kThreads) {
    const float s = sum_at(c);
    if constexpr (!kFp8) p.y[row * p.ldy + c] = from_f32<E>(s * rstd * p.weight[c]);
    if (p.res_out) p.res_out[row * p.ldres_out + c] = from_f32<E>(s);
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const BwdParams<E> p) {
  __shared__ float red[kThreads / 32];
  float* part = p.part + static_cast<size_t>(blockIdx.x) * p.C;
  for (int c = threadIdx.x; c < p.C; c += kThreads) part[c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const E* s = p.s + row * p.lds;
    const E* dy = p.dy + row * p.lddy;
    float ss = 0.f, dot = 0.f;
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
      const float v = to_f32(s[c]);
      ss = fmaf(v, v, ss);
      dot = fmaf(to_f32(dy[c]) * p.weight[c], v, dot);
    }
    const float rstd = rsqrtf(block_reduce<false>(ss, red) / static_cast<float>(p.C) + p.eps);
    const float m = block_reduce<false>(dot, red) * rstd / static_cast<float>(p.C);  // mean(w dy n)
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
      const float n = to_f32(s[c]) * rstd, d = to_f32(dy[c]);
      float dx = rstd * (p.weight[c] * d - n * m);
      if (p.dres) dx += to_f32(p.dres[row * p.lddres + c]);
      p.dx[row * p.lddx + c] = from_f32<E>(dx);
      part[c] = fmaf(d, n, part[c]);
    }
  }
}

// out[c] = sum over rows of part[rows][C], in row order.
__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float* part, int rows, int C, float* out) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int i = 0; i < rows; ++i) s += part[static_cast<size_t>(i) * C + c];
  out[c] = s;
}

}  // namespace lan
