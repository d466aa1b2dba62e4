// la_rotary_kernels.cuh -- kernels of the norm and position rotation of queries and keys
// (include/la_rotary.h).
//
// A head of D elements is held by D / (2 kVec) threads: each has kVec pairs that rotate together,
// as two vectors of kVec elements, so that a pair never leaves its thread and the only exchange is
// the sum of squares over those threads.  With kVec * sizeof(E) = 16 both vectors are 16-byte
// accesses; kVec = 1 takes any alignment and any rotated part R.  The work is bound by the bytes of
// the heads (read once, written once); a token's cosines and sines are shared by all of its heads,
// so a block takes whole tokens and computes them once into shared memory.
//
// The angle of a pair, in turns, is position * frequency / 2 pi modulo 1: the frequency is scaled
// to a 64-bit fraction of a turn once, and the product wraps around by itself.  Its error is
// |position| 2^-53 |frequency| radians, 2^-24 of a turn's half after the conversion to FP32.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "la_vec.cuh"
#include "sm103_ptx.cuh"

namespace lar {

constexpr int kThreads = 256;

// One tensor of heads: element (t, h, d) lies at p[t * ld + h * hs + d].
template <typename E>
struct Heads {
  E* p;
  int64_t ld, hs;
};

template <typename E>
struct FwdParams {
  Heads<const E> x[2];  // q, k
  Heads<E> y[2];
  const float* weight[2];
  const int32_t* positions;
  const float* inv_freq;
  float eps;
  int tokens, heads[2], R, interleaved, per_block;  // tokens of a block
};

template <typename E>
struct BwdParams {
  Heads<const E> x[2], dy[2];
  Heads<E> dx[2];
  const float* weight[2];
  const int32_t* positions;
  const float* inv_freq;
  float* part;  // [2][blocks][D] sums of each block's rows; null: no weight gradients
  float eps;
  int tokens, heads[2], R, interleaved, per_block;
};

template <typename E, int kVec, int D>
struct Layout {
  static constexpr int kPairs = D / (2 * kVec);  // groups of kVec pairs in a head
  static constexpr int kLanes = kPairs < 32 ? kPairs : 32;
  static constexpr int kChunks = kPairs / kLanes;
  static constexpr int kGroups = kThreads / kLanes;  // heads that a block holds at once
};

// Where the two vectors of pair group c begin.
template <int kVec>
__device__ __forceinline__ void places(int c, int R, int interleaved, int& a, int& b) {
  const int rotated = R / (2 * kVec);
  if (c >= rotated || interleaved) {
    a = 2 * kVec * c;
    b = a + kVec;
  } else {
    a = kVec * c;
    b = a + R / 2;
  }
}

// cos and sin of the angle of pair i at a position.
__device__ __forceinline__ float2 angle(int32_t position, float inv_freq) {
  const double turn = static_cast<double>(inv_freq) * 0.15915494309189535;  // 1 / 2 pi
  const long long unit = __double2ll_rn((turn - rint(turn)) * 0x1p63);      // half fractions of 2^64
  const long long phase = static_cast<long long>(static_cast<unsigned long long>(unit) *
                                                 (2ull * static_cast<unsigned long long>(static_cast<long long>(position))));
  float s, c;
  sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);
  return make_float2(c, s);
}

// The rotation of kVec pairs; sign = -1 turns back.
template <int kVec>
__device__ __forceinline__ void turn(float (&a)[kVec], float (&b)[kVec], const float2* cs, int interleaved, float sign) {
  if (interleaved && kVec > 1) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      float& lo = 2 * e < kVec ? a[(2 * e) % kVec] : b[(2 * e) % kVec];
      float& hi = 2 * e < kVec ? a[(2 * e + 1) % kVec] : b[(2 * e + 1) % kVec];
      const float c = cs[e].x, s = sign * cs[e].y, x = lo, y = hi;
      lo = x * c - y * s;
      hi = x * s + y * c;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const float c = cs[e].x, s = sign * cs[e].y, x = a[e], y = b[e];
      a[e] = x * c - y * s;
      b[e] = x * s + y * c;
    }
  }
}

// kVec elements as loaded: the next head's are on their way while one is computed.
template <typename E, int kVec>
struct Raw {
  using T = std::conditional_t<kVec == 1, E, uint4>;
  T v;
  __device__ __forceinline__ void load(const E* p) { v = *reinterpret_cast<const T*>(p); }
  __device__ __forceinline__ void expand(float (&f)[kVec]) const { lan::load<kVec>(reinterpret_cast<const E*>(&v), f); }
};

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <int kVec>
__device__ __forceinline__ void load_weight(const float* p, float (&v)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e) v[e] = p ? __ldg(p + e) : 1.f;
}

// A thread's own elements of a head and their weights.
template <typename E, int kVec, int D>
__device__ __forceinline__ void own_weights(const float* w, int lane, int R, int interleaved,
                                            int (&at)[Layout<E, kVec, D>::kChunks], int (&bt)[Layout<E, kVec, D>::kChunks],
                                            float (&wa)[Layout<E, kVec, D>::kChunks][kVec],
                                            float (&wb)[Layout<E, kVec, D>::kChunks][kVec]) {
#pragma unroll
  for (int i = 0; i < Layout<E, kVec, D>::kChunks; ++i) {
    places<kVec>(lane + 32 * i, R, interleaved, at[i], bt[i]);
    load_weight<kVec>(w ? w + at[i] : nullptr, wa[i]);
    load_weight<kVec>(w ? w + bt[i] : nullptr, wb[i]);
  }
}

// Cosines and sines of a block's tokens into shared memory, [tokens][R / 2].
template <typename P>
__device__ __forceinline__ void fill_angles(const P& p, float2* cs, int first, int count) {
  const int half = p.R / 2;
  for (int i = threadIdx.x; i < count * half; i += kThreads) {
    const int t = i / half;
    cs[i] = angle(__ldg(p.positions + first + t), __ldg(p.inv_freq + (i - t * half)));
  }
}

template <typename E, int kVec, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(const FwdParams<E> p) {
  using L = Layout<E, kVec, D>;
  extern __shared__ float2 cs[];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int first = blockIdx.x * p.per_block;
  const int count = min(p.per_block, p.tokens - first);
  const int lane = threadIdx.x % L::kLanes, group = threadIdx.x / L::kLanes;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = p.heads[which], rows = count * heads;
    const Heads<const E> hx = p.x[which];
    const Heads<E> hy = p.y[which];
    int at[L::kChunks], bt[L::kChunks];
    float wa[L::kChunks][kVec], wb[L::kChunks][kVec];
    own_weights<E, kVec, D>(p.weight[which], lane, p.R, p.interleaved, at, bt, wa, wb);
    Raw<E, kVec> xa[L::kChunks], xb[L::kChunks];
    auto fetch = [&](int r) {
      if (r >= rows) return;
      const int t = r / heads, h = r - t * heads;
      const E* x = hx.p + (first + t) * hx.ld + h * hx.hs;
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        xa[i].load(x + at[i]);
        xb[i].load(x + bt[i]);
      }
    };
    fetch(group);
    if (which == 0) {
      fill_angles(p, cs, first, count);
      __syncthreads();
    }
    // every lane of a warp takes the same number of turns (the sums are over whole warps)
    for (int r0 = 0; r0 < rows; r0 += L::kGroups) {
      const int r = r0 + group;
      const bool live = r < rows;
      const int t = live ? r / heads : 0, h = live ? r - t * heads : 0;
      E* y = hy.p + (first + t) * hy.ld + h * hy.hs;
      float a[L::kChunks][kVec], b[L::kChunks][kVec], ss = 0.f;
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        xa[i].expand(a[i]);
        xb[i].expand(b[i]);
      }
      fetch(r + L::kGroups);
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          ss = fmaf(a[i][e], a[i][e], ss);
          ss = fmaf(b[i][e], b[i][e], ss);
        }
      }
      ss = sum_lanes<L::kLanes>(ss);
      const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        const int c = lane + 32 * i;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          a[i][e] *= rstd * wa[i][e];
          b[i][e] *= rstd * wb[i][e];
        }
        if (c < p.R / (2 * kVec)) turn<kVec>(a[i], b[i], cs + t * (p.R / 2) + c * kVec, p.interleaved, 1.f);
        if (live) {
          lan::store<kVec>(y + at[i], a[i]);
          lan::store<kVec>(y + bt[i], b[i]);
        }
      }
    }
  }
}

// The gradients.  A block walks over its share of the tokens, first all of its queries, then
// all of its keys, and keeps the sums for the weight gradients of its threads' own elements in registers.
template <typename E, int kVec, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const BwdParams<E> p) {
  using L = Layout<E, kVec, D>;
  extern __shared__ float2 cs[];
  __shared__ float sums[L::kGroups][D];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int lane = threadIdx.x % L::kLanes, group = threadIdx.x / L::kLanes;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = p.heads[which];
    const Heads<const E> hx = p.x[which], hdy = p.dy[which];
    const Heads<E> hdx = p.dx[which];
    int at[L::kChunks], bt[L::kChunks];
    float wa[L::kChunks][kVec], wb[L::kChunks][kVec];
    own_weights<E, kVec, D>(p.weight[which], lane, p.R, p.interleaved, at, bt, wa, wb);
    float da[L::kChunks][kVec] = {}, db[L::kChunks][kVec] = {};
    const int64_t stop = static_cast<int64_t>(blockIdx.x + 1) * p.tokens / gridDim.x;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * p.tokens / gridDim.x; first < stop; first += p.per_block) {
      const int count = static_cast<int>(min(static_cast<int64_t>(p.per_block), stop - first));
      const int rows = count * heads;
      Raw<E, kVec> xa[L::kChunks], xb[L::kChunks], ya[L::kChunks], yb[L::kChunks];
      auto fetch = [&](int r) {
        if (r >= rows) return;
        const int t = r / heads, h = r - t * heads;
        const E* x = hx.p + (first + t) * hx.ld + h * hx.hs;
        const E* dy = hdy.p + (first + t) * hdy.ld + h * hdy.hs;
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
          xa[i].load(x + at[i]);
          xb[i].load(x + bt[i]);
          ya[i].load(dy + at[i]);
          yb[i].load(dy + bt[i]);
        }
      };
      fetch(group);
      __syncthreads();
      fill_angles(p, cs, static_cast<int>(first), count);
      __syncthreads();
      for (int r0 = 0; r0 < rows; r0 += L::kGroups) {
        const int r = r0 + group;
        const bool live = r < rows;
        const int t = live ? r / heads : 0, h = live ? r - t * heads : 0;
        float a[L::kChunks][kVec], b[L::kChunks][kVec], ga[L::kChunks][kVec], gb[L::kChunks][kVec];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
          xa[i].expand(a[i]);
          xb[i].expand(b[i]);
          ya[i].expand(ga[i]);
          yb[i].expand(gb[i]);
        }
        fetch(r + L::kGroups);
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
          const int c = lane + 32 * i;
          if (c < p.R / (2 * kVec)) turn<kVec>(ga[i], gb[i], cs + t * (p.R / 2) + c * kVec, p.interleaved, -1.f);
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            ss = fmaf(a[i][e], a[i][e], ss);
            ss = fmaf(b[i][e], b[i][e], ss);
            dot = fmaf(wa[i][e] * ga[i][e], a[i][e], dot);
            dot = fmaf(wb[i][e] * gb[i][e], b[i][e], dot);
          }
        }
        ss = sum_lanes<L::kLanes>(ss);
        dot = sum_lanes<L::kLanes>(dot);
        const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = dot * rstd * (1.f / D);  // mean of weight g n
        E* dx = hdx.p + (first + t) * hdx.ld + h * hdx.hs;
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const float na = a[i][e] * rstd, nb = b[i][e] * rstd;
            if (live) {
              da[i][e] = fmaf(ga[i][e], na, da[i][e]);
              db[i][e] = fmaf(gb[i][e], nb, db[i][e]);
            }
            a[i][e] = rstd * (wa[i][e] * ga[i][e] - na * m);
            b[i][e] = rstd * (wb[i][e] * gb[i][e] - nb * m);
          }
          if (live) {
            lan::store<kVec>(dx + at[i], a[i]);
            lan::store<kVec>(dx + bt[i], b[i]);
          }
        }
      }
    }
    if (p.part == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::kChunks; ++i) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        sums[group][at[i] + e] = da[i][e];
        sums[group][bt[i] + e] = db[i][e];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < L::kGroups; ++g) s += sums[g][d];
      p.part[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * D + d] = s;
    }
  }
}

// dweight[which][d] = sum over blocks of part, 32 elements a block, in a fixed order.
static __global__ void __launch_bounds__(1024) weight_sum_kernel(const float* part, int blocks, int D, float* dq,
                                                                 float* dk) {
  __shared__ float sums[32][33];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int x = threadIdx.x % 32, y = threadIdx.x / 32;
  const int which = blockIdx.y, d = blockIdx.x * 32 + x;  // D is a multiple of 32
  float s = 0.f;
  for (int b = y; b < blocks; b += 32) s += part[(static_cast<int64_t>(which) * blocks + b) * D + d];
  sums[y][x] = s;
  __syncthreads();
  s = sums[x][y];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
  float* out = which ? dk : dq;
  if (x == 0 && out) out[blockIdx.x * 32 + y] = s;
}

}  // namespace lar
