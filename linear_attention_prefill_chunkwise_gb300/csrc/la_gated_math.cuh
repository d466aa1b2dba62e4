// la_gated_math.cuh -- element arithmetic of the gated linear recurrence (include/la_gated.h),
// shared by its scan, gradient and decode kernels: the gates, the decay and the input weight of
// one token and channel, and the loads and stores of BF16 and FP32 activations.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace lag {

// ---------------------------------------------------------------- element types

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---------------------------------------------------------------- one token of one channel

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
  float d;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}

// 1 / (1 + exp(-z)); 0 at -inf, 1 at +inf.
template <bool kPrecise>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (kPrecise) return 1.f / (1.f + expf(-z));
  return rcp_approx(1.f + ex2_approx(-kLog2e * z));
}

// What the recurrence and its gradient need of one decay gate: u = slope sig(r), lambda =
// exp(-u), beta = sqrt(1 - lambda^2) and 1 / beta (0 where u = 0: the gradient's convention).
struct Decay {
  float lambda, beta, inv_beta;
};

// kPrecise (FP32 activations) calls the CUDA math functions.  Otherwise (BF16 activations, whose
// own rounding is 2^-9 relative) the hardware approximations, arranged so that the FP32 states
// keep FP32 accuracy over long memories: for u < 1/4, where 1 / (1 - lambda) tokens accumulate
// lambda's error, 1 - lambda comes from its alternating series u - u^2/2! + ... - u^6/6! (the next
// term is u^6 / 7! of the value, 4.8e-8 at u = 1/4), so that lambda is off by its own rounding alone and 1 - lambda^2 =
// (1 - lambda)(1 + lambda) has no cancellation.
template <bool kPrecise>
__device__ __forceinline__ Decay decay_of(float u) {
  Decay d;
  if constexpr (kPrecise) {
    d.lambda = expf(-u);
    d.beta = sqrtf(-expm1f(-2.f * u));
    d.inv_beta = u > 0.f ? 1.f / d.beta : 0.f;
  } else {
    float p = fmaf(u, -1.f / 720.f, 1.f / 120.f);
    p = fmaf(u, -p, 1.f / 24.f);
    p = fmaf(u, -p, 1.f / 6.f);
    p = fmaf(u, -p, 0.5f);
    p = fmaf(u, -p, 1.f);
    const float near = u * p;                             // 1 - lambda
    const float far = 1.f - ex2_approx(-kLog2e * u);
    const float m = u < 0.25f ? near : far;
    d.lambda = 1.f - m;
    const float w = m * (2.f - m);                        // 1 - lambda^2
    const float rs = rsqrt_approx(fmaxf(w, 1.17549435e-38f));
    d.beta = w * rs;
    d.inv_beta = u > 0.f ? rs : 0.f;
  }
  return d;
}

// The gradients of one token and channel, given G = dL/dh_t and h_prev = h_{t-1}.
struct Grads {
  float dx, dr, dg, ds, lambda;  // ds: the token's term of dslopes
};

template <bool kPrecise>
__device__ __forceinline__ Grads grads_of(float x, float r, float g, float slope, float G, float h_prev) {
  const float sr = sigmoid<kPrecise>(r), sg = sigmoid<kPrecise>(g);
  const float u = slope * sr;
  const Decay d = decay_of<kPrecise>(u);
  Grads q;
  const float gs = G * sg;
  q.dx = gs * d.beta;
  q.dg = q.dx * x * (1.f - sg);
  const float du = d.lambda * (gs * x * (d.lambda * d.inv_beta) - G * h_prev);
  q.dr = du * u * (1.f - sr);
  q.ds = du * sr;
  q.lambda = d.lambda;
  return q;
}

}  // namespace lag
