// la_gated_math.cuh -- element arithmetic of the gated linear recurrence (include/la_gated.h),
// shared by its scan, gradient and decode kernels: the gates, the decay and the input weight of
// one token, for one channel and for two at once.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm103_ptx.cuh"

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

// The hardware's exp2, reciprocal and rsqrt (each within 2^-22 relative) are arranged so that the
// FP32 states keep FP32 accuracy over long memories.  With m = 1 - lambda:
//   u < 1/8    m = u (1 + c1 u + c2 u^2 + c3 u^3), a polynomial fitted to (1 - e^-u) / u for the
//              least relative error on [0, 1/8] (2e-8; evaluated in FP32: 1e-7).  Such a lambda
//              is off by its own rounding alone, and it is here that 1 / m tokens add up its error.
//   otherwise  m = 1 - exp2(-u log2 e), good to 2^-23 / m relative: 1e-6 at 1/8.
// lambda is 1 - m where u < 1/8 and the exp2 itself beyond, so steep slopes keep its digits too (as
// 1 - m it is off by 2e-5 of itself at u = 8, and 0 from 17.4 on).
// Then 1 - lambda^2 = m (1 + lambda) has no cancellation, and beta = w rsqrt(w) with w = 1 - lambda^2
// (kept from rsqrt(0) by the smallest normal number; w = 0 gives beta = 0).
constexpr float kNear = 0.125f;
constexpr float kC1 = -0.4999971091747284f, kC2 = 0.16652604937553406f, kC3 = -0.039715882390737534f;
constexpr float kLeast = 1.17549435e-38f;

// ---------------------------------------------------------------- two channels at once

// Pairs of FP32 values in one 64-bit register pair: one instruction for two channels where the
// operation is an add, a multiply or both.
using lap::f2_fma;
using lap::f2_mul;
using lap::f2_pack;
using lap::f2_sub;
using lap::f2_unpack;
typedef uint64_t f2;

__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 f2_all(float v) { return f2_pack(v, v); }
__device__ __forceinline__ f2 f2_of(float2 v) { return f2_pack(v.x, v.y); }

template <typename F>
__device__ __forceinline__ f2 f2_each(f2 v, F f) {
  const float2 t = f2_unpack(v);
  return f2_pack(f(t.x), f(t.y));
}

__device__ __forceinline__ f2 exp_of2(f2 z) {
  return f2_each(f2_mul(z, f2_all(kLog2e)), [](float v) { return ex2_approx(v); });
}
__device__ __forceinline__ f2 exp_minus2(f2 z) {
  return f2_each(f2_mul(z, f2_all(-kLog2e)), [](float v) { return ex2_approx(v); });
}
// sig(z) from e = exp(-z): 1 at z = +inf, 0 at -inf.
__device__ __forceinline__ f2 sigmoid_of2(f2 e) {
  return f2_each(f2_add(e, f2_all(1.f)), [](float v) { return rcp_approx(v); });
}
__device__ __forceinline__ f2 sigmoid2(f2 z) { return sigmoid_of2(exp_minus2(z)); }
// sig(z) and 1 - sig(z) from e = exp(-z), the latter as e sig(z), so that a gate far open keeps the digits
// of what is left (1 minus a rounded sigmoid is off by 5e-4 of itself at z = 10, and 0 from 17 on).  Where e
// has overflowed, e sig(z) is inf * 0, which the saturating product turns into 0: there `rest` only
// stands in products with `open` = 0.  NaN stays in `open`.
struct Gate {
  f2 open, rest;
};
__device__ __forceinline__ Gate gate_of2(f2 e) {
  const f2 open = sigmoid_of2(e);
  const float2 v = f2_unpack(e), s = f2_unpack(open);
  return {open, f2_pack(__saturatef(v.x * s.x), __saturatef(v.y * s.y))};
}

// A logit from which on sig is 1 in FP32: exp(-40) is 2^-57.7; (1 + exp(40))^2 is 2^115.
constexpr float kOpen = 40.f;
__device__ __forceinline__ f2 at_most_open2(f2 z) {  // NaN stays
  return f2_each(z, [](float v) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v), "f"(kOpen));
    return d;
  });
}
__device__ __forceinline__ uint32_t at_most_open_bf16x2(uint32_t z) {
  const uint32_t open = __float_as_uint(kOpen) >> 16;  // kOpen is a BF16 number
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(z), "r"(open << 16 | open));
  return d;
}

// lambda = exp(-u) of two channels, and m = 1 - lambda.  kSmall: u < kNear is known.
struct Decay {
  f2 lambda, m;
};
template <bool kSmall>
__device__ __forceinline__ Decay decay2(f2 u) {
  f2 p = f2_fma(u, f2_all(kC3), f2_all(kC2));
  p = f2_fma(u, p, f2_all(kC1));
  p = f2_fma(u, p, f2_all(1.f));
  const f2 near = f2_mul(u, p), left = f2_sub(f2_all(1.f), near);
  if constexpr (kSmall) return {left, near};
  const f2 e = f2_each(f2_mul(u, f2_all(-kLog2e)), [](float v) { return ex2_approx(v); });
  const float2 n = f2_unpack(near), l = f2_unpack(left), x = f2_unpack(e), far = f2_unpack(f2_sub(f2_all(1.f), e)),
               v = f2_unpack(u);
  return {f2_pack(v.x < kNear ? l.x : x.x, v.y < kNear ? l.y : x.y),
          f2_pack(v.x < kNear ? n.x : far.x, v.y < kNear ? n.y : far.y)};
}

// Both in one word per channel, the one that has more digits: m, or -lambda where u >= kNear.
template <bool kSmall>
__device__ __forceinline__ f2 fold2(f2 u, const Decay& d) {
  if constexpr (kSmall) return d.m;
  const float2 m = f2_unpack(d.m), l = f2_unpack(d.lambda), v = f2_unpack(u);
  return f2_pack(v.x < kNear ? m.x : -l.x, v.y < kNear ? m.y : -l.y);
}
__device__ __forceinline__ Decay unfold2(f2 kept) {
  const float2 t = f2_unpack(kept), o = make_float2(1.f - fabsf(t.x), 1.f - fabsf(t.y));
  return {f2_pack(signbit(t.x) ? -t.x : o.x, signbit(t.y) ? -t.y : o.y),
          f2_pack(signbit(t.x) ? o.x : t.x, signbit(t.y) ? o.y : t.y)};
}

// 1 - lambda^2 = m (1 + lambda).
__device__ __forceinline__ f2 one_minus_square2(const Decay& d) { return f2_fma(d.m, d.lambda, d.m); }
// w >= 0 kept from 0 (NaN too becomes kLeast).
__device__ __forceinline__ f2 positive2(f2 w) {
  return f2_each(w, [](float v) { return fmaxf(v, kLeast); });
}
__device__ __forceinline__ f2 rsqrt2(f2 w) {
  return f2_each(w, [](float v) { return rsqrt_approx(v); });
}

}  // namespace lag
