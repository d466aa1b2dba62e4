// la_attention_softmax.cuh -- a thread's row of scores in tensor memory to probabilities, with a
// running maximum and sum, as the forward kernels share it.
//
//     p = 2^(c S - m) with c = scale log2 e,  O += p v,  l += sum p;   o = O / l
// The running maximum and sum of a softmax in one pass (Milakov and Gimelshein, "Online normalizer
// calculation for softmax", 2018), with a maximum m that moves only when a row outgrows it by
// 2^kSlack, so that O is rarely rescaled: any m gives the same quotient as long as p stays in range.  p is
// rounded to BF16 as an operand of the product with v: 2^-8 of each term, no more than the
// output's own rounding; l sums the values before that rounding.  (Outputs are 0.0020 RMS from 64 bits, where
// FP32 probabilities give 0.0015 to 0.0017; a second BF16 operand for the rest of p would cost half as many
// products again.)
#pragma once

#include "la_attention_tiles.cuh"

namespace laa {

constexpr float kSlack = 8.f;  // log2 of how far a row may outgrow its maximum

// Which of a tile's keys a row sees: all, its first `keep`, or (64 at most) those whose bits are set.
enum Seen { kAll, kFirst, kBits };
struct Keys {
  int keep;
  uint32_t bits[2];
};
template <Seen kSeen>
__device__ __forceinline__ bool sees(const Keys& keys, int k) {
  if (kSeen == kAll) return true;
  if (kSeen == kFirst) return k < keys.keep;
  return k < 64 && (keys.bits[(k >> 5) & 1] >> (k & 31) & 1u);
}

// Where a row's maximum begins: the first tile's largest c S, or, where none of those is within FP32 (c S
// overflows for |c| > 1), a value below every other.  From -inf the first score in range would meet inf - inf.
__device__ __forceinline__ float first_maximum(float z) { return fmaxf(z, -3.4e38f); }

// A row's scores of a tile, in registers, and c times the largest (c < 0: smallest) of those that the
// row sees; about -3.4e38 |c| for none.  What it does not see becomes that as well.
template <Seen kSeen>
__device__ __forceinline__ float load_scores(uint32_t t_s, float (&s)[kTile], float c, const Keys& keys) {
  const bool up = c >= 0.f;
  const float out = up ? -3.4e38f : 3.4e38f;
  lap::tmem_ld128(t_s, s);
  if (kSeen != kAll)
#pragma unroll
    for (int k = 0; k < kTile; ++k) s[k] = sees<kSeen>(keys, k) ? s[k] : out;
  float t[4] = {out, out, out, out};
  if (up) {
#pragma unroll
    for (int k = 0; k < kTile; k += 2) t[k / 2 & 3] = lap::max3(t[k / 2 & 3], s[k], s[k + 1]);
    return c * lap::max3(fmaxf(t[0], t[1]), t[2], t[3]);
  }
#pragma unroll
  for (int k = 0; k < kTile; k += 2) t[k / 2 & 3] = lap::min3(t[k / 2 & 3], s[k], s[k + 1]);
  return c * lap::min3(fminf(t[0], t[1]), t[2], t[3]);
}

// Half of the row's probabilities over its scores, in registers and, as BF16, in tensor memory.
template <Seen kSeen>
__device__ __forceinline__ void probabilities(float (&s)[kTile], int half, uint32_t t_p, float c, float m, const Keys& keys) {
  const uint64_t c2 = lap::f2_pack(c, c), m2 = lap::f2_pack(-m, -m);
#pragma unroll
  for (int g = 2 * half; g < 2 * half + 2; ++g) {
    uint32_t u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = 32 * g + 2 * i;
      const float2 z = lap::f2_unpack(lap::f2_fma(lap::f2_pack(s[k], s[k + 1]), c2, m2));
      s[k] = lap::exp2_approx(z.x);
      s[k + 1] = lap::exp2_approx(z.y);
      if (kSeen != kAll) {
        s[k] = sees<kSeen>(keys, k) ? s[k] : 0.f;
        s[k + 1] = sees<kSeen>(keys, k + 1) ? s[k + 1] : 0.f;
      }
      u[i] = lap::pack_bf16x2(s[k], s[k + 1]);
    }
    lap::tmem_st16_nowait(t_p + 16 * g, u);
  }
  lap::tmem_wait_st();
}

// The sum of a row's probabilities, as two partial sums, added to l.
__device__ __forceinline__ void add_sums(const float (&s)[kTile], uint64_t& l) {
  uint64_t t[4] = {l, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kTile; k += 2) t[k / 2 & 3] = lap::f2_add(t[k / 2 & 3], lap::f2_pack(s[k], s[k + 1]));
  l = lap::f2_add(lap::f2_add(t[0], t[1]), lap::f2_add(t[2], t[3]));
}

// Multiplies this thread's row of O in tensor memory.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t t_o, float f) {
  const uint64_t f2 = lap::f2_pack(f, f);
#pragma unroll 1
  for (int g = 0; g < D / 16; ++g) {
    float o[16];
    uint32_t u[16];
    lap::tmem_ld16(t_o + 16 * g, o);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 r = lap::f2_unpack(lap::f2_mul(lap::f2_pack(o[i], o[i + 1]), f2));
      u[i] = __float_as_uint(r.x);
      u[i + 1] = __float_as_uint(r.y);
    }
    lap::tmem_st16_nowait(t_o + 16 * g, u);
  }
  lap::tmem_wait_st();
}

// Where a row outgrows its maximum: the new one, and the factor of what was summed under the old.  Each
// row moves by itself, so that its result does not depend on the rows beside it.
__device__ __forceinline__ float outgrow(float z, float& m, uint64_t& l) {
  const float top = z > m + kSlack ? z : m, f = top == m ? 1.f : lap::exp2_approx(m - top);
  m = top;
  l = lap::f2_mul(l, lap::f2_pack(f, f));
  return f;
}

}  // namespace laa
