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
// What bounds it beside the bytes is the number of instructions and the bytes in flight, so elements go
// in packed FP32 pairs, a thread's pointers move from head to head without a division, and rows
// are read ahead into shared memory.  16384 tokens, heads of 128 BF16: forward, 64 + 8 heads, 95 us (0.95 of
// the copy rate); gradients, 32 + 4 heads, 82 us (0.82).
//
// The angle of a pair, in turns, is position * frequency / 2 pi modulo 1: the frequency is scaled
// to a 64-bit fraction of a turn, and the product wraps around by itself.  Its error is |position|
// (1 + |frequency|) 2^-64 turns, 2^-24 of a turn's half after the conversion to FP32.
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
  int tokens, heads[2], R, per_block;  // tokens of a block
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
  int tokens, heads[2], R, per_block;
};

template <typename E, int kVec, int D>
struct Layout {
  static constexpr int kPairs = D / (2 * kVec);  // groups of kVec pairs in a head
  static constexpr int kLanes = kPairs < 32 ? kPairs : 32;
  static constexpr int kChunks = kPairs / kLanes;
  static constexpr int kGroups = kThreads / kLanes;  // heads that a block holds at once
};

// Where the two vectors of group c begin, so that each access of a warp covers whole sectors: neighbouring groups
// have neighbouring vectors also where elements do not rotate or rotate with their neighbours (16384 tokens
// of 64 + 8 heads of 128, half of each rotated: 105 us with the two vectors of the other half side by side;
// neighbours rotated: 126 us, gradients 239).
template <int kVec, int D, bool kNear>
__device__ __forceinline__ void places(int c, int R, int& a, int& b) {
  const int rotated = R / (2 * kVec);
  if (kNear && kVec > 1) {  // each vector holds whole pairs
    a = kVec * c;
    b = a + D / 2;
  } else if (c >= rotated) {
    a = R + kVec * (c - rotated);
    b = a + (D - R) / 2;
  } else if (kNear) {
    a = 2 * c;
    b = a + 1;
  } else {
    a = kVec * c;
    b = a + R / 2;
  }
}

// A frequency as a fraction of a turn per position, in units of 2^-64 turns, cut: mantissa times 2^64 / 2 pi, 88
// bits, shifted by the exponent.  (In integers: FP64 instructions for this cost more than the rest of an angle.)
__device__ __forceinline__ uint64_t turn_units(float inv_freq) {
  constexpr uint64_t kUnits = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
  const uint32_t bits = __float_as_uint(inv_freq), field = bits >> 23 & 255u;
  const uint64_t m = (bits & 0x7FFFFFu) | (field ? 0x800000u : 0u);
  const int down = 150 - static_cast<int>(max(field, 1u));
  const uint64_t lo = m * kUnits, hi = __umul64hi(m, kUnits);
  uint64_t r;
  if (down <= 0)
    r = down > -64 ? lo << -down : 0;
  else if (down < 64)
    r = lo >> down | hi << (64 - down);
  else
    r = down < 128 ? hi >> (down - 64) : 0;
  return bits >> 31 ? 0 - r : r;
}

// cos and sin of the angle of pair i at a position.
__device__ __forceinline__ float2 angle(int32_t position, float inv_freq) {
  const int64_t phase = static_cast<int64_t>(turn_units(inv_freq) * static_cast<uint64_t>(static_cast<int64_t>(position)));
  float s, c;
  sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);  // half turns
  return make_float2(c, s);
}

// kVec neighbouring elements as packed FP32 pairs; a single one is a pair whose other half is zero.
template <int kVec>
struct Vec {
  static constexpr int kN = kVec > 1 ? kVec / 2 : 1;
  uint64_t v[kN];
};
template <int kVec>
__device__ __forceinline__ Vec<kVec> mul(const Vec<kVec>& x, const Vec<kVec>& y) {
  Vec<kVec> r;
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) r.v[i] = lap::f2_mul(x.v[i], y.v[i]);
  return r;
}
template <int kVec>
__device__ __forceinline__ Vec<kVec> mul(const Vec<kVec>& x, uint64_t f) {
  Vec<kVec> r;
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) r.v[i] = lap::f2_mul(x.v[i], f);
  return r;
}
template <int kVec>
__device__ __forceinline__ void add_product(Vec<kVec>& sum, const Vec<kVec>& x, const Vec<kVec>& y) {
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) sum.v[i] = lap::f2_fma(x.v[i], y.v[i], sum.v[i]);
}
template <int kVec>
__device__ __forceinline__ void add_dot(uint64_t& sum, const Vec<kVec>& x, const Vec<kVec>& y) {
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) sum = lap::f2_fma(x.v[i], y.v[i], sum);
}
__device__ __forceinline__ uint64_t both(float f) { return lap::f2_pack(f, f); }
__device__ __forceinline__ float halves_sum(uint64_t v) {
  const float2 f = lap::f2_unpack(v);
  return f.x + f.y;
}

template <int kVec>
__device__ __forceinline__ Vec<kVec> load_floats(const float* p) {  // aligned for kVec > 1
  Vec<kVec> r;
  if constexpr (kVec == 1) {
    r.v[0] = lap::f2_pack(*p, 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 f = reinterpret_cast<const float4*>(p)[i];
      r.v[2 * i] = lap::f2_pack(f.x, f.y);
      r.v[2 * i + 1] = lap::f2_pack(f.z, f.w);
    }
  }
  return r;
}
template <int kVec>
__device__ __forceinline__ Vec<kVec> load_weight(const float* w, int at) {
  Vec<kVec> r;
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i)
    r.v[i] = lap::f2_pack(w ? __ldg(w + at + 2 * i) : 1.f, kVec == 1 ? 0.f : w ? __ldg(w + at + (kVec == 1 ? 0 : 2 * i + 1)) : 1.f);
  return r;
}

// kVec elements as loaded: the next head's are on their way while one is computed.
template <typename E, int kVec>
struct Raw {
  using T = std::conditional_t<kVec == 1, E, uint4>;
  T v;
  __device__ __forceinline__ void load(const E* p) { v = *reinterpret_cast<const T*>(p); }
  __device__ __forceinline__ Vec<kVec> expand() const {
    Vec<kVec> r;
    if constexpr (kVec == 1) {
      r.v[0] = lap::f2_pack(static_cast<float>(v), 0.f);
    } else if constexpr (kVec == 4) {
      r.v[0] = lap::f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
      r.v[1] = lap::f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
    } else {
      r.v[0] = lap::bf16x2_to_f2(v.x), r.v[1] = lap::bf16x2_to_f2(v.y);
      r.v[2] = lap::bf16x2_to_f2(v.z), r.v[3] = lap::bf16x2_to_f2(v.w);
    }
    return r;
  }
};
// The rows that a thread reads ahead, kN vectors of each.  With 16-byte vectors they wait in shared
// memory, kDepth - 1 rows ahead (a thread reads only what it has copied itself, so nothing is waited
// for but its own copies); single elements in registers, one row ahead.  Of one row ahead in
// registers, 32 KiB per SM, the gradients came to 0.6 of the copy rate.
constexpr int kDepth = 4;
template <typename E, int kVec, int kN>
struct Ahead {
  static constexpr int kRows = kVec > 1 ? kDepth - 1 : 1;                    // rows ahead
  static constexpr int kBytes = kVec > 1 ? kDepth * kN * kThreads * 16 : 0;  // of shared memory
  Raw<E, kVec> one[kVec > 1 ? 1 : kN];
  uint4* mine;  // [kDepth][kN][kThreads]
  int in = 0, out = 0;
  __device__ explicit Ahead(void* ring) : mine(static_cast<uint4*>(ring) + threadIdx.x) {}
  __device__ __forceinline__ void load(int i, const E* p) {
    if constexpr (kVec > 1)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(lap::smem_u32(mine + (in * kN + i) * kThreads)),
                   "l"(__cvta_generic_to_global(p))
                   : "memory");
    else
      one[i].load(p);
  }
  // a row's loads have been issued (or there was none)
  __device__ __forceinline__ void close() {
    if constexpr (kVec > 1) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      in = in + 1 == kDepth ? 0 : in + 1;
    }
  }
  // the next row has arrived
  __device__ __forceinline__ void open() {
    if constexpr (kVec > 1) asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
  }
  __device__ __forceinline__ Vec<kVec> get(int i) const {
    if constexpr (kVec > 1) {
      Raw<E, kVec> r;
      r.v = mine[(out * kN + i) * kThreads];
      return r.expand();
    } else {
      return one[i].expand();
    }
  }
  __device__ __forceinline__ void drop() {
    if constexpr (kVec > 1) out = out + 1 == kDepth ? 0 : out + 1;
  }
};

template <typename E, int kVec>
__device__ __forceinline__ void store(E* p, const Vec<kVec>& x) {
  float f[kVec];
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) {
    const float2 t = lap::f2_unpack(x.v[i]);
    f[kVec == 1 ? 0 : 2 * i] = t.x;
    if (kVec > 1) f[(2 * i + 1) % kVec] = t.y;
  }
  lan::store<kVec>(p, f);
}

// The rotation of a vector of neighbouring pairs by the angles of cos[] and sin[]; kBack turns back.
template <int kVec, bool kBack>
__device__ __forceinline__ void turn_near(Vec<kVec>& v, const float* cos, const float* sin) {
#pragma unroll
  for (int i = 0; i < Vec<kVec>::kN; ++i) {
    // (x, y) (c, c) + (y, x) (-s, s)
    const float2 f = lap::f2_unpack(v.v[i]);
    const float s = kBack ? -sin[i] : sin[i];
    v.v[i] = lap::f2_fma(v.v[i], both(cos[i]), lap::f2_mul(lap::f2_pack(f.y, f.x), lap::f2_pack(-s, s)));
  }
}
// That of a group's elements, which begin at a0 and b0 (places), by the angles of their token.
template <int kVec, bool kNear, bool kBack>
__device__ __forceinline__ void turn(Vec<kVec>& a, Vec<kVec>& b, int a0, int b0, const float* cos, const float* sin, int R) {
  constexpr uint64_t kBoth = 0x8000000080000000ull;  // sign bits
  if (kNear && kVec > 1) {
    if (a0 < R) turn_near<kVec, kBack>(a, cos + a0 / 2, sin + a0 / 2);
    if (b0 < R) turn_near<kVec, kBack>(b, cos + b0 / 2, sin + b0 / 2);
  } else if (a0 < (kNear ? R : R / 2)) {
    const int pair = kNear ? a0 / 2 : a0;  // the first
    const Vec<kVec> c = load_floats<kVec>(cos + pair), s = load_floats<kVec>(sin + pair);
#pragma unroll
    for (int i = 0; i < Vec<kVec>::kN; ++i) {
      const uint64_t x = a.v[i], y = b.v[i], minus = s.v[i] ^ kBoth;
      a.v[i] = lap::f2_fma(x, c.v[i], lap::f2_mul(y, kBack ? s.v[i] : minus));
      b.v[i] = lap::f2_fma(x, kBack ? minus : s.v[i], lap::f2_mul(y, c.v[i]));
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// Cosines and sines of a block's tokens into shared memory, [tokens][R / 2] each.
template <typename P>
__device__ __forceinline__ void fill_angles(const P& p, float* cos, float* sin, int64_t first, int count) {
  const int half = p.R / 2;
  for (int i = threadIdx.x; i < count * half; i += kThreads) {
    const int t = i / half;
    const float2 cs = angle(__ldg(p.positions + first + t), __ldg(p.inv_freq + (i - t * half)));
    cos[i] = cs.x;
    sin[i] = cs.y;
  }
}

// Heads kGroups rows apart, in the order (token, head): a pointer's steps, and the token within the tile.
struct Step {
  int tokens, heads;  // kGroups rows are so many tokens and heads
  __device__ __forceinline__ Step(int groups, int heads_of) : tokens(groups / heads_of), heads(groups % heads_of) {}
};
// Where a thread's rows are: token and head, `rows` rows on each time.
struct Place {
  int t, h;
  __device__ __forceinline__ bool next(const Step& s, int heads) {
    h += s.heads;
    const bool wrapped = h >= heads;
    if (wrapped) h -= heads;
    t += s.tokens + wrapped;
    return wrapped;
  }
};
template <typename E>
struct Walk {
  E* p;
  int64_t step, back;
  __device__ __forceinline__ Walk(const Heads<E>& h, int64_t t, int head, int heads, const Step& s)
      : p(h.p + t * h.ld + head * h.hs), step(s.tokens * h.ld + s.heads * h.hs), back(h.ld - heads * h.hs) {}
  __device__ __forceinline__ void next(bool wrapped) { p += wrapped ? step + back : step; }
};

template <typename E, int kVec, int D, bool kNear>
__global__ void __launch_bounds__(kThreads, kVec > 1 ? 3 : 1) norm_rope_fwd_kernel(const FwdParams<E> p) {
  using L = Layout<E, kVec, D>;
  extern __shared__ __align__(16) float angles[];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_block;
  const int count = static_cast<int>(min(static_cast<int64_t>(p.per_block), p.tokens - first));
  const int lane = threadIdx.x % L::kLanes, group = threadIdx.x / L::kLanes, half = p.R / 2;
  using Rows = Ahead<E, kVec, 2 * L::kChunks>;
  float *cos = angles + Rows::kBytes / 4, *sin = cos + p.per_block * half;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = p.heads[which], rows = count * heads;
    const Step step(L::kGroups, heads);
    Place now{group / heads, group % heads}, then = now;
    Walk<const E> x(p.x[which], first + now.t, now.h, heads, step);
    Walk<E> y(p.y[which], first + now.t, now.h, heads, step);
    int at[L::kChunks], bt[L::kChunks];
    Vec<kVec> wa[L::kChunks], wb[L::kChunks];
#pragma unroll
    for (int i = 0; i < L::kChunks; ++i) places<kVec, D, kNear>(lane + 32 * i, p.R, at[i], bt[i]);
    Rows in(angles);
    auto fetch = [&](int r) {
      if (r < rows)
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
          in.load(2 * i, x.p + at[i]);
          in.load(2 * i + 1, x.p + bt[i]);
        }
      in.close();
      x.next(then.next(step, heads));
    };
#pragma unroll
    for (int k = 0; k < Rows::kRows; ++k) fetch(group + k * L::kGroups);
#pragma unroll
    for (int i = 0; i < L::kChunks; ++i) {
      wa[i] = load_weight<kVec>(p.weight[which], at[i]);
      wb[i] = load_weight<kVec>(p.weight[which], bt[i]);
    }
    if (which == 0) {
      fill_angles(p, cos, sin, first, count);
      __syncthreads();
    }
    // every lane of a warp takes the same number of turns (the sums are over whole warps)
    for (int r = group; r - group < rows; r += L::kGroups) {
      const bool live = r < rows;
      Vec<kVec> a[L::kChunks], b[L::kChunks];
      const float *c = cos + now.t * half, *s = sin + now.t * half;
      in.open();
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        a[i] = in.get(2 * i);
        b[i] = in.get(2 * i + 1);
      }
      in.drop();
      fetch(r + Rows::kRows * L::kGroups);
      uint64_t ss = 0;
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        add_dot(ss, a[i], a[i]);
        add_dot(ss, b[i], b[i]);
      }
      const uint64_t rstd = both(rsqrtf(sum_lanes<L::kLanes>(halves_sum(ss)) * (1.f / D) + p.eps));
#pragma unroll
      for (int i = 0; i < L::kChunks; ++i) {
        a[i] = mul(mul(a[i], rstd), wa[i]);
        b[i] = mul(mul(b[i], rstd), wb[i]);
        if (live) {
          turn<kVec, kNear, false>(a[i], b[i], at[i], bt[i], c, s, p.R);
          store(y.p + at[i], a[i]);
          store(y.p + bt[i], b[i]);
        }
      }
      y.next(now.next(step, heads));
    }
  }
}

// The gradients.  A block walks over its share of the tokens, first all of its queries, then
// all of its keys, and keeps the sums for the weight gradients of its threads' own elements in registers.
template <typename E, int kVec, int D, bool kNear>
__global__ void __launch_bounds__(kThreads, kVec > 1 ? 2 : 1) norm_rope_bwd_kernel(const BwdParams<E> p) {
  using L = Layout<E, kVec, D>;
  extern __shared__ __align__(16) float angles[];
  __shared__ float sums[L::kGroups][D];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int lane = threadIdx.x % L::kLanes, group = threadIdx.x / L::kLanes, half = p.R / 2;
  using Rows = Ahead<E, kVec, 4 * L::kChunks>;
  float *cos = angles + Rows::kBytes / 4, *sin = cos + p.per_block * half;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int heads = p.heads[which];
    const Step step(L::kGroups, heads);
    int at[L::kChunks], bt[L::kChunks];
    Vec<kVec> wa[L::kChunks], wb[L::kChunks], da[L::kChunks] = {}, db[L::kChunks] = {};
#pragma unroll
    for (int i = 0; i < L::kChunks; ++i) {
      places<kVec, D, kNear>(lane + 32 * i, p.R, at[i], bt[i]);
      wa[i] = load_weight<kVec>(p.weight[which], at[i]);
      wb[i] = load_weight<kVec>(p.weight[which], bt[i]);
    }
    const int64_t start = static_cast<int64_t>(blockIdx.x) * p.tokens / gridDim.x;
    const int64_t stop = static_cast<int64_t>(blockIdx.x + 1) * p.tokens / gridDim.x;
    for (int64_t first = start; first < stop; first += p.per_block) {
      const int count = static_cast<int>(min(static_cast<int64_t>(p.per_block), stop - first));
      const int rows = count * heads;
      Place now{group / heads, group % heads}, then = now;
      Walk<const E> x(p.x[which], first + now.t, now.h, heads, step), dy(p.dy[which], first + now.t, now.h, heads, step);
      Walk<E> dx(p.dx[which], first + now.t, now.h, heads, step);
      Rows in(angles);
      auto fetch = [&](int r) {
        if (r < rows)
#pragma unroll
          for (int i = 0; i < L::kChunks; ++i) {
            in.load(4 * i, x.p + at[i]);
            in.load(4 * i + 1, x.p + bt[i]);
            in.load(4 * i + 2, dy.p + at[i]);
            in.load(4 * i + 3, dy.p + bt[i]);
          }
        in.close();
        const bool wrapped = then.next(step, heads);
        x.next(wrapped);
        dy.next(wrapped);
      };
#pragma unroll
      for (int k = 0; k < Rows::kRows; ++k) fetch(group + k * L::kGroups);
      if (which == 0 || stop - start > p.per_block) {  // (the keys' tokens are the queries')
        __syncthreads();
        fill_angles(p, cos, sin, first, count);
        __syncthreads();
      }
      for (int r = group; r - group < rows; r += L::kGroups) {
        const bool live = r < rows;
        Vec<kVec> a[L::kChunks], b[L::kChunks], ga[L::kChunks], gb[L::kChunks];
        const float *c = cos + now.t * half, *s = sin + now.t * half;
        in.open();
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
          a[i] = in.get(4 * i);
          b[i] = in.get(4 * i + 1);
          ga[i] = in.get(4 * i + 2);
          gb[i] = in.get(4 * i + 3);
        }
        in.drop();
        fetch(r + Rows::kRows * L::kGroups);
        uint64_t ss = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < L::kChunks; ++i) {
            if (live) turn<kVec, kNear, true>(ga[i], gb[i], at[i], bt[i], c, s, p.R);
          add_dot(ss, a[i], a[i]);
          add_dot(ss, b[i], b[i]);
          add_dot(dot, mul(wa[i], ga[i]), a[i]);
          add_dot(dot, mul(wb[i], gb[i]), b[i]);
        }
        const float rstd = rsqrtf(sum_lanes<L::kLanes>(halves_sum(ss)) * (1.f / D) + p.eps);
        const float m = sum_lanes<L::kLanes>(halves_sum(dot)) * rstd * (1.f / D);  // mean of weight g n
        const uint64_t r2 = both(rstd), m2 = both(-rstd * m);
        if (live) {
#pragma unroll
          for (int i = 0; i < L::kChunks; ++i) {
            // dx = rstd weight g - n rstd m
            const Vec<kVec> na = mul(a[i], r2), nb = mul(b[i], r2);
            add_product(da[i], ga[i], na);
            add_product(db[i], gb[i], nb);
            Vec<kVec> oa = mul(na, m2), ob = mul(nb, m2);
            add_product(oa, mul(ga[i], r2), wa[i]);
            add_product(ob, mul(gb[i], r2), wb[i]);
            store(dx.p + at[i], oa);
            store(dx.p + bt[i], ob);
          }
        }
        dx.next(now.next(step, heads));
      }
    }
    if (p.part == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::kChunks; ++i)
#pragma unroll
      for (int e = 0; e < Vec<kVec>::kN; ++e) {
        const float2 fa = lap::f2_unpack(da[i].v[e]), fb = lap::f2_unpack(db[i].v[e]);
        sums[group][at[i] + 2 * e] = fa.x;
        sums[group][bt[i] + 2 * e] = fb.x;
        if (kVec > 1) {
          sums[group][at[i] + 2 * e + 1] = fa.y;
          sums[group][bt[i] + 2 * e + 1] = fb.y;
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
