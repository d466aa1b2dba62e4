// la_attention_tiles.cuh -- what the tensor-core attention kernels share: tiles of 128 rows in shared
// memory, the products between them, and the walk over a batch's query tiles.
//
// A tile is 128 rows of D BF16 values as D / 64 boxes of 64 columns (128-byte rows, 128-byte
// swizzle, 16 KiB each), the form in which a tensor map with 64-column boxes delivers rows of a
// tensor of heads and in which both a product along D (K-major) and one along the rows (MN-major)
// can read it.
#pragma once

#include "la_attention_params.cuh"
#include "sm103_ptx.cuh"

namespace laa {

constexpr int kTile = 128;                 // rows of a tile: the M of one MMA
constexpr uint32_t kBox = kTile * 128;     // bytes of a box
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D>
using TileMem = uint8_t[D / 64][kBox];

// A tile as an operand whose rows are M or N and whose columns are summed over (desc_rows), and as one
// whose columns are M or N and whose rows are summed over (desc_columns): the low word of the matrix
// descriptor lap::sdesc_sw128 builds; the high word is the same for both.
__device__ __forceinline__ uint32_t desc_rows(const void* tile) {
  return static_cast<uint32_t>(lap::sdesc_sw128(lap::smem_u32(tile), 16, 1024));
}
__device__ __forceinline__ uint32_t desc_columns(const void* tile) {
  return static_cast<uint32_t>(lap::sdesc_sw128(lap::smem_u32(tile), kBox, 1024));
}
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

// The products and commits are whole-warp calls without a branch: one elected lane issues, and
// descriptors stay warp-uniform values to which constants are added.  (A branch to one lane with
// 64-bit descriptors cost 85 cycles an instruction, more than the 64 that one of 128 x 128 x 16 runs.)

// Four instructions of d (+)= a b^T along 64 columns of two tiles (16 columns, 32 bytes, each).
template <uint32_t kIdesc>
__device__ __forceinline__ void mma4_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b32 x, y;\n\t.reg .b64 s, t;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 s, {%1, %3};\n\tmov.b64 t, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], s, t, %4, p;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\tmov.b64 s, {x, %3};\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], s, t, %4, 1;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\tmov.b64 s, {x, %3};\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], s, t, %4, 1;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\tmov.b64 s, {x, %3};\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], s, t, %4, 1;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHigh), "r"(kIdesc), "r"(accumulate)
      : "memory");
}
// One instruction of d += a b^T, 16 columns of two tiles.
template <uint32_t kIdesc>
__device__ __forceinline__ void mma1_rows(uint32_t d, uint32_t a, uint32_t b) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 s, t;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "mov.b64 s, {%1, %3};\n\tmov.b64 t, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], s, t, %4, 1;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHigh), "r"(kIdesc)
      : "memory");
}
// Four instructions of d (+)= a b with 64 summed elements of a in tensor memory (8 columns for each
// instruction, the second two kGap columns behind the first) and 64 rows of b (16 rows, 2048 bytes, each).
template <uint32_t kIdesc, uint32_t kGap = 16>
__device__ __forceinline__ void mma4_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b32 x, y;\n\t.reg .b64 t;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 t, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], t, %4, p;\n\t"
      "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], t, %4, 1;\n\t"
      "add.u32 x, %1, %6;\n\tadd.u32 y, %2, 256;\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], t, %4, 1;\n\t"
      "add.u32 x, %1, %7;\n\tadd.u32 y, %2, 384;\n\tmov.b64 t, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], t, %4, 1;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHigh), "r"(kIdesc), "r"(accumulate), "n"(kGap), "n"(kGap + 8)
      : "memory");
}
// Arrives once on `bar` when every product issued so far has completed.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(lap::smem_u32(bar))
      : "memory");
}

// d = a b^T over D columns: scores, dP.
template <int D>
__device__ __forceinline__ void product_rows(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = lap::idesc_bf16_f32(kTile, kTile, false, false);
#pragma unroll
  for (int h = 0; h < D / 64; ++h) mma4_rows<id>(d, a + h * (kBox >> 4), b + h * (kBox >> 4), h > 0);
}
// d (+)= a b with a [128 rows, 128 summed] BF16 in tensor memory and b's rows summed; its two halves
// along the sum apart.  a lies in four parts of 16 columns, kGap columns from one to the next.
template <int D, int kGap = 16>
__device__ __forceinline__ void half_product_tmem(uint32_t d, uint32_t a, uint32_t b, int half, bool accumulate) {
  constexpr uint32_t id = lap::idesc_bf16_f32(kTile, D, false, true);
  mma4_tmem<id, kGap>(d, a + half * 2 * kGap, b + half * 512, accumulate);
}
template <int D, int kGap = 16>
__device__ __forceinline__ void product_tmem(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  half_product_tmem<D, kGap>(d, a, b, 0, accumulate);
  half_product_tmem<D, kGap>(d, a, b, 1, true);
}

// A value that is the same in every lane, known to the compiler as such.
template <typename T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Whole-warp wait; false once the block gives up: after a wait of kWaitLimitNs, which sets *abort.
// (Inline: a kernel that moves registers between its warpgroups makes no calls.  A build whose limit
// is short, so that ordinary waits exceed it, polls, as try_wait sits out ordinary latencies itself.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  constexpr bool kPoll = lap::kWaitLimitNs < 1000000ull;
  constexpr uint32_t kEvery = kPoll ? 1 : 16;  // the clock is slow to read: not in an ordinary wait
  bool ok = kPoll ? lap::mbar_test(bar, parity) : lap::mbar_try_wait(bar, parity);
  uint64_t t0 = 0;
  for (uint32_t i = 1; !ok; ++i) {
    ok = kPoll ? lap::mbar_test(bar, parity) : lap::mbar_try_wait(bar, parity);
    if (i % kEvery == 0u && !ok) {
      if (*abort) break;
      const uint64_t now = lap::globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > lap::kWaitLimitNs) {
        *abort = 1;
        break;
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}
// lap::mbar_wait_drain, inline.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = lap::globaltimer_ns();
  while (!lap::mbar_try_wait(bar, parity))
    if (lap::globaltimer_ns() - t0 > lap::kDrainLimitNs) return;
}
// One arrival for the warp, after all of its lanes' work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) lap::mbar_arrive(bar);
}

// A tile of `rows` query rows of a sequence, for one head; len < 0 ends the list.
struct Item {
  int lo, len, tile, head;
};
__device__ __forceinline__ Item uniform(const Item& it) {
  return {uniform(it.lo), uniform(it.len), uniform(it.tile), uniform(it.head)};
}

// The block's items: each round of gridDim.x items goes to the blocks in order, every other one
// backwards, and the costliest items come first, so that the sums are alike.  Heads are innermost, so
// that blocks that run side by side read the same keys.  Tiles are taken by level: level x holds, of
// every sequence of more than x tiles, the one that x others of it cost less than (tile x, which sees
// x + 1 tiles of keys; kAscending: the one that x tiles follow), the highest level first.  Packed
// sequences are walked 32 at a time by the warp's lanes, by level within those.  Whole-warp calls.
// (Packed sequences one after the other, 24 of up to 2047 tokens of 16 heads: the busiest block had
// 1.25 times the mean, by level 1.02.)
template <bool kAscending>
struct ItemWalk {
  int64_t round = 0;
  int n0 = 0, rows, heads;
  int64_t before = 0;              // tiles before the level
  int lo = 0, len = 0, tiles = 0;  // this lane's sequence n0 + lane
  int level = -1;

  __device__ ItemWalk(int rows, int heads) : rows(rows), heads(heads) {}

  __device__ __forceinline__ void load(const PrefillParams& p, int lane) {
    const int n = n0 + lane;
    int hi = 0;
    lo = 0;
    if (n < p.N && !sequence_rows(p, n, lo, hi) && blockIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, kErrSeqlens);
    len = hi - lo;
    tiles = (len + rows - 1) / rows;
    level = __reduce_max_sync(0xFFFFFFFFu, tiles) - 1;
  }

  __device__ __forceinline__ Item take(const PrefillParams& p, int lane) {
    const int64_t next = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    const int64_t t = next / heads;
    Item it{0, -1, 0, static_cast<int>(next - t * heads)};
    if (!p.cu_seqlens) {
      ++round;
      const int tiles_each = (p.T + rows - 1) / rows;
      if (t < static_cast<int64_t>(p.N) * tiles_each) {
        const int down = static_cast<int>(t / p.N);
        it.lo = (static_cast<int>(t) - down * p.N) * p.T;
        it.len = p.T;
        it.tile = kAscending ? down : tiles_each - 1 - down;
      }
      return it;
    }
    if (round == 0) load(p, lane);
    ++round;
    for (;;) {
      while (level < 0) {
        if ((n0 += 32) >= p.N) return it;
        load(p, lane);
      }
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, tiles > level);
      const int at = static_cast<int>(min(t - before, static_cast<int64_t>(32)));
      if (at < __popc(here)) {
        const int l = __fns(here, 0, at + 1);
        it.lo = __shfl_sync(0xFFFFFFFFu, lo, l);
        it.len = __shfl_sync(0xFFFFFFFFu, len, l);
        it.tile = kAscending ? __shfl_sync(0xFFFFFFFFu, tiles, l) - 1 - level : level;
        return it;
      }
      before += __popc(here);
      --level;
    }
  }
};

// Bits of a packed pair of BF16 values that are infinite or NaN (bit 15, bit 31).
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// Makes a row of a box of values harmless where its probabilities are zero because of a mask: 0 * inf
// is NaN.  A row behind the sequence becomes zero; in a row within it, what is not finite becomes
// zero and is added again by `restore`.  Returns whether the row held such a value.
__device__ __forceinline__ bool clean_box(uint8_t (&box)[kBox], int row, bool behind) {
  uint4* at = reinterpret_cast<uint4*>(box + row * 128);
  if (behind) {
#pragma unroll
    for (int c = 0; c < 8; ++c) at[c] = make_uint4(0, 0, 0, 0);
    return false;
  }
  uint32_t any = 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v = at[c ^ (row & 7)];  // lanes of neighbouring rows read different banks
    any |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
  }
  if (!any) return false;
  uint32_t* w = reinterpret_cast<uint32_t*>(at);
  for (int c = 0; c < 32; ++c) {
    const uint32_t f = not_finite(w[c]);
    w[c] &= ~((f >> 15 & 1u) * 0xFFFFu) & ~((f >> 31) * 0xFFFF0000u);
  }
  return true;
}
template <int D>
__device__ __forceinline__ bool clean_row(TileMem<D>& tile, int row, bool behind) {
  bool found = false;
#pragma unroll
  for (int b = 0; b < D / 64; ++b) found |= clean_box(tile[b], row, behind);
  return found;
}

// Adds the values of a row that are not finite to a part of an output row.
template <int N>
__device__ __forceinline__ void restore(float (&o)[N], const bf16* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float x = __bfloat162float(v[i]);
    if (!isfinite(x)) o[i] += x;
  }
}

// An output row's part of 32 columns.
__device__ __forceinline__ void store_row32(bf16* p, const float (&o)[32]) {
  uint4* out = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = make_uint4(lap::pack_bf16x2(o[8 * i], o[8 * i + 1]), lap::pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                        lap::pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), lap::pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
}

}  // namespace laa
