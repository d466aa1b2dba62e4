// la_attention_bwd.cuh -- gradients of causal attention (include/la_attention.h) on the tensor cores.
//
// With p = 2^(c q.k - lse log2 e), c = scale log2 e, and delta_t = sum_d dO o:
//     dS = p (dO.v - delta),   dv_j = sum_t p dO_t,   dk_j = scale sum_t dS q_t,   dq_t = scale sum_j dS k_j
// p and dS are rounded to BF16 as operands of those products, 2^-8 of each term, as much as the gradients'
// own rounding (0.0024 RMS from 64 bits, where FP32 ones give 0.0017); what is summed and subtracted is FP32.
// Two kernels, so that every sum stays in tensor memory, in one order, without atomics or partial
// sums in memory.  (A single pass would save two of the seven products and add dq in memory in FP32, in an
// order that changes or in turns that blocks wait for; what the latter costs has not been measured.)
//   dk, dv: a block owns 128 keys and walks over the rows that see them, of every head of the group.
//     K Q^T and V dO^T give scores and dP transposed, keys along the lanes, so that p and dS, written
//     back over them as BF16, are operands from tensor memory of p^T dO and dS^T Q.
//   dq: a block owns 128 rows and walks over the keys that they see: Q K^T, dO V^T, then dS K.
// Four warpgroups share each tile of scores, 32 columns each (a thread has one row).  Warp 16 issues the
// products in an order that leaves a product or two to run whenever the warpgroups work:
//   dk, dv:  p^T dO (n), S (n + 1; D = 64: n + 2), dS^T Q (n), dP (n + 1)
//   dq:      S (n + 1), dP (n + 1), dS K (n)
// Warp 17 loads: a pair of tiles that stays for the item, and rings for the operands that pass, as long as
// each is in use.  Warp 18 brings lse and delta of the rows that pass (dk, dv).
//
// Where a batch has few key/value heads and tiles for the SMs, a group's heads are shared out among
// several items, whose FP32 sums a last kernel adds in order.
//
// Bound: the tensor cores at D = 128 (2 x 8192 tokens, 32 heads of 128 on 4: 2.43 ms in a row, the seven
// products at 1.58 PFLOP/s under the power limit; 2.19 ms when cool); at D = 64 the warpgroups' way from
// scores to probabilities to dS (24 packed sequences of up to 2047 tokens, 16 heads: 0.45 ms; 2100 cycles
// per tile of scores and SM for dk and dv, 1474 for dq, of which the products take 1152 and 768 and the
// warps' instructions 800: what is left is the latency of barriers and tensor memory, which all warps meet
// at the same time).  There, two teams of eight warps with 64 columns a thread, a tile each in turn, were no
// faster: tensor memory has room for one dP, which each team holds for most of its tile (dk, dv 235 us
// against 240 for 2 x 4096 tokens of 32 heads on 8; dq 245 against 202); neither was taking scores and dP out of
// tensor memory before the last stores there are done (319 against 266).  Two blocks per SM with 64 rows
// passing at a time took 428 us for the packed case, but 438 against 430 for the other, and where items are
// few 110 against 75 (4096 tokens, 8 heads of 64 on 1).
#pragma once

#include "la_attention_softmax.cuh"

namespace laa {

constexpr int kParts = 4, kColumns = kTile / kParts;  // warpgroups of a tile of scores, columns of each
constexpr int kBwdThreads = kParts * kTile + 128, kBwdItems = 2, kDeltaThreads = 256;

// dk, dv: a thread needs lse and delta of 32 rows per tile, and 512 threads that read them from shared memory
// keep it busy for 1024 cycles.  Where shared memory has room (D = 64) they go through the products instead: 16
// columns more of Q (dO) hold -lse / scale (-delta) in three BF16 parts, 24 bits, against ones in K (V).
// (2 x 4096 tokens, 32 heads of 64 on 8, dk and dv: 266 us without, 258 with.)
template <int D>
constexpr bool kFold = D == 64;
struct FoldedStats {
  uint8_t stats[2][kBox];  // columns 0 .. 2: -lse log2 e / c, 16 .. 18: -delta of the rows
  uint8_t ones[kBox];      // 1 in those columns, 0 up to 31
};
struct PlainStats {
  float lse[2][kTile], delta[2][kTile];
};

template <int D>
struct alignas(1024) BwdShared {
  static constexpr uint32_t kLong = D == 64 ? 4 : 3, kBrief = D == 64 ? 3 : 2;  // slots of the rings
  TileMem<D> own[2];         // dk, dv: K, V of the item; dq: Q, dO
  TileMem<D> long_[kLong];   // dk, dv: Q;  dq: K     (in use by two products)
  TileMem<D> brief[kBrief];  // dk, dv: dO; dq: V
  std::conditional_t<kFold<D>, FoldedStats, PlainStats> st;  // dk, dv
  Item items[kBwdItems];
  uint64_t item_full[kBwdItems], item_empty[kBwdItems];
  uint64_t own_full, own_empty, long_full[kLong], long_empty[kLong], brief_full[kBrief], brief_empty[kBrief];
  uint64_t stat_full[2], stat_empty[2];
  uint64_t s_full[2], s_free, dp_full, dp_free, p_ready[2], ds_ready, acc_full, acc_free, final_bar;
  uint32_t tmem;
  int abort;
};

struct BwdMaps {
  CUtensorMap q, k, v, dout;
};

// What an item of either kernel walks over: tile n is rows (keys) of tile `first + n % each`, of head
// `head + n / each`; `own` is the head of the item's own tiles.  (dk, dv: items go by key/value head and
// by part of its group's heads.)
struct Passes {
  int first, each, count, head, own;
};
template <bool kDq>
__device__ __forceinline__ Passes passes_of(const PrefillParams& p, const Item& it) {
  const int tiles = (it.len + kTile - 1) / kTile, group = p.H / p.HK;
  if (kDq) return {0, it.tile + 1, it.tile + 1, it.head / group, it.head};
  const int hk = it.head / p.splits, part = it.head - hk * p.splits, most = (group + p.splits - 1) / p.splits;
  return {it.tile, tiles - it.tile, (tiles - it.tile) * min(most, group - part * most), hk * group + part * most, hk};
}

template <int D, bool kDq>
__device__ __forceinline__ void bwd_load(BwdShared<D>& sm, const PrefillParams& p, const BwdMaps& maps, int lane,
                                         volatile int* abort) {
  constexpr uint32_t kBytes = kBox * (D / 64), kLong = BwdShared<D>::kLong, kBrief = BwdShared<D>::kBrief;
  ItemWalk<!kDq> walk(kTile, kDq ? p.H : p.HK * p.splits);
  const CUtensorMap *own0 = kDq ? &maps.q : &maps.k, *own1 = kDq ? &maps.dout : &maps.v;
  const CUtensorMap *lng = kDq ? &maps.k : &maps.q, *brf = kDq ? &maps.v : &maps.dout;
  uint32_t items = 0, own_loads = 0, longs = 0, briefs = 0;
  bool ok = true;
  auto load = [&](const CUtensorMap* map, TileMem<D>& dst, uint64_t* bar, int head, int row) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) lap::tma_load_3d(dst[b], map, bar, 64 * b, head, row);
  };
  for (; ok; ++items) {
    const uint32_t is = items % kBwdItems;
    if (!warp_wait(&sm.item_empty[is], ((items / kBwdItems) & 1u) ^ 1u, abort)) break;
    const Item it = walk.take(p, lane);
    if (lane == 0) {
      sm.items[is] = it;
      lap::mbar_arrive(&sm.item_full[is]);
    }
    __syncwarp();
    if (it.len < 0) break;
    const Passes w = passes_of<kDq>(p, it);
    int head = w.head, tile = w.first;
    for (int n = 0; n < w.count; ++n) {
      const uint32_t l = longs % kLong, b = briefs % kBrief;
      if (!(ok = warp_wait(&sm.long_empty[l], ((longs / kLong) & 1u) ^ 1u, abort))) break;
      if (lane == 0) {
        lap::mbar_arrive_expect_tx(&sm.long_full[l], kBytes);
        load(lng, sm.long_[l], &sm.long_full[l], head, it.lo + tile * kTile);
      }
      ++longs;
      if (!(ok = warp_wait(&sm.brief_empty[b], ((briefs / kBrief) & 1u) ^ 1u, abort))) break;
      if (lane == 0) {
        lap::mbar_arrive_expect_tx(&sm.brief_full[b], kBytes);
        load(brf, sm.brief[b], &sm.brief_full[b], head, it.lo + tile * kTile);
      }
      ++briefs;
      if (n == 0) {  // the first tiles that pass are on their way while the last item still reads its own
        if (!(ok = warp_wait(&sm.own_empty, (own_loads & 1u) ^ 1u, abort))) break;
        if (lane == 0) {
          lap::mbar_arrive_expect_tx(&sm.own_full, 2 * kBytes);
          load(own0, sm.own[0], &sm.own_full, w.own, it.lo + it.tile * kTile);
          load(own1, sm.own[1], &sm.own_full, w.own, it.lo + it.tile * kTile);
        }
        ++own_loads;
      }
      if (++tile == w.first + w.each) tile = w.first, ++head;
    }
  }
  // every load has landed before the block's shared memory is given up, also after an abort
  if (lane == 0) {
    if (own_loads) drain(&sm.own_full, (own_loads - 1) & 1u);
    for (uint32_t i = 1; i <= kLong && i <= longs; ++i) drain(&sm.long_full[(longs - i) % kLong], ((longs - i) / kLong) & 1u);
    for (uint32_t i = 1; i <= kBrief && i <= briefs; ++i)
      drain(&sm.brief_full[(briefs - i) % kBrief], ((briefs - i) / kBrief) & 1u);
  }
  __syncwarp();
}

// A value as three BF16 parts, the first three of eight elements.
__device__ __forceinline__ uint4 three_parts(float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x)), rest = x - hi;
  const float mid = __bfloat162float(__float2bfloat16_rn(rest));
  return make_uint4(lap::pack_bf16x2(hi, mid), lap::pack_bf16x2(rest - mid, 0.f), 0, 0);
}

// c, and where it is so small that lse / c may be infinite, a c that changes no score.
__device__ __forceinline__ float fold_scale(float c) { return fabsf(c) < 1e-30f ? copysignf(1e-30f, c) : c; }

// dk, dv: -lse log2 e and delta of the rows that pass.
template <int D>
__device__ __forceinline__ void bwd_stats(BwdShared<D>& sm, const PrefillParams& p, int lane, volatile int* abort) {
  uint32_t tiles = 0;
  const float per_c = 1.f / fold_scale(p.scale * kLog2e);
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kBwdItems;
    if (!warp_wait(&sm.item_full[is], (i / kBwdItems) & 1u, abort)) return;
    const Item it = sm.items[is];
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) return;
    const Passes w = passes_of<false>(p, it);
    int head = w.head, tile = w.first;
    for (int n = 0; n < w.count; ++n, ++tiles) {
      float lse[4], delta[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = tile * kTile + 32 * e + lane;
        const int64_t at = static_cast<int64_t>(head) * p.tokens + it.lo + row;
        lse[e] = row < it.len ? -__ldg(p.lse_in + at) * kLog2e : 0.f;
        delta[e] = row < it.len ? p.delta[at] : 0.f;
      }
      const uint32_t st = tiles & 1;
      if (!warp_wait(&sm.stat_empty[st], ((tiles >> 1) & 1u) ^ 1u, abort)) return;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 32 * e + lane;
        if constexpr (kFold<D>) {
          uint4* at = reinterpret_cast<uint4*>(sm.st.stats[st] + row * 128);  // 16-byte chunk x lies at x ^ (row % 8)
          at[row & 7] = three_parts(lse[e] * per_c);
          at[2 ^ (row & 7)] = three_parts(-delta[e]);
        } else {
          sm.st.lse[st][row] = lse[e];
          sm.st.delta[st][row] = delta[e];
        }
      }
      if (kFold<D>) lap::fence_proxy_async_smem();
      warp_arrive(&sm.stat_full[st], lane);
      if (++tile == w.first + w.each) tile = w.first, ++head;
    }
  }
}

// Tensor memory: S at 0, dP behind it, then dv and dk, or two buffers of dS and dq.  For dk and dv at D = 64 there is
// room for a second S, whose product then need not wait for the last p (258 us to 240).
template <int D, bool kDq>
constexpr bool kTwo = !kDq && D == 64;
template <int D, bool kDq>
constexpr int kColDp = kTwo<D, kDq> ? 2 * kTile : kTile;
template <int D>
constexpr int kColDv = kColDp<D, false> + kTile;
constexpr int kColDs = 2 * kTile, kColDq = 3 * kTile;

// (Slots and parities are running values, as in the forward kernel.)
template <int D, bool kDq>
__device__ __forceinline__ void bwd_products(BwdShared<D>& sm, const PrefillParams& p, uint32_t tmem, int lane,
                                             volatile int* abort) {
  constexpr uint32_t kSlot = sizeof(TileMem<D>) >> 4, kLong = BwdShared<D>::kLong, kBrief = BwdShared<D>::kBrief;
  constexpr bool kFolded = !kDq && kFold<D>, kTwoS = kTwo<D, kDq>;
  const uint32_t t_dp = tmem + kColDp<D, kDq>, t_dv = tmem + kColDv<D>, t_dk = t_dv + D;
  const uint32_t own0 = desc_rows(sm.own[0]), long_rows = desc_rows(sm.long_[0]), long_columns = desc_columns(sm.long_[0]);
  const uint32_t brief_rows = desc_rows(sm.brief[0]), brief_columns = desc_columns(sm.brief[0]);
  constexpr uint32_t kId = lap::idesc_bf16_f32(kTile, kTile, false, false), kStat = kBox >> 4;
  uint32_t ones = 0, stats = 0;
  if constexpr (kFolded) ones = desc_rows(sm.st.ones), stats = desc_rows(sm.st.stats[0]);
  uint32_t next = 0, next_phase = 0, slot = 0;     // long slots: of the next scores, of the tile whose sums are next
  uint32_t bnext = 0, bnext_phase = 0, bslot = 0;  // brief slots: of the next dP, of the next p^T dO
  uint32_t tiles = 0;                              // tiles whose sums have begun
  bool ok = true;
  // scores and dP of tile x, in order
  auto scores = [&](uint32_t x) {
    if (!warp_wait(&sm.long_full[next], next_phase, abort) ||
        (kFolded && !warp_wait(&sm.stat_full[x & 1], x >> 1 & 1u, abort)) ||
        (kDq && !warp_wait(&sm.s_free, (x & 1u) ^ 1u, abort)))
      return false;
    const uint32_t t_s = tmem + (kTwoS ? (x & 1) * kTile : 0);
    lap::tc_fence_after();
    product_rows<D>(t_s, own0, long_rows + next * kSlot);
    if (kFolded) mma1_rows<kId>(t_s, ones, stats + (x & 1) * kStat);
    commit(&sm.s_full[kTwoS ? x & 1 : 0]);
    if (++next == kLong) next = 0, next_phase ^= 1;
    return true;
  };
  auto dps = [&](uint32_t x, bool last) {
    if (!warp_wait(&sm.brief_full[bnext], bnext_phase, abort) || (kDq && !warp_wait(&sm.dp_free, (x & 1u) ^ 1u, abort)))
      return false;
    lap::tc_fence_after();
    product_rows<D>(t_dp, own0 + kSlot, brief_rows + bnext * kSlot);
    if (kFolded) {
      mma1_rows<kId>(t_dp, ones + 2, stats + (x & 1) * kStat + 2);
      commit(&sm.stat_empty[x & 1]);
    }
    commit(&sm.dp_full);
    if (kDq) commit(&sm.brief_empty[bnext]);
    if (last) commit(&sm.own_empty);
    if (++bnext == kBrief) bnext = 0, bnext_phase ^= 1;
    return true;
  };
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t is = i % kBwdItems;
    if (!warp_wait(&sm.item_full[is], (i / kBwdItems) & 1u, abort)) break;
    const Item it = uniform(sm.items[is]);
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) break;
    const int count = passes_of<kDq>(p, it).count;
    if (!(ok = warp_wait(&sm.own_full, i & 1u, abort))) break;
    // the first tile's scores and dP; their columns were read before the last item's last product
    if (!(ok = scores(tiles)) || !(ok = dps(tiles, count == 1))) break;
    if (kTwoS && count > 1 && !(ok = scores(tiles + 1))) break;
    for (int n = 0; n < count; ++n, ++tiles) {
      const bool more = n + 1 < count;
      const uint32_t parity = tiles & 1;
      if (kDq) {
        if (more && (!(ok = scores(tiles + 1)) || !(ok = dps(tiles + 1, n + 2 == count)))) break;
        if (!(ok = warp_wait(&sm.ds_ready, parity, abort))) break;
        if (n == 0 && !(ok = warp_wait(&sm.acc_free, (i & 1u) ^ 1u, abort))) break;
        lap::tc_fence_after();
        product_tmem<D>(tmem + kColDq, tmem + kColDs + 64 * parity, long_columns + slot * kSlot, n > 0);
        commit(&sm.long_empty[slot]);
        if (!more) commit(&sm.acc_full);
      } else {
        constexpr int kAhead = kTwoS ? 2 : 1;  // tiles that the scores are ahead
        if (!(ok = warp_wait(&sm.p_ready[kTwoS ? parity : 0], kTwoS ? tiles >> 1 & 1u : parity, abort))) break;
        if (n == 0 && !(ok = warp_wait(&sm.acc_free, (i & 1u) ^ 1u, abort))) break;
        lap::tc_fence_after();
        product_tmem<D, kColumns>(t_dv, tmem + (kTwoS ? parity * kTile : 0), brief_columns + bslot * kSlot, n > 0);
        commit(&sm.brief_empty[bslot]);
        if (++bslot == kBrief) bslot = 0;
        if (n + kAhead < count && !(ok = scores(tiles + kAhead))) break;
        if (!(ok = warp_wait(&sm.ds_ready, parity, abort))) break;
        lap::tc_fence_after();
        product_tmem<D, kColumns>(t_dk, t_dp, long_columns + slot * kSlot, n > 0);
        commit(&sm.long_empty[slot]);
        if (!more) commit(&sm.acc_full);
        if (more && !(ok = dps(tiles + 1, n + 2 == count))) break;
      }
      if (++slot == kLong) slot = 0;
    }
  }
  commit(&sm.final_bar);
  drain(&sm.final_bar, 0);  // every product has retired, also after an abort
  __syncwarp();
}

// Rows of a tile that lie behind the sequence become zero: box `box` of row `row`.
template <int D>
__device__ __forceinline__ void clear_row(TileMem<D>& tile, int box, int row) {
  if (box >= D / 64) return;
  uint4* at = reinterpret_cast<uint4*>(tile[box] + row * 128);
#pragma unroll
  for (int c = 0; c < 8; ++c) at[c] = make_uint4(0, 0, 0, 0);
}

// An output row's D columns from tensor memory, times a factor.
template <int D>
__device__ __forceinline__ void write_row(uint32_t t, bf16* out, float f, bool live, int from, int to) {
#pragma unroll 1
  for (int g = from; g < to; ++g) {
    float o[32];
    lap::tmem_ld32(t + 32 * g, o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] *= f;
    if (live) store_row32(out + 32 * g, o);
  }
}

// The same in FP32.
template <int D>
__device__ __forceinline__ void write_part(uint32_t t, float* out, float f, bool live, int from, int to) {
#pragma unroll 1
  for (int g = from; g < to; ++g) {
    float o[32];
    lap::tmem_ld32(t + 32 * g, o);
    if (live)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        reinterpret_cast<float4*>(out + 32 * g)[e] =
            make_float4(o[4 * e] * f, o[4 * e + 1] * f, o[4 * e + 2] * f, o[4 * e + 3] * f);
  }
}

// dk, dv.  A thread has one key and kColumns of a tile's rows.
template <int D>
__device__ __forceinline__ void bwd_dkdv(BwdShared<D>& sm, const PrefillParams& p, uint32_t tmem, int tid,
                                         volatile int* abort) {
  const int part = tid / kTile, key = tid % kTile, lane = tid % 32;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(key & ~31) << 16);
  constexpr bool kTwoS = kTwo<D, false>;
  const uint32_t t_s0 = t_lane + kColumns * part, t_dp = t_s0 + kColDp<D, false>;
  const float c = kFold<D> ? fold_scale(p.scale * kLog2e) : p.scale * kLog2e;
  const uint64_t c2 = lap::f2_pack(c, c);
  uint32_t tiles = 0, slot = 0, bslot = 0;  // slots of the rings
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kBwdItems;
    if (!warp_wait(&sm.item_full[is], (i / kBwdItems) & 1u, abort)) return;
    const Item it = sm.items[is];
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) return;
    const Passes w = passes_of<false>(p, it);
    int tile = w.first;
    for (int n = 0; n < w.count; ++n, ++tiles) {
      const uint32_t st = tiles & 1, t_s = t_s0 + (kTwoS ? st * kTile : 0);
      const int valid = it.len - tile * kTile;
      if (!kFold<D> && !warp_wait(&sm.stat_full[st], (tiles >> 1) & 1u, abort)) return;  // there long before the scores
      if (!warp_wait(&sm.s_full[kTwoS ? st : 0], kTwoS ? tiles >> 1 & 1u : st, abort)) return;
      if (valid < kTile) {
        // rows behind the sequence must not enter the sums over rows (0 * inf is NaN)
        if (!warp_wait(&sm.dp_full, tiles & 1u, abort)) return;
        if (key >= valid) clear_row<D>(part < 2 ? sm.long_[slot] : sm.brief[bslot], part & 1, key);
        lap::fence_proxy_async_smem();
      }
      // this thread's rows [from, to) see the key
      const bool masked = tile == it.tile || valid < kTile;
      const int from = tile == it.tile ? key - kColumns * part : 0, to = valid - kColumns * part;
      lap::tc_fence_after();
      float s[kColumns];
      lap::tmem_ld32(t_s, s);
      const float4 *lse = nullptr, *delta = nullptr;
      if constexpr (!kFold<D>) {
        lse = reinterpret_cast<const float4*>(sm.st.lse[st] + kColumns * part);
        delta = reinterpret_cast<const float4*>(sm.st.delta[st] + kColumns * part);
      }
      auto weights = [&](auto has_mask) {
        constexpr bool kMasked = decltype(has_mask)::value;
        uint32_t u[kColumns / 2];
#pragma unroll
        for (int k = 0; k < kColumns; k += 4) {
          uint64_t z01 = lap::f2_pack(s[k], s[k + 1]), z23 = lap::f2_pack(s[k + 2], s[k + 3]);
          if constexpr (kFold<D>) {
            z01 = lap::f2_mul(z01, c2), z23 = lap::f2_mul(z23, c2);
          } else {
            const float4 l = lse[k / 4];  // minus lse log2 e
            z01 = lap::f2_fma(z01, c2, lap::f2_pack(l.x, l.y)), z23 = lap::f2_fma(z23, c2, lap::f2_pack(l.z, l.w));
          }
          const float2 z0 = lap::f2_unpack(z01), z1 = lap::f2_unpack(z23);
          s[k] = lap::exp2_approx(z0.x), s[k + 1] = lap::exp2_approx(z0.y);
          s[k + 2] = lap::exp2_approx(z1.x), s[k + 3] = lap::exp2_approx(z1.y);
          if (kMasked)
#pragma unroll
            for (int x = k; x < k + 4; ++x) s[x] = x >= from && x < to ? s[x] : 0.f;
          u[k / 2] = lap::pack_bf16x2(s[k], s[k + 1]);
          u[k / 2 + 1] = lap::pack_bf16x2(s[k + 2], s[k + 3]);
        }
        lap::tmem_st16_nowait(t_s, u);
      };
      if (masked) weights(std::true_type{}); else weights(std::false_type{});
      lap::tmem_wait_st();
      lap::tc_fence_before();
      warp_arrive(&sm.p_ready[kTwoS ? st : 0], lane);
      if (!warp_wait(&sm.dp_full, tiles & 1u, abort)) return;
      lap::tc_fence_after();
      float dp[kColumns];
      lap::tmem_ld32(t_dp, dp);
      auto slopes = [&](auto has_mask) {
        constexpr bool kMasked = decltype(has_mask)::value;
        uint32_t u[kColumns / 2];
#pragma unroll
        for (int k = 0; k < kColumns; k += 4) {
          uint64_t d01 = lap::f2_pack(dp[k], dp[k + 1]), d23 = lap::f2_pack(dp[k + 2], dp[k + 3]);
          if constexpr (!kFold<D>) {
            const float4 d = delta[k / 4];
            d01 = lap::f2_sub(d01, lap::f2_pack(d.x, d.y)), d23 = lap::f2_sub(d23, lap::f2_pack(d.z, d.w));
          }
          float2 a = lap::f2_unpack(lap::f2_mul(lap::f2_pack(s[k], s[k + 1]), d01));
          float2 b = lap::f2_unpack(lap::f2_mul(lap::f2_pack(s[k + 2], s[k + 3]), d23));
          if (kMasked) {
            a.x = k >= from && k < to ? a.x : 0.f;
            a.y = k + 1 >= from && k + 1 < to ? a.y : 0.f;
            b.x = k + 2 >= from && k + 2 < to ? b.x : 0.f;
            b.y = k + 3 >= from && k + 3 < to ? b.y : 0.f;
          }
          u[k / 2] = lap::pack_bf16x2(a.x, a.y);
          u[k / 2 + 1] = lap::pack_bf16x2(b.x, b.y);
        }
        lap::tmem_st16_nowait(t_dp, u);
      };
      if (masked) slopes(std::true_type{}); else slopes(std::false_type{});
      lap::tmem_wait_st();
      lap::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        lap::mbar_arrive(&sm.ds_ready);
        if (!kFold<D>) lap::mbar_arrive(&sm.stat_empty[st]);
      }
      if (++tile == w.first + w.each) tile = w.first;
      if (++slot == BwdShared<D>::kLong) slot = 0;
      if (++bslot == BwdShared<D>::kBrief) bslot = 0;
    }
    if (!warp_wait(&sm.acc_full, i & 1u, abort)) return;
    lap::tc_fence_after();
    const int64_t at = it.lo + it.tile * kTile + key;
    const bool live = it.tile * kTile + key < it.len;
    const int g = (part & 1) * (D / 64), is_dk = part >> 1;
    const uint32_t t_sum = t_lane + kColDv<D> + D * is_dk;
    const float f = is_dk ? p.scale : 1.f;
    if (p.part == nullptr) {
      write_row<D>(t_sum, (is_dk ? p.dk : p.dv).row(at, w.own), f, live, g, g + D / 64);
    } else {
      const int split = it.head - w.own * p.splits;
      if (live && split == 0 && part == 0) p.marks[static_cast<int64_t>(w.own) * p.tokens + at] = 1;
      write_part<D>(t_sum, p.part + (((static_cast<int64_t>(split) * 2 + is_dk) * p.HK + w.own) * p.tokens + at) * D, f, live,
                    g, g + D / 64);
    }
    lap::tc_fence_before();
    warp_arrive(&sm.acc_free, lane);
  }
}

// dq.  A thread has one row and kColumns of a tile's keys.
template <int D>
__device__ __forceinline__ void bwd_dq(BwdShared<D>& sm, const PrefillParams& p, uint32_t tmem, int tid,
                                       volatile int* abort) {
  const int part = tid / kTile, row = tid % kTile, lane = tid % 32;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(row & ~31) << 16);
  const uint32_t t_s = t_lane + kColumns * part, t_dp = t_lane + kColDp<D, true> + kColumns * part;
  const float c = p.scale * kLog2e;
  const uint64_t c2 = lap::f2_pack(c, c);
  uint32_t tiles = 0, slot = 0;  // slot of the long ring
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kBwdItems;
    if (!warp_wait(&sm.item_full[is], (i / kBwdItems) & 1u, abort)) return;
    const Item it = sm.items[is];
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) return;
    const int64_t at = it.lo + it.tile * kTile + row, stat = static_cast<int64_t>(it.head) * p.tokens + at;
    const bool live = it.tile * kTile + row < it.len;
    const float lse = live ? __ldg(p.lse_in + stat) * kLog2e : 0.f, delta = live ? p.delta[stat] : 0.f;
    const uint64_t l2 = lap::f2_pack(-lse, -lse), d2 = lap::f2_pack(delta, delta);
    for (int n = 0; n <= it.tile; ++n, ++tiles) {
      const bool masked = n == it.tile;
      const int keep = row + 1 - kColumns * part;  // of this thread's keys, on the diagonal
      if (!warp_wait(&sm.s_full[0], tiles & 1u, abort)) return;
      if (masked && it.len < (it.tile + 1) * kTile) {
        // keys behind the sequence must not enter the sum over keys (0 * inf is NaN)
        if (it.tile * kTile + row >= it.len && part < 2) clear_row<D>(sm.long_[slot], part, row);
        lap::fence_proxy_async_smem();
      }
      lap::tc_fence_after();
      float s[kColumns];
      lap::tmem_ld32(t_s, s);
      lap::tc_fence_before();
      warp_arrive(&sm.s_free, lane);
#pragma unroll
      for (int k = 0; k < kColumns; k += 2) {
        const float2 z = lap::f2_unpack(lap::f2_fma(lap::f2_pack(s[k], s[k + 1]), c2, l2));
        s[k] = lap::exp2_approx(z.x), s[k + 1] = lap::exp2_approx(z.y);
      }
      if (!warp_wait(&sm.dp_full, tiles & 1u, abort)) return;
      lap::tc_fence_after();
      float dp[kColumns];
      lap::tmem_ld32(t_dp, dp);
      lap::tc_fence_before();
      warp_arrive(&sm.dp_free, lane);
      auto slopes = [&](auto has_mask) {
        constexpr bool kMasked = decltype(has_mask)::value;
        uint32_t u[kColumns / 2];
#pragma unroll
        for (int k = 0; k < kColumns; k += 2) {
          float2 a = lap::f2_unpack(lap::f2_mul(lap::f2_pack(s[k], s[k + 1]), lap::f2_sub(lap::f2_pack(dp[k], dp[k + 1]), d2)));
          if (kMasked) {
            a.x = k < keep ? a.x : 0.f;
            a.y = k + 1 < keep ? a.y : 0.f;
          }
          u[k / 2] = lap::pack_bf16x2(a.x, a.y);
        }
        lap::tmem_st16_nowait(t_lane + kColDs + 64 * (tiles & 1) + kColumns / 2 * part, u);
      };
      if (masked) slopes(std::true_type{}); else slopes(std::false_type{});
      lap::tmem_wait_st();
      lap::tc_fence_before();
      warp_arrive(&sm.ds_ready, lane);
      if (++slot == BwdShared<D>::kLong) slot = 0;
    }
    if (!warp_wait(&sm.acc_full, i & 1u, abort)) return;
    lap::tc_fence_after();
    if (part < 2) write_row<D>(t_lane + kColDq, p.dq.row(at, it.head), p.scale, live, part * (D / 64), (part + 1) * (D / 64));
    lap::tc_fence_before();
    warp_arrive(&sm.acc_free, lane);
  }
}

template <int D, bool kDq>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_bwd_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem_tiles[];  // without room to align it: it begins aligned
  BwdShared<D>& sm = *reinterpret_cast<BwdShared<D>*>(smem_tiles);
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
  volatile int* abort = &sm.abort;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  if (lap::smem_u32(smem_tiles) & 1023u) {  // swizzled tiles would land elsewhere: leave at once
    if (tid == 0 && p.dev_error) atomicOr(p.dev_error, kErrTimeout);
    return;
  }
  if (warp == 16) {
    lap::tmem_alloc(&sm.tmem, 512);
    lap::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kBwdItems; ++i) {
      lap::mbar_init(&sm.item_full[i], 1);
      lap::mbar_init(&sm.item_empty[i], kDq ? 17 : 18);
    }
    lap::mbar_init(&sm.own_full, 1);
    lap::mbar_init(&sm.own_empty, 1);
    for (uint32_t i = 0; i < BwdShared<D>::kLong; ++i) {
      lap::mbar_init(&sm.long_full[i], 1);
      lap::mbar_init(&sm.long_empty[i], 1);
    }
    for (uint32_t i = 0; i < BwdShared<D>::kBrief; ++i) {
      lap::mbar_init(&sm.brief_full[i], 1);
      lap::mbar_init(&sm.brief_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      lap::mbar_init(&sm.stat_full[i], 1);
      lap::mbar_init(&sm.stat_empty[i], kFold<D> ? 1 : 16);
      lap::mbar_init(&sm.s_full[i], 1);
      lap::mbar_init(&sm.p_ready[i], 16);
    }
    lap::mbar_init(&sm.s_free, 16);
    lap::mbar_init(&sm.dp_full, 1);
    lap::mbar_init(&sm.dp_free, 16);
    lap::mbar_init(&sm.ds_ready, 16);
    lap::mbar_init(&sm.acc_full, 1);
    lap::mbar_init(&sm.acc_free, 16);
    lap::mbar_init(&sm.final_bar, 1);
    sm.abort = 0;
    lap::fence_mbar_init();
    lap::tma_prefetch_desc(&maps.q);
    lap::tma_prefetch_desc(&maps.k);
    lap::tma_prefetch_desc(&maps.v);
    lap::tma_prefetch_desc(&maps.dout);
  }
  if constexpr (!kDq && kFold<D>) {
    for (int x = tid; x < kTile * 8; x += kBwdThreads) {
      const int row = x / 8, chunk = x % 8;
      const uint32_t one = 0x3F80u;
      reinterpret_cast<uint4*>(sm.st.ones + row * 128)[chunk ^ (row & 7)] =
          chunk == 0 || chunk == 2 ? make_uint4(one | one << 16, one, 0, 0) : make_uint4(0, 0, 0, 0);
      for (int s = 0; s < 2; ++s) reinterpret_cast<uint4*>(sm.st.stats[s] + row * 128)[chunk ^ (row & 7)] = make_uint4(0, 0, 0, 0);
    }
    lap::fence_proxy_async_smem();
  }
  lap::tc_fence_before();
  __syncthreads();
  lap::tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  if (warp < 16) {
    if constexpr (kDq)
      bwd_dq<D>(sm, p, tmem, tid, abort);
    else
      bwd_dkdv<D>(sm, p, tmem, tid, abort);
  } else if (warp == 16) {
    bwd_products<D, kDq>(sm, p, tmem, lane, abort);
  } else if (warp == 17) {
    bwd_load<D, kDq>(sm, p, maps, lane, abort);
  } else if (warp == 18 && !kDq) {
    bwd_stats<D>(sm, p, lane, abort);
  }
  lap::tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort && p.dev_error) atomicOr(p.dev_error, kErrTimeout);
  if (warp == 16) {
    __syncwarp();
    lap::tc_fence_after();
    lap::tmem_dealloc(tmem, 512);
  }
}

// delta[h][t] = sum over D of dO o, D / 8 threads a row; bound by reading both once.
template <int D>
__global__ void __launch_bounds__(kDeltaThreads) attn_delta_kernel(const __grid_constant__ PrefillParams p) {
  constexpr int kLanes = D / 8;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * kDeltaThreads + threadIdx.x) / kLanes;
  const int64_t t = r / p.H;
  const int h = static_cast<int>(r - t * p.H), c = threadIdx.x % kLanes * 8;
  float sum = 0.f;
  if (t < p.tokens) {
    const uint4 a = *reinterpret_cast<const uint4*>(p.dout.row(t, h) + c), b = *reinterpret_cast<const uint4*>(p.o_in.row(t, h) + c);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = fmaf(lap::bf16lo_to_f32(x[i]), lap::bf16lo_to_f32(y[i]), sum);
      sum = fmaf(lap::bf16hi_to_f32(x[i]), lap::bf16hi_to_f32(y[i]), sum);
    }
  }
#pragma unroll
  for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (t < p.tokens && c == 0) {
    p.delta[h * static_cast<int64_t>(p.tokens) + t] = sum;
    if (p.part && h < p.HK) p.marks[h * static_cast<int64_t>(p.tokens) + t] = 0;
  }
}

// dk and dv from the sums over the parts of their group's heads, in order; 8 columns a thread, rows that
// belong to a sequence.
template <int D>
__global__ void __launch_bounds__(kDeltaThreads) attn_sum_kernel(const __grid_constant__ PrefillParams p) {
  constexpr int kLanes = D / 8;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int64_t r = (static_cast<int64_t>(blockIdx.x) * kDeltaThreads + threadIdx.x) / kLanes;
  const int64_t t = r / p.HK;
  const int hk = static_cast<int>(r - t * p.HK), c = threadIdx.x % kLanes * 8;
  if (t >= p.tokens || !p.marks[static_cast<int64_t>(hk) * p.tokens + t]) return;
#pragma unroll
  for (int is_dk = 0; is_dk < 2; ++is_dk) {
    float s[8] = {};
#pragma unroll 4
    for (int x = 0; x < p.splits; ++x) {
      const float4* at = reinterpret_cast<const float4*>(
          p.part + (((static_cast<int64_t>(x) * 2 + is_dk) * p.HK + hk) * p.tokens + t) * D + c);
      const float4 a = at[0], b = at[1];
      s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
      s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
    }
    *reinterpret_cast<uint4*>((is_dk ? p.dk : p.dv).row(t, hk) + c) =
        make_uint4(lap::pack_bf16x2(s[0], s[1]), lap::pack_bf16x2(s[2], s[3]), lap::pack_bf16x2(s[4], s[5]),
                   lap::pack_bf16x2(s[6], s[7]));
  }
}

}  // namespace laa
