// la_attention_fwd.cuh -- causal attention over whole prompts (include/la_attention.h) on the tensor
// cores.
//
// A block takes 256 query rows of one head, as two tiles of 128, and walks over the sequence's keys,
// 128 at a time, with an unnormalised output and a running maximum and sum per row.
// Warps 0-7 and 8-15 own one query tile each, two threads per row, each with 64 of a tile's keys: S is
// read from tensor memory and p goes back over it as the operand of the second product; O is rarely
// rescaled and always by its owners, which need no extra warps for it.  The two threads of a row meet
// to agree on its maximum: they tell each other what they found and compute on with the old one
// meanwhile.  (A thread per row, with half the warps, left each scheduler two warps to hide their
// latencies: 3250 cycles for a round of both tiles, 1.53 ms for 2 x 8192 tokens of 64 heads of 128.)
// Warp 16
// issues the products: while one tile's softmax runs, the other tile's two products keep the tensor
// cores busy (S_a, S_b, then p v and the next S of each in turn, in one queue, so that S can
// overwrite p).  Warp 17 loads: queries once per item, keys and values through a ring.
// The two tiles share keys and values, which halves their traffic from L2.
//
// Bound: the tensor cores at D = 128; at D = 64, where the products halve, the softmax.
#pragma once

#include "la_attention_softmax.cuh"

namespace laa {

constexpr int kFwdRows = 2 * kTile, kFwdThreads = 640, kItems = 4;
// Registers: 5 x 96 at launch.
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;
static_assert(4 * kSoftmaxRegs + kOtherRegs <= 5 * 96, "register shares");

template <int D>
struct alignas(1024) FwdShared {
  static constexpr int kStages = D == 128 ? 5 : 8;
  TileMem<D> q[2];
  TileMem<D> kv[kStages];
  Item items[kItems];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2][2], o_full[2], o_free[2];
  uint64_t final_bar;
  uint64_t pair[2][4];       // [tile][warp]: the two halves of its rows meet
  float said[2][2][kTile];   // [tile][half][row]
  uint32_t bad[2][2][2][4];  // [item parity][tile][box][32 rows]: value rows that are not finite
  uint32_t tmem;
  int abort;
};

struct FwdMaps {
  CUtensorMap q, k, v;
};

// Tiles of keys that query tile s of an item sees; 0 where it has no row.
__device__ __forceinline__ int key_tiles(const Item& it, int s) {
  const int r0 = it.tile * kFwdRows + s * kTile;
  return r0 < it.len ? r0 / kTile + 1 : 0;
}

template <int D>
__device__ __forceinline__ void fwd_load(FwdShared<D>& sm, const PrefillParams& p, const FwdMaps& maps, int lane,
                                         volatile int* abort) {
  constexpr int kStages = FwdShared<D>::kStages;
  constexpr uint32_t kBytes = kBox * (D / 64);
  const int group = p.H / p.HK;
  ItemWalk<false> walk(kFwdRows, p.H);
  uint32_t slots = 0, q_loads[2] = {0, 0};
  bool ok = true;
  auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int head, int row) {
    lap::mbar_arrive_expect_tx(bar, kBytes);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) lap::tma_load_3d(dst + b * kBox, map, bar, 64 * b, head, row);
  };
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t is = i % kItems;
    if (!warp_wait(&sm.item_empty[is], ((i / kItems) & 1u) ^ 1u, abort)) break;
    const Item it = walk.take(p, lane);
    if (lane == 0) {
      sm.items[is] = it;
      lap::mbar_arrive(&sm.item_full[is]);
    }
    __syncwarp();
    if (it.len < 0) break;
    const int n = max(key_tiles(it, 0), key_tiles(it, 1)), hk = it.head / group;
    for (int j = 0; j < 2 * n && ok; ++j) {
      const uint32_t st = slots % kStages;
      if (!(ok = warp_wait(&sm.kv_empty[st], ((slots / kStages) & 1u) ^ 1u, abort))) break;
      if (lane == 0)
        load(j & 1 ? &maps.v : &maps.k, sm.kv[st][0], &sm.kv_full[st], hk, it.lo + (j >> 1) * kTile);
      ++slots;
      if (j == 0)  // the first keys are on their way while the last item still reads its queries
        for (int s = 0; s < 2 && ok; ++s) {
          if (key_tiles(it, s) == 0) continue;
          if (!(ok = warp_wait(&sm.q_empty[s], (q_loads[s] & 1u) ^ 1u, abort))) break;
          if (lane == 0) load(&maps.q, sm.q[s][0], &sm.q_full[s], it.head, it.lo + it.tile * kFwdRows + s * kTile);
          ++q_loads[s];
        }
    }
  }
  // every load has landed before the block's shared memory is given up, also after an abort
  if (lane == 0) {
    for (uint32_t i = 0; i < static_cast<uint32_t>(kStages) && i < slots; ++i) {
      const uint32_t j = slots - 1 - i;
      drain(&sm.kv_full[j % kStages], (j / kStages) & 1u);
    }
    for (int s = 0; s < 2; ++s)
      if (q_loads[s]) drain(&sm.q_full[s], (q_loads[s] - 1) & 1u);
  }
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void fwd_products(FwdShared<D>& sm, uint32_t tmem, int lane, volatile int* abort) {
  constexpr int kStages = FwdShared<D>::kStages;
  uint32_t slots = 0, q_uses[2] = {0, 0}, p_uses[2] = {0, 0};
  bool ok = true;
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t is = i % kItems;
    if (!warp_wait(&sm.item_full[is], (i / kItems) & 1u, abort)) break;
    const Item it = uniform(sm.items[is]);
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) break;
    const int n[2] = {key_tiles(it, 0), key_tiles(it, 1)};
    const int most = max(n[0], n[1]);
    auto slot_of = [&](int j, bool value) { return slots + 2 * j + value; };
    auto wait_slot = [&](uint32_t x) { return warp_wait(&sm.kv_full[x % kStages], (x / kStages) & 1u, abort); };
    auto scores = [&](int s, uint32_t x) {
      lap::tc_fence_after();
      product_rows<D>(tmem + s * kTile, desc_rows(sm.q[s]), desc_rows(sm.kv[x % kStages]));
      commit(&sm.s_full[s]);
    };
    if (!(ok = wait_slot(slot_of(0, false)))) break;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (!ok || !n[s]) continue;
      if (!(ok = warp_wait(&sm.q_full[s], q_uses[s] & 1u, abort))) continue;
      scores(s, slot_of(0, false));
      if (n[s] == 1) commit(&sm.q_empty[s]);
    }
    if (!ok) break;
    commit(&sm.kv_empty[slot_of(0, false) % kStages]);
    for (int j = 0; j < most && ok; ++j) {
      const uint32_t xv = slot_of(j, true), xk = slot_of(j + 1, false);
      bool keys = false;
      if (!(ok = wait_slot(xv))) break;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!ok || j >= n[s]) continue;
        // the product with the first 64 values runs while the other probabilities are made
        if (!(ok = warp_wait(&sm.p_ready[s][0], p_uses[s] & 1u, abort))) continue;
        if (j == 0 && !(ok = warp_wait(&sm.o_free[s], (q_uses[s] & 1u) ^ 1u, abort))) continue;
        lap::tc_fence_after();
        const uint32_t t_o = tmem + 2 * kTile + s * D, t_p = tmem + s * kTile, v = desc_columns(sm.kv[xv % kStages]);
        half_product_tmem<D, 64>(t_o, t_p, v, 0, j > 0);
        if (!(ok = warp_wait(&sm.p_ready[s][1], p_uses[s]++ & 1u, abort))) continue;
        lap::tc_fence_after();
        half_product_tmem<D, 64>(t_o, t_p, v, 1, true);
        if (j == n[s] - 1) {
          commit(&sm.o_full[s]);
          ++q_uses[s];
        } else {
          if (!keys && !(ok = wait_slot(xk))) continue;
          keys = true;
          scores(s, xk);
          if (j + 1 == n[s] - 1) commit(&sm.q_empty[s]);
        }
      }
      if (!ok) break;
      commit(&sm.kv_empty[xv % kStages]);
      if (keys) commit(&sm.kv_empty[xk % kStages]);
    }
    slots += 2 * most;
  }
  commit(&sm.final_bar);
  drain(&sm.final_bar, 0);  // every product has retired, also after an abort
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void fwd_softmax(FwdShared<D>& sm, const PrefillParams& p, uint32_t tmem, int tid,
                                            volatile int* abort) {
  constexpr int kStages = FwdShared<D>::kStages;
  const int s = tid / (2 * kTile), half = tid / kTile & 1, row = tid % kTile, warp = row / 32, lane = tid % 32;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
  const uint32_t t_s = t_lane + s * kTile + 64 * half;  // probabilities go over their own scores
  const uint32_t t_o = t_lane + 2 * kTile + s * D + half * (D / 2);
  const float c = p.scale * kLog2e;
  uint64_t* pair = &sm.pair[s][warp];
  uint32_t slots = 0, tiles = 0, uses = 0, meets = 0;
  // Tells the row's other half; both halves call it, and then hear what the other said.
  auto say = [&](float mine) {
    sm.said[s][half][row] = mine;
    warp_arrive(pair, lane);
  };
  auto meet = [&] { return warp_wait(pair, meets++ & 1u, abort); };
  const volatile float* theirs = &sm.said[s][half ^ 1][row];
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kItems;
    if (!warp_wait(&sm.item_full[is], (i / kItems) & 1u, abort)) return;
    const Item it = sm.items[is];
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) return;
    const int n = key_tiles(it, s), first_slot = slots;
    slots += 2 * max(n, key_tiles(it, s ^ 1));
    if (n == 0) continue;
    const int r0 = it.tile * kFwdRows + s * kTile;
    const int keep = row + 1 - 64 * half;  // keys of this half that the row sees in the tile on the diagonal
    float m = 0.f;
    uint64_t l = 0;
    auto tile = [&](auto on_diagonal, bool first) {
      constexpr bool kMasked = decltype(on_diagonal)::value;
      float x[64];
      uint32_t u[32];
      float z = half_scores<kMasked>(t_s, x, c, keep);
      if (first && uses > 0 && !meet()) return false;  // the other half has heard the last item's sum
      say(z);
      if (first) {
        if (!meet()) return false;
        m = fmaxf(z, *theirs);
      }
      uint64_t sum = half_probabilities<kMasked>(x, u, c, m, keep);
      if (!first) {
        // made with the maximum as it was, and again where the row outgrew it
        if (!meet()) return false;
        z = fmaxf(z, *theirs);
        if (__any_sync(0xFFFFFFFFu, z > m + kSlack)) {
          // S follows the last product into O in the queue, so O may be rescaled
          rescale_row<D / 2>(t_o, outgrow(z, m, l));
          half_scores<kMasked>(t_s, x, c, keep);
          sum = half_probabilities<kMasked>(x, u, c, m, keep);
        }
      }
      lap::tmem_st32_nowait(t_s, u);
      lap::tmem_wait_st();
      lap::tc_fence_before();
      warp_arrive(&sm.p_ready[s][half], lane);
      l = lap::f2_add(l, sum);
      return true;
    };
    for (int j = 0; j < n - 1; ++j) {
      if (!warp_wait(&sm.s_full[s], tiles++ & 1u, abort)) return;
      lap::tc_fence_after();
      if (!tile(std::false_type{}, j == 0)) return;
    }
    {
      // the tile on the diagonal: row r sees its keys 0 .. r; its values are made harmless first, each
      // half those that its own probabilities meet.  (The scores, made from the slot before, prove that
      // the ring has come to this phase of the values'.)
      const uint32_t x = first_slot + 2 * (n - 1) + 1;
      if (!warp_wait(&sm.s_full[s], tiles++ & 1u, abort)) return;
      if (!warp_wait(&sm.kv_full[x % kStages], (x / kStages) & 1u, abort)) return;
      const int v = 64 * half + row % 64, box = row / 64;
      const uint32_t bad =
          __ballot_sync(0xFFFFFFFFu, box < D / 64 && clean_box(sm.kv[x % kStages][box < D / 64 ? box : 0], v, r0 + v >= it.len));
      if (lane == 0) sm.bad[i & 1][s][box][v / 32] = bad;
      lap::fence_proxy_async_smem();
      lap::tc_fence_after();
      if (!tile(std::true_type{}, n == 1)) return;
    }
    const int64_t at = it.lo + r0 + row;
    const bool live = r0 + row < it.len;
    // (the last product proves that the other half has heard the last maximum)
    if (!warp_wait(&sm.o_full[s], uses++ & 1u, abort)) return;
    lap::tc_fence_after();
    const float2 lp = lap::f2_unpack(l);
    float total = lp.x + lp.y;
    say(total);
    if (!meet()) return;
    total = half ? *theirs + total : total + *theirs;
    warp_arrive(pair, lane);  // heard: see the next item's first tile
    const float inv = 1.f / total;
    uint32_t bad[4], any_bad = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      bad[w] = sm.bad[i & 1][s][0][w] | sm.bad[i & 1][s][1][w];
      any_bad |= bad[w];
    }
    bf16* out = p.o.row(at, it.head) + half * (D / 2);
#pragma unroll 1
    for (int g = 0; g < D / 64; ++g) {
      float o[32];
      lap::tmem_ld32(t_o + 32 * g, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] *= inv;
      if (any_bad)
        for (int r = 0; r <= row; ++r) {
          const uint32_t w = r < 64 ? (r < 32 ? bad[0] : bad[1]) : (r < 96 ? bad[2] : bad[3]);
          if (w >> (r & 31) & 1u)
            restore(o, p.v.row(it.lo + r0 + r, it.head / (p.H / p.HK)) + half * (D / 2) + 32 * g);
        }
      if (live) store_row32(out + 32 * g, o);
    }
    lap::tc_fence_before();
    warp_arrive(&sm.o_free[s], lane);
    if (p.lse && live && half == 0) p.lse[static_cast<int64_t>(it.head) * p.tokens + at] = (m + log2f(total)) * kLn2;
  }
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd_kernel(const __grid_constant__ FwdMaps maps, const __grid_constant__ PrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem_tiles[];  // without room to align it: it begins aligned
  FwdShared<D>& sm = *reinterpret_cast<FwdShared<D>*>(smem_tiles);
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
    for (int i = 0; i < kItems; ++i) {
      lap::mbar_init(&sm.item_full[i], 1);
      lap::mbar_init(&sm.item_empty[i], 17);
    }
    for (int i = 0; i < FwdShared<D>::kStages; ++i) {
      lap::mbar_init(&sm.kv_full[i], 1);
      lap::mbar_init(&sm.kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      lap::mbar_init(&sm.q_full[s], 1);
      lap::mbar_init(&sm.q_empty[s], 1);
      lap::mbar_init(&sm.s_full[s], 1);
      lap::mbar_init(&sm.p_ready[s][0], 4);
      lap::mbar_init(&sm.p_ready[s][1], 4);
      lap::mbar_init(&sm.o_full[s], 1);
      lap::mbar_init(&sm.o_free[s], 8);
      for (int w = 0; w < 4; ++w) lap::mbar_init(&sm.pair[s][w], 2);
    }
    lap::mbar_init(&sm.final_bar, 1);
    sm.abort = 0;
    lap::fence_mbar_init();
    lap::tma_prefetch_desc(&maps.q);
    lap::tma_prefetch_desc(&maps.k);
    lap::tma_prefetch_desc(&maps.v);
  }
  lap::tc_fence_before();
  __syncthreads();
  lap::tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  if (tid < 16) sm.bad[tid / 8][tid / 4 % 2][1][tid % 4] = 0;  // D = 64: there is no second box
  if (warp < 16) {
    lap::registers_grow<kSoftmaxRegs>();
    fwd_softmax<D>(sm, p, tmem, tid, abort);
  } else {
    lap::registers_shrink<kOtherRegs>();
    if (warp == 16)
      fwd_products<D>(sm, tmem, lane, abort);
    else if (warp == 17)
      fwd_load<D>(sm, p, maps, lane, abort);
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

}  // namespace laa
