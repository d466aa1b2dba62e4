// la_attention_fwd.cuh -- causal attention over whole prompts (include/la_attention.h) on the tensor
// cores.
//
// A block takes 256 query rows of one head, as two tiles of 128, and walks over the sequence's keys in
// steps of 64, with an unnormalised output and a running maximum and sum per row.
// Warps 0-3 and 4-7 own one query tile each, a thread per row: S is read from tensor memory and p goes
// back over it as the operand of the second product; O is rarely rescaled and always by its owners,
// which need no extra warps for it.  Warp 8 issues the products: for each tile in turn p v of a step,
// then S of the step after next, so that the next step's scores are there when a tile's softmax comes
// to them.  Warp 9 loads: queries once per item, keys and values through a ring of 128-row tiles.
// The two query tiles share keys and values, which halves their traffic from L2.
//
// Steps: an S of 128 x 128 and one operand p over it would fill tensor memory beside two O of D = 128,
// and the next S would wait for p v: a round of both tiles then took 3250 cycles for 2048 cycles of
// products, with a thread or with two per row alike.  With 64 keys there is room for two S of each
// tile; their products read the queries from shared memory twice as often and take 768 cycles
// instead of 512 for 128 keys (measured alone), 2480 for the round.
//
// Bound: the tensor cores at D = 128; at D = 64, where the products halve, the softmax.
#pragma once

#include "la_attention_softmax.cuh"

namespace laa {

constexpr int kFwdRows = 2 * kTile, kStep = 64, kFwdThreads = 320, kItems = 4;

template <int D>
struct alignas(1024) FwdShared {
  static constexpr int kStages = D == 128 ? 5 : 8;
  TileMem<D> q[2];
  TileMem<D> kv[kStages];
  Item items[kItems];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2][2], p_ready[2][2], pv_done[2], o_full[2], o_free[2];
  uint64_t final_bar;
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

// The queue must never run dry, and this warp shares its scheduler with busy ones: it keeps slots and
// parities as running values, its branches over tile and half are unrolled, and it commits no more
// than is waited for.  (Computing them anew cost 1100 cycles a visit where its products take 640.)
template <int D>
__device__ __forceinline__ void fwd_products(FwdShared<D>& sm, uint32_t tmem, int lane, volatile int* abort) {
  constexpr uint32_t kStages = FwdShared<D>::kStages, kSlot = sizeof(TileMem<D>) >> 4;
  constexpr uint32_t id_scores = lap::idesc_bf16_f32(kTile, kStep, false, false);
  constexpr uint32_t id_values = lap::idesc_bf16_f32(kTile, D, false, true);
  const uint32_t q0 = desc_rows(sm.q[0]), k0 = desc_rows(sm.kv[0]), v0 = desc_columns(sm.kv[0]);
  uint32_t slot = 0, phase = 0, items_of[2] = {0, 0}, parity[2] = {0, 0};
  auto advance = [&] {
    if (++slot == kStages) slot = 0, phase ^= 1;
  };
  auto scores = [&](int s, int h, uint32_t k) {
#pragma unroll
    for (int x = 0; x < D / 64; ++x)
      mma4_rows<id_scores>(tmem + s * kTile + h * kStep, q0 + s * kSlot + x * (kBox >> 4),
                           k + h * 512 + x * (kBox >> 4), x > 0);
    commit(&sm.s_full[s][h]);
  };
  bool ok = true;
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t is = i % kItems;
    if (!warp_wait(&sm.item_full[is], (i / kItems) & 1u, abort)) break;
    const Item it = uniform(sm.items[is]);
    warp_arrive(&sm.item_empty[is], lane);
    if (it.len < 0) break;
    const int n[2] = {key_tiles(it, 0), key_tiles(it, 1)};
    const int most = max(n[0], n[1]);
    if (!(ok = warp_wait(&sm.kv_full[slot], phase, abort))) break;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (!ok || !n[s]) continue;
      if (!(ok = warp_wait(&sm.q_full[s], items_of[s] & 1u, abort))) continue;
      lap::tc_fence_after();
      scores(s, 0, k0 + slot * kSlot);
      scores(s, 1, k0 + slot * kSlot);
      if (n[s] == 1) commit(&sm.q_empty[s]);
    }
    if (!ok) break;
    commit(&sm.kv_empty[slot]);
    advance();
    for (int j = 0; j < most; ++j) {
      const uint32_t vs = slot, v = v0 + slot * kSlot;
      if (!(ok = warp_wait(&sm.kv_full[slot], phase, abort))) break;
      advance();
      const uint32_t k = k0 + slot * kSlot;  // of the next tile, where there is one
      const bool more = j + 1 < most;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || j >= n[s]) continue;
          if (!(ok = warp_wait(&sm.p_ready[s][h], parity[s], abort))) continue;
          if (h == 0 && j == 0 && !(ok = warp_wait(&sm.o_free[s], (items_of[s] & 1u) ^ 1u, abort))) continue;
          lap::tc_fence_after();
          mma4_tmem<id_values>(tmem + 2 * kTile + s * D, tmem + s * kTile + h * kStep, v + h * 512, h > 0 || j > 0);
          if (j + 1 < n[s]) {
            // (tile 1 sees every key tile that tile 0 sees, so tile 0 waits for it first if it does)
            if (h == 0 && (s == 0 || j + 1 >= n[0]) && !(ok = warp_wait(&sm.kv_full[slot], phase, abort))) continue;
            scores(s, h, k);
            if (h == 1 && j + 2 == n[s]) commit(&sm.q_empty[s]);
          } else {
            commit(h == 0 ? &sm.pv_done[s] : &sm.o_full[s]);
            if (h == 1) ++items_of[s];
          }
          if (h == 1) parity[s] ^= 1;
        }
      }
      if (!ok) break;
      commit(&sm.kv_empty[vs]);
      if (more) {
        commit(&sm.kv_empty[slot]);
        advance();
      }
    }
  }
  commit(&sm.final_bar);
  drain(&sm.final_bar, 0);  // every product has retired, also after an abort
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void fwd_softmax(FwdShared<D>& sm, const PrefillParams& p, uint32_t tmem, int tid,
                                            volatile int* abort) {
  constexpr int kStages = FwdShared<D>::kStages;
  const int s = tid / kTile, row = tid % kTile, warp = row / 32, lane = tid % 32;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
  const uint32_t t_o = t_lane + 2 * kTile + s * D;
  const float c = p.scale * kLog2e;
  uint32_t slots = 0, steps = 0, uses = 0;
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
    float m = 0.f;
    uint64_t l = 0;
    // One step: 64 keys, of which the row sees the first `keep` (kMasked).
    auto step = [&](auto masked, bool first, bool last, int keep) {
      constexpr bool kMasked = decltype(masked)::value;
      const uint32_t b = steps & 1, t_s = t_lane + s * kTile + b * kStep;
      lap::tc_fence_after();
      float x[kStep];
      const float z = half_scores<kMasked>(t_s, x, c, keep);
      if (first) {
        m = z;
      } else if (__any_sync(0xFFFFFFFFu, z > m + kSlack)) {
        // the scores were made ahead of the last product into O, which has to be done: it is followed by
        // the next step's scores, or in the last step by a commit of its own
        if (!(last ? warp_wait(&sm.pv_done[s], uses & 1u, abort)
                   : warp_wait(&sm.s_full[s][b ^ 1], (steps + 1) >> 1 & 1u, abort)))
          return false;
        lap::tc_fence_after();
        rescale_row<D>(t_o, outgrow(z, m, l));
      }
      uint32_t u[kStep / 2];
      const uint64_t sum = half_probabilities<kMasked>(x, u, c, m, keep);
      lap::tmem_st32_nowait(t_s, u);
      lap::tmem_wait_st();
      lap::tc_fence_before();
      warp_arrive(&sm.p_ready[s][b], lane);
      l = lap::f2_add(l, sum);
      ++steps;
      return true;
    };
    for (int u = 0; u < 2 * n - 2; ++u) {
      if (!warp_wait(&sm.s_full[s][steps & 1], steps >> 1 & 1u, abort)) return;
      if (!step(std::false_type{}, u == 0, false, kStep)) return;
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      // the tile on the diagonal: row r sees its keys 0 .. r; the values of a step are made harmless
      // first.  (The scores, made from the slot before, prove that the ring has come to this phase of
      // the values'.)
      const uint32_t x = first_slot + 2 * (n - 1) + 1;
      if (!warp_wait(&sm.s_full[s][steps & 1], steps >> 1 & 1u, abort)) return;
      if (!warp_wait(&sm.kv_full[x % kStages], (x / kStages) & 1u, abort)) return;
      const int v = kStep * h + row % kStep, box = row / kStep;
      const uint32_t bad =
          __ballot_sync(0xFFFFFFFFu, box < D / 64 && clean_box(sm.kv[x % kStages][box < D / 64 ? box : 0], v, r0 + v >= it.len));
      if (lane == 0) sm.bad[i & 1][s][box][v / 32] = bad;
      lap::fence_proxy_async_smem();
      if (!step(std::true_type{}, n == 1 && h == 0, h == 1, row + 1 - kStep * h)) return;
    }
    const int64_t at = it.lo + r0 + row;
    const bool live = r0 + row < it.len;
    const float2 lp = lap::f2_unpack(l);
    const float total = lp.x + lp.y, inv = 1.f / total;
    if (!warp_wait(&sm.o_full[s], uses++ & 1u, abort)) return;
    lap::tc_fence_after();
    uint32_t bad[4], any_bad = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      bad[w] = sm.bad[i & 1][s][0][w] | sm.bad[i & 1][s][1][w];
      any_bad |= bad[w];
    }
    bf16* out = p.o.row(at, it.head);
#pragma unroll 1
    for (int g = 0; g < D / 32; ++g) {
      float o[32];
      lap::tmem_ld32(t_o + 32 * g, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] *= inv;
      if (any_bad)
        for (int r = 0; r <= row; ++r) {
          const uint32_t w = r < 64 ? (r < 32 ? bad[0] : bad[1]) : (r < 96 ? bad[2] : bad[3]);
          if (w >> (r & 31) & 1u) restore(o, p.v.row(it.lo + r0 + r, it.head / (p.H / p.HK)) + 32 * g);
        }
      if (live) store_row32(out + 32 * g, o);
    }
    lap::tc_fence_before();
    warp_arrive(&sm.o_free[s], lane);
    if (p.lse && live) p.lse[static_cast<int64_t>(it.head) * p.tokens + at] = (m + log2f(total)) * kLn2;
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
  if (warp == 8) {
    lap::tmem_alloc(&sm.tmem, 512);
    lap::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kItems; ++i) {
      lap::mbar_init(&sm.item_full[i], 1);
      lap::mbar_init(&sm.item_empty[i], 9);
    }
    for (int i = 0; i < FwdShared<D>::kStages; ++i) {
      lap::mbar_init(&sm.kv_full[i], 1);
      lap::mbar_init(&sm.kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      lap::mbar_init(&sm.q_full[s], 1);
      lap::mbar_init(&sm.q_empty[s], 1);
      lap::mbar_init(&sm.o_free[s], 4);
      for (int b = 0; b < 2; ++b) {
        lap::mbar_init(&sm.s_full[s][b], 1);
        lap::mbar_init(&sm.p_ready[s][b], 4);
      }
      lap::mbar_init(&sm.pv_done[s], 1);
      lap::mbar_init(&sm.o_full[s], 1);
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
  if (warp < 8)
    fwd_softmax<D>(sm, p, tmem, tid, abort);
  else if (warp == 8)
    fwd_products<D>(sm, tmem, lane, abort);
  else
    fwd_load<D>(sm, p, maps, lane, abort);
  lap::tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort && p.dev_error) atomicOr(p.dev_error, kErrTimeout);
  if (warp == 8) {
    __syncwarp();
    lap::tc_fence_after();
    lap::tmem_dealloc(tmem, 512);
  }
}

}  // namespace laa
