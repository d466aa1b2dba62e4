// la_attention_fwd.cuh -- causal attention over whole prompts (include/la_attention.h) on the tensor
// cores.
//
// A block takes 256 query rows of one head, as two tiles of 128, and walks over the sequence's keys,
// 128 at a time, with an unnormalised output and a running maximum and sum per row.
// Warps 0-3 and 4-7 own one query tile each, a thread per row: S is read from tensor memory and p goes
// back over it as the operand of the second product, a half at a time; O is rarely rescaled and always
// by its owners, which need no extra warps for it.  Warp 8 issues the products: while one tile's
// softmax runs, the other tile's two products keep the tensor cores busy (p v and the next S of each in
// turn, in one queue, so that S can overwrite p).  Warp 9 loads: queries once per item, keys and values
// through a ring.  The two tiles share keys and values, which halves their traffic from L2.
//
// Bound: the tensor cores at D = 128 (2 x 8192 tokens, 64 heads of 128 on 8: 1.40 ms, 1.57 PFLOP/s, where
// the power limit holds the clock; 1.28 ms when cool).  At D = 64, where the products halve, the latency of
// handing scores and probabilities over: 1229 cycles per tile of scores and SM (1524 at D = 128) for 768 of
// products and 512 of the special function unit.  The tensor pipe and that unit are busy 37 % of the time and
// issue slots 42 %, as a tile's next S waits until its p v has read p from the same columns (8192 tokens,
// 16 heads of 64: 138 us, 0.51 of the tensor cores' rate).
// Measured against it on the first case: two threads per row, which meet to agree on a maximum, 1.57 ms; steps
// of 64 keys with two buffers of scores per tile, whose products read the queries twice as often, 1.53 ms;
// half of p made before the new maximum is known, 1.61 ms.
#pragma once

#include "la_attention_softmax.cuh"

namespace laa {

constexpr int kFwdRows = 2 * kTile, kFwdThreads = 384, kItems = 4;
// Registers: 3 x 168 at launch; a softmax thread holds a row of scores.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "register shares");
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
  uint32_t bad[kItems][2][4];  // [item][tile][warp]: value rows on its diagonal that are not finite
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
// parities as running values, its branches over tiles and halves are unrolled, and it commits no more
// than is waited for.
template <int D>
__device__ __forceinline__ void fwd_products(FwdShared<D>& sm, uint32_t tmem, int lane, volatile int* abort) {
  constexpr uint32_t kStages = FwdShared<D>::kStages, kSlot = sizeof(TileMem<D>) >> 4;
  const uint32_t q0 = desc_rows(sm.q[0]), k0 = desc_rows(sm.kv[0]), v0 = desc_columns(sm.kv[0]);
  uint32_t slot = 0, phase = 0, items_of[2] = {0, 0}, parity[2] = {0, 0};
  auto advance = [&] {
    if (++slot == kStages) slot = 0, phase ^= 1;
  };
  auto scores = [&](int s, uint32_t k) {
    product_rows<D>(tmem + s * kTile, q0 + s * kSlot, k);
    commit(&sm.s_full[s]);
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
      scores(s, k0 + slot * kSlot);
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
      for (int s = 0; s < 2; ++s) {
        if (!ok || j >= n[s]) continue;
        const uint32_t t_o = tmem + 2 * kTile + s * D, t_p = tmem + s * kTile;
        if (!(ok = warp_wait(&sm.p_ready[s][0], parity[s], abort))) continue;
        if (j == 0 && !(ok = warp_wait(&sm.o_free[s], (items_of[s] & 1u) ^ 1u, abort))) continue;
        lap::tc_fence_after();
        half_product_tmem<D>(t_o, t_p, v, 0, j > 0);
        if (!(ok = warp_wait(&sm.p_ready[s][1], parity[s], abort))) continue;
        parity[s] ^= 1;
        lap::tc_fence_after();
        half_product_tmem<D>(t_o, t_p, v, 1, true);
        if (j + 1 < n[s]) {
          // (tile 1 sees every key tile that tile 0 sees, so tile 0 waits for it if it does)
          if ((s == 0 || j + 1 >= n[0]) && !(ok = warp_wait(&sm.kv_full[slot], phase, abort))) continue;
          scores(s, k);
          if (j + 2 == n[s]) commit(&sm.q_empty[s]);
        } else {
          commit(&sm.o_full[s]);
          ++items_of[s];
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
  const uint32_t t_s = tmem + s * kTile + (static_cast<uint32_t>(32 * warp) << 16);
  const uint32_t t_o = tmem + 2 * kTile + s * D + (static_cast<uint32_t>(32 * warp) << 16);
  const float c = p.scale * kLog2e;
  const Keys keys{row + 1, {0, 0}};
  uint32_t slots = 0, tiles = 0, uses = 0;
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kItems;
    if (!warp_wait(&sm.item_full[is], (i / kItems) & 1u, abort)) return;
    const Item it = sm.items[is];
    if (it.len < 0) return;
    const int n = key_tiles(it, s), first_slot = slots;
    slots += 2 * max(n, key_tiles(it, s ^ 1));
    if (n == 0) {
      warp_arrive(&sm.item_empty[is], lane);
      continue;
    }
    const int r0 = it.tile * kFwdRows + s * kTile;
    float m = 0.f;
    uint64_t l = 0;
    float scores[kTile];
    auto step = [&](auto seen, bool first) {
      constexpr Seen kSeen = decltype(seen)::value;
      lap::tc_fence_after();
      const float z = load_scores<kSeen>(t_s, scores, c, keys);
      // S follows the last product into O in the queue, so O may be rescaled
      if (first)
        m = first_maximum(z);
      else if (__any_sync(0xFFFFFFFFu, z > m + kSlack))
        rescale_row<D>(t_o, outgrow(z, m, l));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        probabilities<kSeen>(scores, half, t_s, c, m, keys);
        lap::tc_fence_before();
        warp_arrive(&sm.p_ready[s][half], lane);
      }
      add_sums(scores, l);
    };
    for (int j = 0; j < n - 1; ++j) {
      if (!warp_wait(&sm.s_full[s], tiles++ & 1u, abort)) return;
      step(std::integral_constant<Seen, kAll>{}, j == 0);
    }
    {
      // the tile on the diagonal: row r sees its keys 0 .. r; its values are made harmless first.  (The
      // scores, made from the slot before, prove that the ring has come to this phase of the values'.)
      const uint32_t x = first_slot + 2 * (n - 1) + 1;
      if (!warp_wait(&sm.s_full[s], tiles++ & 1u, abort)) return;
      if (!warp_wait(&sm.kv_full[x % kStages], (x / kStages) & 1u, abort)) return;
      const uint32_t bad =
          __ballot_sync(0xFFFFFFFFu, clean_row<D>(sm.kv[x % kStages], row, r0 + row >= it.len));
      if (lane == 0) sm.bad[is][s][warp] = bad;
      lap::fence_proxy_async_smem();
      step(std::integral_constant<Seen, kFirst>{}, n == 1);
    }
    const float2 lp = lap::f2_unpack(l);
    const float total = lp.x + lp.y, inv = 1.f / total;
    const int64_t at = it.lo + r0 + row;
    const bool live = r0 + row < it.len;
    if (!warp_wait(&sm.o_full[s], uses++ & 1u, abort)) return;
    lap::tc_fence_after();
    // Tile 1 reads the values on tile 0's diagonal from the same memory: what was taken out of them
    // there it gets back as well, every row of it.
    uint32_t any_bad = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) any_bad |= sm.bad[is][s][w] | (s ? sm.bad[is][0][w] : 0u);
    bf16* out = p.o.row(at, it.head);
#pragma unroll 1
    for (int g = 0; g < D / 32; ++g) {
      float o[32];
      lap::tmem_ld32(t_o + 32 * g, o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] *= inv;
      if (any_bad)
        for (int x = 0; x <= s; ++x)
          for (int r = 0; r < kTile && (x < s || r <= row); ++r)
            if (sm.bad[is][x][r >> 5] >> (r & 31) & 1u)
              restore(o, p.v.row(it.lo + it.tile * kFwdRows + x * kTile + r, it.head / (p.H / p.HK)) + 32 * g);
      if (live) store_row32(out + 32 * g, o);
    }
    lap::tc_fence_before();
    warp_arrive(&sm.o_free[s], lane);
    warp_arrive(&sm.item_empty[is], lane);
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
      lap::mbar_init(&sm.s_full[s], 1);
      lap::mbar_init(&sm.p_ready[s][0], 4);
      lap::mbar_init(&sm.p_ready[s][1], 4);
      lap::mbar_init(&sm.o_full[s], 1);
      lap::mbar_init(&sm.o_free[s], 4);
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
  if (warp < 8) {
    lap::registers_grow<kSoftmaxRegs>();
    fwd_softmax<D>(sm, p, tmem, tid, abort);
  } else {
    lap::registers_shrink<kOtherRegs>();
    if (warp == 8)
      fwd_products<D>(sm, tmem, lane, abort);
    else if (warp == 9)
      fwd_load<D>(sm, p, maps, lane, abort);
  }
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
