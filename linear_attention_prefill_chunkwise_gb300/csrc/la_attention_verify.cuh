// la_attention_verify.cuh -- drafted tokens (or one token) of many requests over a key/value cache
// (include/la_attention.h) on the tensor cores.
//
// Up to 128 rows per key/value head the work is bound by reading the cache once.  The rows that share a
// key/value head (a request's tokens times the heads of a group, 128 at most at a time) are one tile of
// queries; its keys come 128 at a time from the request's pages, and behind them the drafted tokens' own.  An MMA of 128
// rows takes a fraction of the time that HBM takes for its keys and values, so that rows without a
// token cost nothing that counts.  (A tile of D = 128 is 64 KiB: 1.5 us of an SM's share of HBM
// against 0.55 us of products and about as long for the softmax, which overlaps them.)
//
// Lengths differ and are known on the device only, so the blocks (one per SM) share out the tiles
// of all requests evenly.  Tiles are counted head by head, and within a head request by request, so a
// block has a run of one head's tiles (blocks at work on neighbouring heads of a request then share
// its pages' rows in DRAM: 345 us against 387 with the tiles of a request counted first, for 128
// requests of one token, 64 heads of 128 on 8, up to 8192 tokens in pages of 64).  Its pieces are whole
// items (request, head, query tile), which it writes out, and at its ends parts of items, whose
// unnormalised output, maximum and sum go to the workspace; a second kernel joins the parts of each
// item in order.
//
// That case reads at 0.94 to 0.95 of the copy rate.  A load is a box of one page's rows: pages of 16 (2 KiB a
// box) take 240 us where pages of 32 and more take 197 to 201 (16 requests of 16 tokens; four more warps
// that copy 16 bytes a thread instead, three slots ahead, 268).
//
// More rows than 128 take several query tiles, each of which reads the cache again: 64 requests of 64 heads
// of 128 on 8, 1024 to 8192 cached, take 213 us for trees of 16 (one tile, 0.85 of the copy rate), 402 and
// 453 of 17 and 32 (two), 675 of 64 (four; the products alone 263).
//
// Warps 0-3: softmax, a thread per row; two buffers of scores, so that the product for the next tile
// runs during it.  Warp 4: products.  Warp 5: finds the pieces, looks up pages and loads.
#pragma once

#include "la_attention_softmax.cuh"

namespace laa {

constexpr int kVerifyThreads = 192, kVerifyBlocks = 152, kPieces = 4, kJoinThreads = 256, kJoinShares = 16;

// A block's run of tiles of one item.
struct Piece {
  int b, hk, tile;          // request (< 0: the list ends), key/value head, query tile
  int len;                  // tokens in the cache
  int first, count, tiles;  // tiles of keys first .. first + count - 1 of the item's `tiles`
  int last_block;           // block that holds the item's last tile
};

// What the joining kernel needs to know of an item that begins in a block and ends in another.
struct Split {
  int b, hk, tile, last_block;
};

template <int D>
struct VerifyShared {
  static constexpr int kStages = D == 128 ? 5 : 8;
  TileMem<D> q[2];
  TileMem<D> kv[kStages];
  Piece pieces[kPieces];
  int bad_page[kPieces];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], pv_done[2], o_free;
  uint64_t final_bar;
  uint32_t bad[2][2][4];  // [piece parity][last, last but one drafted tile][warp]: value rows that are not finite
  uint32_t tmem;
  int abort;
};

struct VerifyMaps {
  CUtensorMap q, k, v, k_cache, v_cache;
};

// How items are cut, the same for the whole call.
struct VerifyShape {
  int group, per_tile, q_tiles;  // query heads per key/value head, tokens of a query tile, query tiles
  int box, draft_box;            // rows of a box of the cache and of the drafted tokens
  int rows;                      // rows of a query tile: per_tile * group
  int drafts;                    // tiles of drafted keys, over all query tiles
};

// The workspace: outputs [2 blocks][rows][D], maxima and sums [2 blocks][rows][2], splits [blocks],
// flags [2 blocks] of parts that met a bad page.
struct VerifyParts {
  float* o;
  float2* ml;
  Split* split;
  int* bad;
};
__host__ __device__ inline size_t verify_part_bytes(int rows, int D) {
  return static_cast<size_t>(2 * kVerifyBlocks) * rows * (D + 2) * sizeof(float) +
         kVerifyBlocks * (sizeof(Split) + 2 * sizeof(int));
}
__host__ __device__ inline VerifyParts verify_parts(void* workspace, int rows, int D) {
  VerifyParts w;
  w.o = static_cast<float*>(workspace);
  w.ml = reinterpret_cast<float2*>(w.o + static_cast<size_t>(2 * kVerifyBlocks) * rows * D);
  w.split = reinterpret_cast<Split*>(w.ml + static_cast<size_t>(2 * kVerifyBlocks) * rows);
  w.bad = reinterpret_cast<int*>(w.split + kVerifyBlocks);
  return w;
}

// Tiles of drafted keys that a query tile sees.
__device__ __forceinline__ int draft_tiles(const CacheParams& p, const VerifyShape& v, int tile) {
  return p.mask ? 1 : (min(p.T, (tile + 1) * v.per_tile) + kTile - 1) / kTile;
}

// The pieces of a block, in order.  The batch's tiles count by key/value head first, then by request, query
// tile and tile of keys: with a grid that the heads divide, the blocks that read the same tokens of
// different heads, which lie side by side in the cache, do so at the same time.  Whole-warp calls.
struct PieceWalk {
  int64_t at, end;        // tiles of the whole batch: this block's next, its end
  int64_t line, total;    // tiles of one head, all
  int64_t before = 0;     // tiles of the head before request b0
  int b0 = 0, blocks = 0;
  int len = 0;                 // this lane's request b0 + lane
  int64_t cost = 0, upto = 0;  // its tiles of a head, and those up to it
  bool loaded = false;

  __device__ __forceinline__ int64_t tiles_of(const CacheParams& p, const VerifyShape& v, int b, int& n) const {
    n = b < p.B ? __ldg(p.cache_lens + b) : -1;
    if (n < 0) return 0;
    if (n > capacity(p)) {
      if (blockIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, kErrSeqlens);
      return 0;
    }
    return static_cast<int64_t>(v.q_tiles) * ((n + kTile - 1) / kTile) + v.drafts;
  }

  __device__ PieceWalk(const CacheParams& p, const VerifyShape& v, int lane) {
    line = 0;
    for (int b = lane; b < p.B; b += 32) {
      int n;
      line += tiles_of(p, v, b, n);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) line += __shfl_xor_sync(0xFFFFFFFFu, line, d);
    total = line * p.HK;
    // no more blocks than tiles, so that none between two others is without one
    blocks = total < gridDim.x ? static_cast<int>(total) : static_cast<int>(gridDim.x);
    at = end = 0;
    if (static_cast<int>(blockIdx.x) < blocks) {
      at = total * blockIdx.x / blocks;
      end = total * (blockIdx.x + 1) / blocks;
    }
  }

  // The block that holds a tile.
  __device__ __forceinline__ int block_of(int64_t tile) const {
    return static_cast<int>(((tile + 1) * blocks - 1) / total);
  }

  __device__ __forceinline__ Piece take(const CacheParams& p, const VerifyShape& v, int lane) {
    Piece pc{-1, 0, 0, 0, 0, 0, 0, 0};
    if (at >= end) return pc;
    pc.hk = static_cast<int>(at / line);
    const int64_t place = at - pc.hk * line;
    if (place < before) before = 0, b0 = 0, loaded = false;  // the next head: from the first request
    for (;;) {  // place < line, so some request holds it
      if (!loaded) {
        cost = tiles_of(p, v, b0 + lane, len);
        upto = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
          if (lane >= d) upto += o;
        }
        loaded = true;
      }
      const uint32_t reach = __ballot_sync(0xFFFFFFFFu, before + upto > place);
      if (reach) {
        const int l = __ffs(reach) - 1;
        pc.b = b0 + l;
        pc.len = __shfl_sync(0xFFFFFFFFu, len, l);
        int64_t x = place - (before + __shfl_sync(0xFFFFFFFFu, upto, l) - __shfl_sync(0xFFFFFFFFu, cost, l));
        const int ct = (pc.len + kTile - 1) / kTile;
        pc.tiles = ct + draft_tiles(p, v, 0);
        while (x >= pc.tiles) {
          x -= pc.tiles;
          pc.tiles = ct + draft_tiles(p, v, ++pc.tile);
        }
        pc.first = static_cast<int>(x);
        pc.last_block = block_of(at + pc.tiles - 1 - x);
        pc.count = static_cast<int>(min(static_cast<int64_t>(pc.tiles) - x, end - at));
        at += pc.count;
        return pc;
      }
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
      b0 += 32;
      loaded = false;
      if (b0 >= p.B) return Piece{-1, 0, 0, 0, 0, 0, 0, 0};
    }
  }
};

template <int D>
__device__ __forceinline__ void verify_load(VerifyShared<D>& sm, const CacheParams& p, const VerifyShape& v,
                                            const VerifyMaps& maps, int lane, volatile int* abort) {
  constexpr int kStages = VerifyShared<D>::kStages;
  PieceWalk walk(p, v, lane);
  if (lane == 0) verify_parts(p.part, v.rows, D).split[blockIdx.x].b = -1;
  const int boxes = kTile / v.box;
  uint32_t slots = 0, items = 0, q_loads = 0;
  bool ok = true;
  for (; ok; ++items) {
    const uint32_t is = items % kPieces;
    if (!warp_wait(&sm.piece_empty[is], ((items / kPieces) & 1u) ^ 1u, abort)) break;
    const Piece pc = walk.take(p, v, lane);
    if (lane == 0) {
      sm.pieces[is] = pc;
      sm.bad_page[is] = 0;
      lap::mbar_arrive(&sm.piece_full[is]);
    }
    __syncwarp();
    if (pc.b < 0) break;
    const int cached = (pc.len + kTile - 1) / kTile, qs = items & 1;
    // this lane's box of the next 32: its page, and its first row in it
    int page = pc.b, slot = 0;
    for (int j = pc.first, done = 0; done < pc.count && ok; ++j, ++done) {
      const int fetched = j * boxes % 32;
      if (j < cached && p.page_table && (done == 0 || fetched == 0)) {
        const int64_t row = static_cast<int64_t>(j * boxes - fetched + lane) * v.box;
        if (row < pc.len && row + v.box > static_cast<int64_t>(j) * kTile) {
          page = __ldg(p.page_table + pc.b * p.ld_table + row / p.page_size);
          slot = static_cast<int>(row % p.page_size);
          if (page < 0 || page >= p.pages) {
            sm.bad_page[is] = 1;
            if (p.dev_error) atomicOr(p.dev_error, kErrIndex);
            page = 0;
          }
        }
        __syncwarp();
      }
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const uint32_t st = slots % kStages;
        if (!(ok = warp_wait(&sm.kv_empty[st], ((slots / kStages) & 1u) ^ 1u, abort))) break;
        uint64_t* bar = &sm.kv_full[st];
        if (j >= cached) {
          if (lane == 0) {
            const CUtensorMap* map = kv ? &maps.v : &maps.k;
            lap::mbar_arrive_expect_tx(bar, v.draft_box * 128 * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              lap::tma_load_3d(sm.kv[st][h], map, bar, 64 * h, pc.hk, pc.b * p.T + (j - cached) * kTile);
          }
        } else {
          const CUtensorMap* map = kv ? &maps.v_cache : &maps.k_cache;
          const int here = min(boxes, (pc.len - j * kTile + v.box - 1) / v.box);
          if (lane == 0) lap::mbar_arrive_expect_tx(bar, here * v.box * 128 * (D / 64));
          __syncwarp();
          if (p.page_table) {
            // lane `fetched + x` issues its own box x of the tile
            const int x = lane - fetched;
            if (x >= 0 && x < here)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                lap::tma_load_4d(sm.kv[st][h] + x * v.box * 128, map, bar, 64 * h, pc.hk, slot, page);
          } else if (lane == 0) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) lap::tma_load_4d(sm.kv[st][h], map, bar, 64 * h, pc.hk, j * kTile, pc.b);
          }
        }
        __syncwarp();
        ++slots;
        if (kv == 0 && done == 0) {
          if (!(ok = warp_wait(&sm.q_empty[qs], ((items >> 1) & 1u) ^ 1u, abort))) break;
          if (lane == 0) {
            lap::mbar_arrive_expect_tx(&sm.q_full[qs], v.rows * 128 * (D / 64));
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              lap::tma_load_3d(sm.q[qs][h], &maps.q, &sm.q_full[qs], 64 * h, pc.hk * v.group, pc.b * p.T + pc.tile * v.per_tile);
          }
          ++q_loads;
          __syncwarp();
        }
      }
    }
  }
  // every load has landed before the block's shared memory is given up, also after an abort
  if (lane == 0) {
    for (uint32_t i = 0; i < static_cast<uint32_t>(kStages) && i < slots; ++i) {
      const uint32_t j = slots - 1 - i;
      drain(&sm.kv_full[j % kStages], (j / kStages) & 1u);
    }
    for (uint32_t i = 0; i < 2 && i < q_loads; ++i) drain(&sm.q_full[(q_loads - 1 - i) & 1], ((q_loads - 1 - i) >> 1) & 1u);
  }
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void verify_products(VerifyShared<D>& sm, uint32_t tmem, int lane, volatile int* abort) {
  constexpr int kStages = VerifyShared<D>::kStages;
  uint32_t slots = 0, tiles = 0;
  bool ok = true;
  auto wait_slot = [&](uint32_t x) { return warp_wait(&sm.kv_full[x % kStages], (x / kStages) & 1u, abort); };
  for (uint32_t i = 0; ok; ++i) {
    const uint32_t is = i % kPieces, qs = i & 1;
    if (!warp_wait(&sm.piece_full[is], (i / kPieces) & 1u, abort)) break;
    const int count = uniform(sm.pieces[is].b < 0 ? 0 : sm.pieces[is].count);
    warp_arrive(&sm.piece_empty[is], lane);
    if (count == 0) break;
    // the scores of tile j go to buffer (tiles + j) & 1, whose last probabilities the product of tile
    // j - 2 has read by then (it is before them in the queue)
    auto scores = [&](int j) {
      const uint32_t x = slots + 2 * j;
      if (!wait_slot(x)) return false;
      lap::tc_fence_after();
      product_rows<D>(tmem + ((tiles + j) & 1) * kTile, desc_rows(sm.q[qs]), desc_rows(sm.kv[x % kStages]));
      commit(&sm.s_full[(tiles + j) & 1]);
      commit(&sm.kv_empty[x % kStages]);
      if (j == count - 1) commit(&sm.q_empty[qs]);
      return true;
    };
    if (!(ok = warp_wait(&sm.q_full[qs], (i >> 1) & 1u, abort)) || !(ok = scores(0))) break;
    for (int j = 0; j < count && ok; ++j) {
      if (j + 1 < count && !(ok = scores(j + 1))) break;
      const uint32_t x = slots + 2 * j + 1, t = tiles + j;
      if (!(ok = wait_slot(x)) || !(ok = warp_wait(&sm.p_ready[t & 1], (t >> 1) & 1u, abort))) break;
      if (j == 0 && !(ok = warp_wait(&sm.o_free, (i & 1u) ^ 1u, abort))) break;
      lap::tc_fence_after();
      product_tmem<D>(tmem + 2 * kTile, tmem + (t & 1) * kTile, desc_columns(sm.kv[x % kStages]), j > 0);
      commit(&sm.pv_done[t & 1]);
      commit(&sm.kv_empty[x % kStages]);
    }
    slots += 2 * count;
    tiles += count;
  }
  commit(&sm.final_bar);
  drain(&sm.final_bar, 0);  // every product has retired, also after an abort
  __syncwarp();
}

template <int D>
__device__ __forceinline__ void verify_softmax(VerifyShared<D>& sm, const CacheParams& p, const VerifyShape& v,
                                               uint32_t tmem, int row, volatile int* abort) {
  constexpr int kStages = VerifyShared<D>::kStages;
  const int warp = row / 32, lane = row % 32;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16), t_o = t_lane + 2 * kTile;
  const float c = p.scale * kLog2e;
  const VerifyParts parts = verify_parts(p.part, v.rows, D);
  uint32_t slots = 0, tiles = 0;
  for (uint32_t i = 0;; ++i) {
    const uint32_t is = i % kPieces;
    if (!warp_wait(&sm.piece_full[is], (i / kPieces) & 1u, abort)) return;
    const Piece pc = sm.pieces[is];
    if (pc.b < 0) {
      warp_arrive(&sm.piece_empty[is], lane);
      return;
    }
    const int t = pc.tile * v.per_tile + row / v.group;  // this row's token
    const bool live = row < v.rows && t < p.T;
    const bool busy = __any_sync(0xFFFFFFFFu, live);     // a warp without rows only keeps step
    const int cached = (pc.len + kTile - 1) / kTile, drafts = pc.tiles - cached;
    uint64_t mask = 0;
    if (p.mask && live) mask = static_cast<uint64_t>(__ldg(p.mask + static_cast<int64_t>(pc.b) * p.T + t));
    if (p.T < 64) mask &= (1ull << p.T) - 1;
    float m = 0.f;
    uint64_t l = 0;
    if (lane < 2) sm.bad[i & 1][lane][warp] = 0;
    __syncwarp();
    for (int j = 0; j < pc.count; ++j, ++tiles) {
      const int x = pc.first + j, d = x - cached;  // tile of the item, of the drafted tokens
      const uint32_t buf = tiles & 1, t_s = t_lane + buf * kTile;
      const int valid = min(kTile, d < 0 ? pc.len - x * kTile : p.T - d * kTile);
      Keys keys{valid, {0, 0}};
      bool all = valid == kTile;
      if (d >= 0) {
        keys.keep = t - d * kTile + 1;  // of drafted tokens without a mask
        keys.bits[0] = static_cast<uint32_t>(mask);
        keys.bits[1] = static_cast<uint32_t>(mask >> 32);
        all = false;
      }
      if (!warp_wait(&sm.s_full[buf], (tiles >> 1) & 1u, abort)) return;
      if (!all) {
        // values that some row must not see: rows behind the tokens, drafted tokens that are masked
        // (the scores prove that the ring slot's last contents have been used: its phase is this one)
        const uint32_t xs = slots + 2 * j + 1;
        if (!warp_wait(&sm.kv_full[xs % kStages], (xs / kStages) & 1u, abort)) return;
        const bool behind = row >= valid, masked = d >= drafts - 2 && d >= 0;
        const bool found = (masked || behind) && clean_row<D>(sm.kv[xs % kStages], row, behind);
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, found);
        // (drafted tiles before the last two are seen whole, by every row)
        if (masked && lane == 0) sm.bad[i & 1][drafts - 1 - d][warp] = bad;
        lap::fence_proxy_async_smem();
      }
      if (busy) {
        lap::tc_fence_after();
        float s[kTile];
        auto step = [&](auto seen) {
          constexpr Seen kSeen = decltype(seen)::value;
          const float z = load_scores<kSeen>(t_s, s, c, keys);
          if (j == 0) {
            m = first_maximum(z);
          } else if (__any_sync(0xFFFFFFFFu, z > m + kSlack)) {
            // the scores were made ahead of the last product into O: it has to be done
            if (!warp_wait(&sm.pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1u, abort)) return false;
            lap::tc_fence_after();
            rescale_row<D>(t_o, outgrow(z, m, l));
          }
          probabilities<kSeen>(s, 0, t_s, c, m, keys);
          probabilities<kSeen>(s, 1, t_s, c, m, keys);
          return true;
        };
        const bool done = all                 ? step(std::integral_constant<Seen, kAll>{})
                          : d >= 0 && p.mask ? step(std::integral_constant<Seen, kBits>{})
                                              : step(std::integral_constant<Seen, kFirst>{});
        if (!done) return;
        lap::tc_fence_before();
        warp_arrive(&sm.p_ready[buf], lane);
        add_sums(s, l);
      } else {
        warp_arrive(&sm.p_ready[buf], lane);
      }
    }
    slots += 2 * pc.count;
    if (!warp_wait(&sm.pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1u, abort)) return;
    lap::tc_fence_after();
    const float2 lp = lap::f2_unpack(l);
    const float total = lp.x + lp.y;
    const bool whole = pc.count == pc.tiles;
    const bool skip = *static_cast<volatile int*>(&sm.bad_page[is]) != 0;
    const int part = 2 * blockIdx.x + (pc.first == 0);  // where a part goes: see Split
    const float inv = !whole ? 1.f : total == 0.f ? 0.f : 1.f / total;
    uint32_t any_bad = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) any_bad |= sm.bad[i & 1][w >> 2][w & 3];
    if (busy) {
      bf16* out = p.o.row(static_cast<int64_t>(pc.b) * p.T + t, pc.hk * v.group + row % v.group);
      float4* part_out = reinterpret_cast<float4*>(parts.o + (static_cast<int64_t>(part) * v.rows + row) * D);
#pragma unroll 1
      for (int g = 0; g < D / 32; ++g) {
        float o[32];
        lap::tmem_ld32(t_o + 32 * g, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (any_bad && live)
          for (int w = 0; w < 8; ++w)
            for (uint32_t bits = sm.bad[i & 1][w >> 2][w & 3]; bits; bits &= bits - 1) {
              const int u = (drafts - 1 - (w >> 2)) * kTile + 32 * (w & 3) + __ffs(bits) - 1;
              if (p.mask ? (mask >> u & 1) != 0 : u <= t)
                restore(o, p.v.row(static_cast<int64_t>(pc.b) * p.T + u, pc.hk) + 32 * g);
            }
        if (!live || (whole && skip)) continue;
        if (whole) {
          store_row32(out + 32 * g, o);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) part_out[8 * g + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (live && !whole) parts.ml[static_cast<int64_t>(part) * v.rows + row] = make_float2(m, total);
    }
    if (!whole && row == 0) {
      parts.bad[part] = skip;
      if (pc.first == 0) parts.split[blockIdx.x] = Split{pc.b, pc.hk, pc.tile, pc.last_block};
    }
    lap::tc_fence_before();
    warp_arrive(&sm.o_free, lane);
    warp_arrive(&sm.piece_empty[is], lane);
  }
}

template <int D>
__global__ void __launch_bounds__(kVerifyThreads, 1)
attn_verify_kernel(const __grid_constant__ VerifyMaps maps, const __grid_constant__ CacheParams p,
                   const __grid_constant__ VerifyShape v) {
  extern __shared__ uint8_t smem_raw[];
  VerifyShared<D>& sm =
      *reinterpret_cast<VerifyShared<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32;
  volatile int* abort = &sm.abort;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  if (warp == 4) {
    lap::tmem_alloc(&sm.tmem, 512);
    lap::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) {
      lap::mbar_init(&sm.piece_full[i], 1);
      lap::mbar_init(&sm.piece_empty[i], 5);
    }
    for (int i = 0; i < VerifyShared<D>::kStages; ++i) {
      lap::mbar_init(&sm.kv_full[i], 1);
      lap::mbar_init(&sm.kv_empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      lap::mbar_init(&sm.q_full[s], 1);
      lap::mbar_init(&sm.q_empty[s], 1);
      lap::mbar_init(&sm.s_full[s], 1);
      lap::mbar_init(&sm.p_ready[s], 4);
      lap::mbar_init(&sm.pv_done[s], 1);
    }
    lap::mbar_init(&sm.o_free, 4);
    lap::mbar_init(&sm.final_bar, 1);
    sm.abort = 0;
    lap::fence_mbar_init();
    lap::tma_prefetch_desc(&maps.q);
    lap::tma_prefetch_desc(&maps.k);
    lap::tma_prefetch_desc(&maps.v);
    lap::tma_prefetch_desc(&maps.k_cache);
    lap::tma_prefetch_desc(&maps.v_cache);
  }
  lap::tc_fence_before();
  __syncthreads();
  lap::tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  if (warp < 4)
    verify_softmax<D>(sm, p, v, tmem, tid, abort);
  else if (warp == 4)
    verify_products<D>(sm, tmem, lane, abort);
  else
    verify_load<D>(sm, p, v, maps, lane, abort);
  lap::tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort && p.dev_error) atomicOr(p.dev_error, kErrTimeout);
  if (warp == 4) {
    __syncwarp();
    lap::tc_fence_after();
    lap::tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the items that begin in block blockIdx.x of the kernel above and end in
// another: parts 2 c + 1 of that block c, then 2 (c + 1), .. of the blocks up to the last, in order.
// Few parts: a warp per row.  Many (few, long requests): a block per row, its warps taking the parts
// in turn, their sums added in order.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ CacheParams p,
                                                                 const __grid_constant__ VerifyShape v) {
  constexpr int kWarps = kJoinThreads / 32, kEach = D / 32;
  __shared__ float sums[kWarps][D];
  __shared__ float tops[kWarps], weights[kWarps];
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const VerifyParts parts = verify_parts(p.part, v.rows, D);
  const int c = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Split sp = parts.split[c];
  if (sp.b < 0) return;
  const int n = sp.last_block - c + 1;
  auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
  const bool wide = n > 32;  // each way, `step` warps share a row's parts, from part `first`
  const int step = wide ? kWarps : 1, first = wide ? warp : 0;
  bool bad = false;
  for (int i = lane; i < n; i += 32) bad = bad || parts.bad[slot(i)];
  if (__any_sync(0xFFFFFFFFu, bad)) return;
  const int rows_at_once = wide ? 1 : kWarps;
  for (int r0 = blockIdx.y * rows_at_once; r0 < v.rows; r0 += gridDim.y * rows_at_once) {
    const int row = r0 + (wide ? 0 : warp), t = sp.tile * v.per_tile + row / v.group;
    const bool live = row < v.rows && t < p.T;
    float top = -INFINITY;
    if (live)
      for (int i = wide ? threadIdx.x : lane; i < n; i += wide ? kJoinThreads : 32) {
        const float2 ml = parts.ml[static_cast<int64_t>(slot(i)) * v.rows + row];
        if (ml.y != 0.f) top = fmaxf(top, ml.x);
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (wide) {
      if (lane == 0) tops[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    }
    float acc[kEach] = {}, total = 0.f;
    if (live)
#pragma unroll 4
      for (int i = first; i < n; i += step) {
        const int64_t at = static_cast<int64_t>(slot(i)) * v.rows + row;
        const float2 ml = parts.ml[at];
        const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
        total += w * ml.y;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const float o = parts.o[at * D + kEach * lane + e];
          acc[e] = ml.y == 0.f ? acc[e] : fmaf(w, o, acc[e]);
        }
      }
    if (wide) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) sums[warp][kEach * lane + e] = acc[e];
      if (lane == 0) weights[warp] = total;
      __syncthreads();
      total = 0.f;
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        total += weights[k];
#pragma unroll
        for (int e = 0; e < kEach; ++e) acc[e] += sums[k][kEach * lane + e];
      }
    }
    if (live && (!wide || warp == 0)) {
      bf16* out = p.o.row(static_cast<int64_t>(sp.b) * p.T + t, sp.hk * v.group + row % v.group) + kEach * lane;
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] = total == 0.f ? 0.f : acc[e] / total;
      if constexpr (kEach == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(lap::pack_bf16x2(acc[0], acc[1]), lap::pack_bf16x2(acc[2], acc[3]));
      else
        *reinterpret_cast<uint32_t*>(out) = lap::pack_bf16x2(acc[0], acc[1]);
    }
    if (wide) __syncthreads();
  }
}

}  // namespace laa
