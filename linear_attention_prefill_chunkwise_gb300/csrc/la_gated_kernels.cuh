// la_gated_kernels.cuh -- kernels of the gated linear recurrence (include/la_gated.h).
//
// The scan.  With a_t = lambda_t and b_t the token's input (beta_t sig(g_t) x_t forward; lambda_t
// dout_t backward, where the state is w_t = lambda_t G_t and tokens are walked from the end), a
// run of tokens maps the state before it to A h + H, A the product of its a's and H its own scan
// from zero; two runs compose as (A2 A1, A2 H1 + H2).
//
// A tile is kWarps x kRows rows of 64 channels, two channels per lane, kRows rows per warp.  Blocks
// are persistent, and each warp has two stages of shared memory for its rows of the inputs: while
// one tile is computed the loads of the next are in flight, each warp's own TMA boxes (or, where
// rows are not 16-byte aligned, its own asynchronous 16-byte copies), so no warp waits for another's
// loads.  A warp composes its rows, the block its warps; once the state before the tile is known,
// each warp walks its rows again (forward: from a and b in registers) and writes the outputs: every
// input is read once and every output written once.  What bounds it is the bytes, then the
// instructions: a row of 64 channels takes a warp 62 forward and 126 for the gradients by chains (0.60
// and 0.63 of the issue slots), 74 forward by tiles (0.51), 207 for unaligned gradients (0.51).
// Measured, BF16, of the bytes at the copy rate: 2 x 8192 tokens of 8192 channels 195 us (0.81),
// gradients 389 (0.81; 19 x 1024 tokens 398, 0.94); 32 packed sequences of up to 4096 tokens of 4096
// channels 303 (0.93); one sequence of 32768 x 4096 240 (0.66), of 131072 x 1024 313 (0.51: the states'
// way from block to block); FP32 8192 x 8192 174 (0.91).
//
// Where the state before a tile comes from (Mode):
// By chains, from the block itself, which walks all tiles of a sequence's channels: nothing waits.
// By tiles, from the blocks that computed the tiles before it.  Tiles are taken in order (by a
// ticket, so that whatever a block waits for is already running), in groups along the sequence.  A
// tile's (A, H) is published in the workspace; a tile composes the published ones before it in its
// group, in order, onto the state that the previous group's last tile published: a long scan is a
// chain of one step per group, not per tile.
// Batches of short packed sequences are one scan over all rows whose state is replaced where a
// sequence begins (kMixed), cut whatever the sequences' lengths.
// The order of every sum is fixed, so results repeat bitwise.
//
// A published word carries its own readiness: the workspace is filled with all-ones before the
// scan, no published word is all-ones, and a reader looks at the words themselves: no fence and no
// second flag on the way from block to block.  A tile asks for the words it needs (one per warp)
// before it computes its last rows, by asynchronous copies, and polls only where one was late.
// Where a sequence begins inside a tile, A becomes -0: products of decays are >= +0, so the sign
// marks "what came before does not matter", and composition then selects H instead of multiplying,
// which keeps infinities and NaN of one sequence out of the next.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "la_gated_math.cuh"
#include "sm103_ptx.cuh"

namespace lag {

constexpr unsigned kErrBadSeqlens = 1u, kErrBadIndex = 2u, kErrTimeout = 4u;
constexpr int kCols = 64;       // channels of a tile: two per lane
constexpr int kThreads = 128;   // threads of the small kernels
constexpr int kMaxInputs = 5;   // x, r, g; backward: dout and o (one row up: h_{t-1}) too
constexpr int kStages = 2;

// How blocks take their work; each is a kernel of its own, since the loop is held up by its own
// instructions and registers (2 x 8192 tokens x 8192 channels by chains, one kernel for all was slower
// by a tenth, when the kernels were split: 1.18 stalls per issue for missing instructions, now 0.13).
enum Mode {
  kByChains,  // one block walks all tiles of a sequence's channels
  kByTiles,   // tiles of one sequence each, states from block to block
  kMixed      // tiles that hold rows of several sequences: packed (states from block to block) or whole ones
};

// Shape of a scan kernel: rows per warp, blocks per SM and the stages' layout.  kTma: rows arrive
// by TMA boxes of kRows x 64 channels; else by 16-byte copies of the aligned chunks that a row's
// channels touch, one chunk more than the channels fill.
// Rows per warp: as many as two blocks' registers (forward: a and b of each) and shared memory hold,
// since every tile costs the same few hundred instructions; more of them spill, or leave the copies
// no cache.  BF16, 2 x 8192 tokens of 8192 channels: forward 18 rows 233 us, 16 195, 14 207, 12 210.
// Gradients by chains 9 rows 380, 8 388, 7 407, and of 32 x 1024 tokens of 4096 channels 365, 346, 358;
// by tiles (32768 tokens of 4096 channels) 10 rows 537, 9 451, 8 474.  Unaligned, 32 sequences of up to
// 4096 tokens of 1001 channels: forward 14 rows 178, 12 171, 11 174, 10 180; gradients 9 rows 444, 8 318,
// 7 329, 6 341, but of 600 sequences of up to 128 tokens of 2047 channels 493, 487, 476, 460.
// FP32, 8192 tokens of 4096 channels: gradients by tiles 5 rows 229, 4 212, 3 253; by chains (2 x 4096
// tokens of 8192 channels) 4 rows 367.
template <typename E, bool kBack, bool kTma, Mode kMode>
struct Shape {
  static constexpr int kWarps = 8;
  static constexpr int kRows = (kBack ? (!kTma ? 6 : kMode == kByChains ? 8 : 9) : (kTma ? 16 : 12)) / (sizeof(E) / 2);
  static constexpr int kBlocks = 2;
  static constexpr int kAsk = kRows * 5 / 8;  // the row before which a warp asks for the published words
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTileRows = kWarps * kRows;
  static constexpr int kInputs = kBack ? 5 : 3;
  static constexpr int kPitch = kCols * sizeof(E) + (kTma ? 0 : 16);  // bytes of a row
  static constexpr int kInputBytes = kTileRows * kPitch;
  static constexpr int kStageBytes = kInputs * kInputBytes;
};

// A tile: its number (-1: none), its channels, its sequence n, its place i in the walk over that
// sequence (kMixed: n is 0 and i the place among all tiles), i's place j in its group and the group's
// number, its lowest row, and the rows from the tile's first to the walk's last (kMixed: -1).  Walked
// from the end, the last tile may begin before the sequence.
// Numbers count in walking order, sequence after sequence; by chains the chain's; kMixed along the rows.
struct __align__(16) Tile {
  int t, column, n, i, j, g, row, left;
};

template <typename E>
struct Params {
  const E* in[kMaxInputs];
  int64_t ld_in[kMaxInputs];
  E* out[3];  // o; dx, dr, dg
  int64_t ld_out[3];
  const float* slopes;
  const float* start;  // [P, C] states the walk begins with (h0; dh_final) or null
  const float* h0;     // backward: [P, C] or null
  float* finish;       // [P, C] states it ends with (h_final; dh0) or null
  float* part;         // backward: [tiles or chains, C] sums of each one's terms of dslopes
  const int32_t* state_indices;
  const int32_t* cu_seqlens;
  const int32_t* accepted_len;  // commit
  int* dev_error;
  // the workspace of a scan
  int* ticket;         // kTicket words: next tile or chain, an abort flag, how many (packed); null: blocks
                       // take theirs in turn.  Packed batches have the tiles' words behind the chains'
  int2* places;        // [tiles + 1] (packed, kMixed) where each tile lies among the sequences
  int32_t* order;      // [N] (packed, by chains) the running sequences of at most `longest` tokens, longest first
  Tile* table;         // [tiles] (packed, by tiles) the others' tiles in the order in which they are taken
  float4* runs;        // [tiles][columns][32] published (A, H) of each lane's two channels; null: nothing waits
  float2* before;      // [groups of all sequences][columns][32] published states after each group
  int T, N, C, pool_size, rows;
  int tiles, columns, stride;  // tiles along the rows, of `stride` rows; along the channels
  int group, groups, spans;    // tiles per group; groups of a sequence of one length, of all sequences
  int longest;
  // Sequences of one length: tiles per sequence (the last may be short); 0: packed, or tiles that
  // hold several whole sequences.
  int per;
};

constexpr int kTicket = 4;
constexpr int kMostListed = 4096;  // sequences of a batch that the plan kernel orders by comparing all

struct Maps {
  CUtensorMap of[kMaxInputs];
};

__device__ __forceinline__ void report(int* dev_error, unsigned bit) {
  if (dev_error) atomicOr(reinterpret_cast<unsigned*>(dev_error), bit);
}

// ---------------------------------------------------------------- before a scan

// Fills the published words, sets the ticket and, for a packed batch, checks cu_seqlens
// (non-decreasing inside [0, T]; if not, the ticket starts past the last tile, so that the scan
// does nothing).  kMixed: it finds each tile's place: x, the first sequence that begins at or
// after its first row; y, whether all its rows lie inside one running sequence, away from its ends.
// By chains, it orders the running sequences, longest first (ties by number); by tiles, it lists the
// running sequences' tiles: the first of each, longest sequence first, then the second of each, ...
// A warp compares a sequence or a tile with all sequences (a thread for each took 118 us for 4000
// sequences, and a fifth of such a call more).
template <typename E>
__global__ void __launch_bounds__(kThreads) scan_plan_kernel(const Params<E> p) {
  __shared__ unsigned long long sums[2];  // tiles and groups of the table
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const size_t id = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
  const size_t all = static_cast<size_t>(gridDim.x) * kThreads;
  auto length = [&](int n) {  // -1: does not run
    const int slot = p.state_indices ? p.state_indices[n] : n;
    return slot < 0 || slot >= p.pool_size ? -1 : min(max(p.cu_seqlens[n + 1] - p.cu_seqlens[n], 0), p.T);
  };
  auto tiles_of = [&](int n) {  // in the table
    const int l = length(n);
    return l <= p.longest ? 0 : l <= p.stride ? 1 : (l + p.stride - 1) / p.stride;
  };
  int tiles = p.tiles, spans = p.spans;
  if (p.table) {
    if (threadIdx.x < 2) sums[threadIdx.x] = 0ull;
    __syncthreads();
    unsigned long long mine = 0ull, groups = 0ull;
    for (int n = threadIdx.x; n < p.N; n += kThreads) {
      const int t = tiles_of(n);
      mine += t;
      groups += (t + p.group - 1) / p.group;
    }
    if (mine) {
      atomicAdd(&sums[0], mine);
      atomicAdd(&sums[1], groups);
    }
    __syncthreads();
    tiles = static_cast<int>(min(sums[0], static_cast<unsigned long long>(tiles)));  // as they are unless
    spans = static_cast<int>(min(sums[1], static_cast<unsigned long long>(spans)));  // cu_seqlens is refused
  }
  auto fill = [&](void* at, size_t chunks) {
    for (size_t i = id; i < chunks; i += all) reinterpret_cast<uint4*>(at)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  };
  if (p.runs) {
    fill(p.runs, static_cast<size_t>(tiles) * p.columns * 32);
    fill(p.before, static_cast<size_t>(spans) * p.columns * 16);
  }
  if (p.places) {
    for (size_t i = id; i <= static_cast<size_t>(p.tiles); i += all) {
      const int64_t row = static_cast<int64_t>(i) * p.stride;
      int a = 0, b = p.N;  // the first n with cu[n] >= row
      while (a < b) {
        const int m = (a + b) / 2;
        if (p.cu_seqlens[m] >= row) b = m; else a = m + 1;
      }
      bool inner = a > 0 && row + p.stride < p.cu_seqlens[a];
      if (inner) {
        const int slot = p.state_indices ? p.state_indices[a - 1] : a - 1;
        inner = slot >= 0 && slot < p.pool_size;
      }
      p.places[i] = make_int2(i == static_cast<size_t>(p.tiles) ? p.N : a, inner);  // the last tile owns the rest
    }
  }
  if (p.cu_seqlens && p.state_indices && !p.places)
    for (size_t i = id; i < static_cast<size_t>(p.N); i += all)
      if (p.state_indices[i] >= p.pool_size) report(p.dev_error, kErrBadIndex);
  // a warp for each sequence and for each tile
  const int lane = threadIdx.x % 32, warp = static_cast<int>(id / 32), warps = static_cast<int>(all / 32);
  constexpr unsigned kAll = 0xFFFFFFFFu;
  if (p.order) {
    auto chain = [&](int n) {  // -1: none
      const int l = length(n);
      return l > p.longest ? -1 : l;
    };
    for (int n = warp; n < p.N; n += warps) {
      const int mine = chain(n);
      int rank = 0, chains = 0;
#pragma unroll 4
      for (int m = lane; m < p.N; m += 32) {
        const int other = chain(m);
        chains += other >= 0;
        rank += other > mine || (other == mine && m < n);
      }
      rank = __reduce_add_sync(kAll, rank);
      chains = __reduce_add_sync(kAll, chains);
      if (lane == 0 && mine >= 0) p.order[rank] = n;
      if (lane == 0 && n == 0) p.ticket[2] = chains;
    }
  }
  if (p.table) {
    for (int t = warp; t < tiles; t += warps) {
      int n = -1, i = t, g = 0;  // t's sequence, its place there, the sequence's first group
      for (int m0 = 0; m0 < p.N && n < 0; m0 += 32) {
        const int here = m0 + lane < p.N ? tiles_of(m0 + lane) : 0;
        int upto = here;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int v = __shfl_up_sync(kAll, upto, d);
          if (lane >= d) upto += v;
        }
        const unsigned found = __ballot_sync(kAll, i < upto);
        const int src = found ? __ffs(found) - 1 : 32;
        g += __reduce_add_sync(kAll, lane < src ? (here + p.group - 1) / p.group : 0);
        i -= __shfl_sync(kAll, found ? upto - here : upto, found ? src : 31);
        if (found) n = m0 + src;
      }
      if (n < 0) continue;
      const int mine = tiles_of(n);
      int at = 0;
      for (int m = lane; m < p.N; m += 32) {
        const int other = tiles_of(m);
        at += min(other, i) + (other > i && (other > mine || (other == mine && m < n)));
      }
      at = __reduce_add_sync(kAll, at);
      const int lo = p.cu_seqlens[n], hi = p.cu_seqlens[n + 1];
      if (lane == 0 && static_cast<unsigned>(at) < static_cast<unsigned>(tiles))  // always, unless cu_seqlens is refused
        p.table[at] = {t, 0, n, i, i % p.group, g + i / p.group,
                       p.part ? hi - (i + 1) * p.stride : lo + i * p.stride, hi - lo - i * p.stride};
    }
  }
  if (blockIdx.x == 0) {
    int wrong = 0;
    if (p.cu_seqlens)
      for (int n = threadIdx.x; n < p.N; n += kThreads)
        wrong |= p.cu_seqlens[n] < 0 || p.cu_seqlens[n] > p.cu_seqlens[n + 1] || p.cu_seqlens[n + 1] > p.T;
    wrong = __syncthreads_or(wrong);
    if (threadIdx.x == 0) {
      p.ticket[0] = p.ticket[kTicket] = wrong ? 1 << 30 : 0;
      p.ticket[1] = p.ticket[kTicket + 1] = 0;
      if (!p.order) p.ticket[2] = 0;
      p.ticket[kTicket + 2] = p.table ? tiles : 0;
      if (wrong) report(p.dev_error, kErrBadSeqlens);
    }
  }
}

// ---------------------------------------------------------------- a warp's rows

// What a warp knows of its rows: bit k of each mask is row k in walking order; lane k holds row
// k's slot.
struct Rows {
  unsigned live, begin, end;  // of a sequence that runs; where the walk enters and leaves one
  int slot;
};

// Sequence n's slot, or -1 where it is padded or its index is out of range.
template <typename E>
__device__ __forceinline__ int checked(const Params<E>& p, int slot) {
  if (slot >= p.pool_size) {
    report(p.dev_error, kErrBadIndex);
    return -1;
  }
  return slot;
}
template <typename E>
__device__ __forceinline__ int slot_of(const Params<E>& p, int n) {
  return checked(p, p.state_indices ? p.state_indices[n] : n);
}

template <Mode kMode, bool kBack, int K, typename E>
__device__ __forceinline__ Rows rows_of(const Params<E>& p, const Tile& q, int warp, int lane) {
  if constexpr (kMode != kMixed) {  // by arithmetic, the same for every lane
    const int slot = p.state_indices ? p.state_indices[q.n] : q.n;
    auto bit = [](int k) { return k >= 0 && k < K ? 1u << k : 0u; };
    auto below = [](int k) { return k <= 0 ? 0u : k >= K ? (1u << K) - 1u : (1u << k) - 1u; };  // bits under k
    Rows r{0u, 0u, 0u, checked(p, slot)};
    if (r.slot < 0) return r;
    // tiles begin where the walk does, so no row begins the sequence: its state comes from outside
    const int left = q.left - warp * K;
    r.live = below(left);
    r.end = bit(left - 1);
    return r;
  } else {
    Rows r{0u, 0u, 0u, -1};
    const int place = warp * K + lane;  // in walking order
    const int at = kBack ? p.stride - 1 - place : place;
    const int64_t row = static_cast<int64_t>(q.t) * p.stride + at;
    bool first = false, last = false;
    if (lane < K && place < p.stride && row < p.rows) {
      if (p.cu_seqlens) {
        int a = p.places[q.t].x, b = p.places[q.t + 1].x;
        while (a < b) {  // the number of sequences that begin at or before the row
          const int m = (a + b) / 2;
          if (p.cu_seqlens[m] <= row) a = m + 1; else b = m;
        }
        if (a > 0) {
          const int lo = p.cu_seqlens[a - 1], hi = p.cu_seqlens[a];
          if (row < hi) {
            r.slot = slot_of(p, a - 1);
            first = row == lo;
            last = row == hi - 1;
          }
        }
      } else {
        const int n = static_cast<int>(row) / p.T, t = static_cast<int>(row) - n * p.T;
        r.slot = slot_of(p, n);
        first = t == 0;
        last = t == p.T - 1;
      }
    }
    r.live = __ballot_sync(0xFFFFFFFFu, r.slot >= 0);
    r.begin = __ballot_sync(0xFFFFFFFFu, r.slot >= 0 && (kBack ? last : first));
    r.end = __ballot_sync(0xFFFFFFFFu, r.slot >= 0 && (kBack ? first : last));
    return r;
  }
}

// Whether some row of the warp may end a sequence or belong to none (kMixed: or begin one).
// `inside`: what was looked up for the tile (its sequence's slot; kMixed: whether the tile lies
// inside a sequence).
template <Mode kMode, int K, typename E>
__device__ __forceinline__ bool has_edges(const Params<E>& p, const Tile& q, int inside, int warp) {
  if constexpr (kMode == kMixed) return !inside;
  return inside < 0 || inside >= p.pool_size || q.left <= (warp + 1) * K;
}

// A lane's two channels: neighbours with TMA rows, else a warp's width apart.
template <bool kTma>
struct Lane {
  int c[2];
  bool ok[2];
  __device__ __forceinline__ Lane(int column, int lane, int C) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = column * kCols + (kTma ? 2 * lane + j : lane + 32 * j);
      ok[j] = c[j] < C;
    }
  }
};

// Output rows from the lane's first channel on: its two channels (a TMA kernel's rows hold an even
// number of channels).
template <bool kTma>
__device__ __forceinline__ void store2(float* at, const Lane<kTma>& l, f2 v) {
  const float2 t = f2_unpack(v);
  if constexpr (kTma) {
    if (l.ok[0]) __stcs(reinterpret_cast<float2*>(at), t);
  } else {
    if (l.ok[0]) __stcs(at, t.x);
    if (l.ok[1]) __stcs(at + 32, t.y);
  }
}
template <bool kTma>
__device__ __forceinline__ void store2(__nv_bfloat16* at, const Lane<kTma>& l, f2 v) {
  const float2 t = f2_unpack(v);
  const __nv_bfloat162 b = __floats2bfloat162_rn(t.x, t.y);
  const unsigned w = *reinterpret_cast<const unsigned*>(&b);
  unsigned short* s = reinterpret_cast<unsigned short*>(at);
  if constexpr (kTma) {
    if (l.ok[0]) __stcs(reinterpret_cast<unsigned*>(s), w);
  } else {
    if (l.ok[0]) __stcs(s, static_cast<unsigned short>(w));
    if (l.ok[1]) __stcs(s + 32, static_cast<unsigned short>(w >> 16));
  }
}

// A state [P, C] of one slot, the lane's channels; 0 without a pool.
template <bool kTma>
__device__ __forceinline__ f2 load_state(const float* pool, int slot, int C, const Lane<kTma>& l) {
  float2 v = make_float2(0.f, 0.f);
  if (pool) {
    const float* s = pool + static_cast<size_t>(slot) * C;
    if (l.ok[0]) v.x = s[l.c[0]];
    if (l.ok[1]) v.y = s[l.c[1]];
  }
  return f2_of(v);
}
template <bool kTma>
__device__ __forceinline__ void store_state(float* pool, int slot, int C, const Lane<kTma>& l, f2 v) {
  const float2 t = f2_unpack(v);
  float* s = pool + static_cast<size_t>(slot) * C;
  if (l.ok[0]) s[l.c[0]] = t.x;
  if (l.ok[1]) s[l.c[1]] = t.y;
}

// ---------------------------------------------------------------- a warp's rows in shared memory

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Starts the loads of a tile's rows of every input into `stage`, whose first row is row `low` of
// the matrices: each warp its own rows, from row `first` of the stage (kTma: one thread of it, a box
// for each input).
template <Mode kMode, bool kBack, bool kTma, typename E>
__device__ __forceinline__ void fetch(const Params<E>& p, const Maps& maps, char* stage, uint64_t* bar, int low,
                                      int column, int first, int lane) {
  using S = Shape<E, kBack, kTma, kMode>;
  if constexpr (kTma) {
    lap::mbar_arrive_expect_tx(bar, S::kInputs * S::kRows * S::kPitch);
#pragma unroll
    for (int i = 0; i < S::kInputs; ++i)  // o one row up; rows outside the matrix arrive as zeros
      lap::tma_load_2d(stage + i * S::kInputBytes + first * S::kPitch, &maps.of[i], bar, column * kCols,
                       low + first - (i == 4));
  } else {
    constexpr int kChunks = S::kPitch / 16, kAtOnce = 32 / kChunks;  // of a row; rows
    const int k0 = lane / kChunks, c = lane - k0 * kChunks;
    const int64_t last = static_cast<int64_t>(p.rows) - 1;
    const int bytes = min(kCols, p.C - column * kCols) * static_cast<int>(sizeof(E));
    const bool on = k0 < kAtOnce && 16 * c < bytes + 15;
#pragma unroll
    for (int i = 0; i < S::kInputs; ++i) {
      const char* begin = reinterpret_cast<const char*>(p.in[i]);  // of the matrix
      const int64_t pitch = p.ld_in[i] * static_cast<int64_t>(sizeof(E)), top = static_cast<int64_t>(low) + first - (i == 4);
      const char* src = begin + (top + k0) * pitch + column * kCols * static_cast<int>(sizeof(E));
      char* dst = stage + i * S::kInputBytes + (first + k0) * S::kPitch + 16 * c;
      if (top * pitch >= 16 && (last - top - (S::kRows - 1)) * pitch >= 32) {
        // what the chunks hold beside the channels lies inside the matrix
#pragma unroll
        for (int k = 0; k < S::kRows; k += kAtOnce) {
          if (on && k + k0 < S::kRows)
            copy16(lap::smem_u32(dst) + k * S::kPitch, src - (reinterpret_cast<uintptr_t>(src) & 15u) + 16 * c);
          src += kAtOnce * pitch;
        }
      } else {
        const char* end = begin + last * pitch + static_cast<int64_t>(p.C) * sizeof(E);
#pragma unroll 1
        for (int k = 0; k < S::kRows; k += kAtOnce, src += kAtOnce * pitch) {
          if (!on || k + k0 >= S::kRows || top + k + k0 < 0 || top + k + k0 > last) continue;
          const char* chunk = src - (reinterpret_cast<uintptr_t>(src) & 15u) + 16 * c;
          if (chunk >= begin && chunk + 16 <= end) {
            copy16(lap::smem_u32(dst) + k * S::kPitch, chunk);
          } else {
            for (int e = 0; e < 16; e += sizeof(E))
              if (chunk + e >= src && chunk + e < src + bytes)
                *reinterpret_cast<E*>(dst + k * S::kPitch + e) = *reinterpret_cast<const E*>(chunk + e);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
}

// Waits for a stage (the `use`-th time it is filled); false after a second.
template <bool kTma>
__device__ __forceinline__ bool arrived(uint64_t* bar, unsigned use, volatile int* abort) {
  if constexpr (kTma) {
    return lap::mbar_wait(bar, use & 1u, abort);
  } else {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");  // all but the next stage's
    __syncwarp();
    return true;
  }
}

// A lane's view of one input's rows in a stage.
template <typename E, bool kBack, bool kTma, Mode kMode>
struct View {
  using S = Shape<E, kBack, kTma, kMode>;
  const char* at;
  unsigned first, step;  // bytes before the first row's first channel in its chunk; more per row
  // `rows`: the warp's first row in the stage, row `low` of the matrix
  __device__ __forceinline__ View(const Params<E>& p, const char* rows, int i, int low, int lane) {
    at = rows + i * S::kInputBytes + lane * sizeof(E) * (kTma ? 2 : 1);
    if constexpr (!kTma) {
      step = static_cast<unsigned>(p.ld_in[i]) * sizeof(E);
      first = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p.in[i])) + static_cast<unsigned>(low - (i == 4)) * step;
    }
  }
  __device__ __forceinline__ f2 get(int k) const {
    const char* s = at + k * S::kPitch;
    if constexpr (kTma) {
      if constexpr (sizeof(E) == 4) return *reinterpret_cast<const f2*>(s);
      else return lap::bf16x2_to_f2(*reinterpret_cast<const uint32_t*>(s));
    } else {
      s += (first + k * step) & 15u;
      if constexpr (sizeof(E) == 4) {
        return f2_pack(*reinterpret_cast<const float*>(s), *reinterpret_cast<const float*>(s + 128));
      } else {
        const unsigned lo = *reinterpret_cast<const unsigned short*>(s);
        const unsigned hi = *reinterpret_cast<const unsigned short*>(s + 64);
        return f2_pack(__uint_as_float(lo << 16), __uint_as_float(hi << 16));
      }
    }
  }
  // min(get(k), kOpen); two BF16 channels in one instruction.
  __device__ __forceinline__ f2 gate(int k) const {
    if constexpr (kTma && sizeof(E) == 2)
      return lap::bf16x2_to_f2(at_most_open_bf16x2(*reinterpret_cast<const uint32_t*>(at + k * S::kPitch)));
    else
      return at_most_open2(get(k));
  }
};

// ---------------------------------------------------------------- composition and publication

// A run of rows of the lane's two channels: h -> a h + h0 per channel; a = -0 marks a beginning.
struct __align__(16) Run {
  f2 a, h;
};

__device__ __forceinline__ f2 apply(const Run& r, f2 before) {
  const float2 a = f2_unpack(r.a), h = f2_unpack(r.h), v = f2_unpack(f2_fma(r.a, before, r.h));
  return f2_pack(signbit(a.x) ? h.x : v.x, signbit(a.y) ? h.y : v.y);
}
// `first`, then `then`.
__device__ __forceinline__ Run compose(const Run& first, const Run& then) {
  const float2 a = f2_unpack(then.a), v = f2_unpack(f2_mul(first.a, then.a));
  return {f2_pack(signbit(a.x) ? -0.f : v.x, signbit(a.y) ? -0.f : v.y), apply(then, first.h)};
}

constexpr unsigned kUnset = ~0u;

__device__ __forceinline__ unsigned ready_bits(float v) {
  const unsigned u = __float_as_uint(v);
  return u == kUnset ? 0x7FFFFFFFu : u;  // a NaN that looks unset becomes another NaN
}
__device__ __forceinline__ void publish_run(float4* at, const Run& r) {
  const float2 a = f2_unpack(r.a), h = f2_unpack(r.h);
  asm volatile("st.relaxed.gpu.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(at), "r"(ready_bits(a.x)),
               "r"(ready_bits(a.y)), "r"(ready_bits(h.x)), "r"(ready_bits(h.y))
               : "memory");
}
__device__ __forceinline__ void publish_state(float2* at, f2 state) {
  const float2 h = f2_unpack(state);
  asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(at), "r"(ready_bits(h.x)), "r"(ready_bits(h.y))
               : "memory");
}
__device__ __forceinline__ bool is_set(f2 v) {
  return static_cast<unsigned>(v) != kUnset && static_cast<unsigned>(v >> 32) != kUnset;
}
__device__ __forceinline__ bool is_set(const Run& r) { return is_set(r.a) && is_set(r.h); }

// Whether a poll may go on: false once a second has passed since `t0` or another block gave up.
__device__ __noinline__ bool keep_polling(int* ticket, int* dev_error, uint64_t t0) {
  int stop;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(stop) : "l"(ticket + 1));
  if (stop) return false;
  if (lap::globaltimer_ns() - t0 <= lap::kWaitLimitNs) return true;
  atomicExch(ticket + 1, 1);
  report(dev_error, kErrTimeout);
  return false;
}

__device__ __forceinline__ Run read_run(const float4* at) {
  float2 a, h;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(a.x), "=f"(a.y), "=f"(h.x), "=f"(h.y)
               : "l"(at)
               : "memory");
  return {f2_of(a), f2_of(h)};
}
__device__ __forceinline__ Run await_run(const float4* at, int* ticket, int* dev_error) {
  Run r;
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    r = read_run(at);
    if (is_set(r)) break;
    if (i == 0) t0 = lap::globaltimer_ns();
    if ((i & 3u) == 3u && !keep_polling(ticket, dev_error, t0)) break;
  }
  return r;
}

__device__ __forceinline__ f2 await_state(const float2* at, int* ticket, int* dev_error) {
  unsigned u, v;
  f2 h;
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(u), "=r"(v) : "l"(at) : "memory");
    h = f2_pack(__uint_as_float(u), __uint_as_float(v));
    if (is_set(h)) break;
    if (i == 0) t0 = lap::globaltimer_ns();
    if ((i & 3u) == 3u && !keep_polling(ticket, dev_error, t0)) break;
  }
  return h;
}

// What a tile shares between its warps; two of them in turn, so that a warp may begin the next
// tile while another still reads this one's.
template <Mode kMode, int kWarps>
struct Exchange {
  Run own[kWarps][32];      // each warp's rows
  Run earlier[kMode == kByChains ? 1 : kWarps][32];  // the group's earlier tiles, or pieces of them, in order
  f2 base[32];              // the state before the group (by chains: before the tile); the last warp's
  unsigned char late[8];    // per warp: a word it asked for had not been published in time
  unsigned char begins[8];  // per warp: some of its rows begin a sequence
  int fresh;                // the tile's first row does: what lies before the tile does not matter
};
template <Mode kMode, int kWarps>
struct ScanSmem {
  Exchange<kMode, kWarps> turn[2];
  Tile tile[4];             // of this turn, the next two and the last
  uint64_t bar[kWarps][kStages];
  int abort;                // a load did not arrive
};

template <typename E, bool kBack, bool kTma, Mode kMode>
__host__ __device__ constexpr int scan_smem_bytes() {
  using S = Shape<E, kBack, kTma, kMode>;
  return kStages * S::kStageBytes + static_cast<int>(sizeof(ScanSmem<kMode, S::kWarps>));
}

// The published words a tile needs: where it has more than kWarps earlier tiles in its group, each
// warp composes a piece [lo, hi) of them.
template <Mode kMode, int kWarps>
struct Needs {
  int j, per, lo, hi;
  template <typename E>
  __device__ __forceinline__ Needs(const Params<E>& p, const Tile& q, int warp) {
    j = q.j;
    per = (j + kWarps - 1) / kWarps;
    lo = min(j, warp * per);
    hi = min(j, lo + per);
  }
  // The run of the group's i-th tile.
  template <typename E>
  __device__ __forceinline__ float4* run(const Params<E>& p, const Tile& q, int i, int lane) const {
    return p.runs + (static_cast<size_t>((kMode == kMixed ? q.i : q.t) - j + i) * p.columns + q.column) * 32 + lane;
  }
  // The state after this tile's group, or after the one `back` before it.
  template <typename E>
  __device__ __forceinline__ float2* state(const Params<E>& p, const Tile& q, int back, int lane) const {
    return p.before + (static_cast<size_t>(q.g - back) * p.columns + q.column) * 32 + lane;
  }

  // Asks for the words, where each warp needs one tile's (the last warp: the base too) ...
  template <typename E, typename X>
  __device__ __forceinline__ void ask(const Params<E>& p, X& ex, const Tile& q, int warp, int lane) const {
    if (per <= 1) {
      if (lo < hi) copy16(lap::smem_u32(&ex.earlier[warp][lane]), run(p, q, lo, lane));
      if (warp == kWarps - 1 && q.i > j && lane % 2 == 0)  // for two lanes: past the L1, which is not coherent
        copy16(lap::smem_u32(&ex.base[lane]), state(p, q, 1, lane));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // ... and notes what has not come.  (Without TMA the next tile's rows, asked for before the words, are
  // waited for too.)
  template <typename X>
  __device__ __forceinline__ void look(X& ex, const Tile& q, int warp, int lane) const {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    unsigned late = per > 1;
    if (per <= 1) {
      const bool run_ok = lo >= hi || is_set(ex.earlier[warp][lane]);
      const bool base_ok = warp != kWarps - 1 || q.i == j || is_set(ex.base[lane]);
      late = !__all_sync(0xFFFFFFFFu, run_ok && base_ok);
    }
    if (lane == 0) ex.late[warp] = static_cast<unsigned char>(late);
  }
  // The warp's piece and (the last warp) the base, by polling, up to four words at once.
  template <typename E, typename X>
  __device__ __forceinline__ void poll(const Params<E>& p, X& ex, const Tile& q, int warp, int lane) const {
    if (lo < hi) {
      Run r = await_run(run(p, q, lo, lane), p.ticket, p.dev_error);
#pragma unroll 1
      for (int i = lo + 1; i < hi; i += 4) {
        Run w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = read_run(run(p, q, min(i + k, hi - 1), lane));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (i + k >= hi) break;
          if (!is_set(w[k])) w[k] = await_run(run(p, q, i + k, lane), p.ticket, p.dev_error);
          r = compose(r, w[k]);
        }
      }
      ex.earlier[warp][lane] = r;
    }
    if (warp == kWarps - 1 && q.i > j) ex.base[lane] = await_state(state(p, q, 1, lane), p.ticket, p.dev_error);
  }
};

// The state before this warp's rows.  `mine` (in ex.own already) is the composition of the warp's
// rows.  Where tiles wait for one another, publishes the tile for those that follow; by chains (where
// `start` is the state before the chain), leaves the state after it in `next`, the exchange of the
// block's next tile.
template <Mode kMode, typename E, int kWarps>
__device__ __forceinline__ f2 state_before(const Params<E>& p, Exchange<kMode, kWarps>& ex,
                                           Exchange<kMode, kWarps>& next, const Tile& q, const Run& mine, f2 start,
                                           int warp, int lane) {
  if constexpr (kMode == kByChains) {
    f2 before = q.i == 0 ? start : ex.base[lane];
#pragma unroll 4
    for (int w = 0; w < warp; ++w) before = f2_fma(ex.own[w][lane].a, before, ex.own[w][lane].h);
    if (warp == kWarps - 1) next.base[lane] = f2_fma(mine.a, before, mine.h);
    return before;
  } else {
    f2 before = f2_all(0.f);
    const bool fresh = kMode == kMixed && __any_sync(0xFFFFFFFFu, ex.fresh);
    if (kMode == kByTiles || p.runs) {
      const Needs<kMode, kWarps> needs(p, q, warp);
      const bool last = needs.j == p.group - 1;
      Run whole;
      if (warp == 0) {
        whole = mine;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) whole = compose(whole, ex.own[w][lane]);
        if (!last) publish_run(needs.run(p, q, needs.j, lane), whole);
      }
      if (!fresh) {
        if (*reinterpret_cast<const unsigned long long*>(ex.late) != 0ull) {
          if (ex.late[warp]) needs.poll(p, ex, q, warp, lane);
          __syncthreads();
        }
        before = ex.base[lane];
        const int pieces = needs.per <= 1 ? needs.j : (needs.j + needs.per - 1) / needs.per;
#pragma unroll 2
        for (int i = 0; i < pieces; ++i) before = apply(ex.earlier[i][lane], before);
      }
      if (warp == 0 && last) publish_state(needs.state(p, q, 0, lane), apply(whole, before));
    }
    if (kMode == kMixed && __any_sync(0xFFFFFFFFu, *reinterpret_cast<const unsigned long long*>(ex.begins) != 0ull)) {
#pragma unroll 1
      for (int w = 0; w < warp; ++w) before = apply(ex.own[w][lane], before);
    } else {
#pragma unroll 4
      for (int w = 0; w < warp; ++w) before = f2_fma(ex.own[w][lane].a, before, ex.own[w][lane].h);
    }
    return before;
  }
}

// The final states of the empty sequences that lie in this tile, or the tile's own: their initial
// ones.
template <Mode kMode, int kWarps, typename E, bool kTma>
__device__ __forceinline__ void empty_sequences(const Params<E>& p, const Tile& q, const Lane<kTma>& l, int warp) {
  if (!p.finish || q.left > 0 || (!p.cu_seqlens && p.T > 0)) return;
  const int lo = kMode != kMixed ? q.n : p.cu_seqlens ? p.places[q.t].x : 0;
  const int hi = kMode != kMixed ? q.n + 1 : p.cu_seqlens ? p.places[q.t + 1].x : p.N;
  for (int n = lo + warp; n < hi; n += kWarps) {
    if (p.cu_seqlens && p.cu_seqlens[n] != p.cu_seqlens[n + 1]) continue;
    const int slot = slot_of(p, n);
    if (slot >= 0) store_state(p.finish, slot, p.C, l, load_state(p.start, slot, p.C, l));
  }
}

// ---------------------------------------------------------------- the forward scan

// a = lambda and b = beta sig(g) x of one token.  With w = beta^2 and p = exp(g), b is
// w x p / sqrt(w (1 + p)^2): one rsqrt stands for beta's root and the gate's reciprocal (the special
// function unit is what bounds the scan after memory; with a reciprocal for the gate 2 x 8192 tokens of
// 8192 channels take 212 us, with this 195).  g comes as min(g, kOpen), where sig is 1 in FP32, so that
// nothing overflows; p keeps its digits down to exp(-87).  NaN passes: a maximum would drop it, but only
// w is kept from 0 in the root, and w's own NaN is in the product.
template <bool kSmall>
__device__ __forceinline__ void step2(f2 slope, f2 x, f2 r, f2 g, f2* a, f2* b) {
  const Decay d = decay2<kSmall>(f2_mul(slope, sigmoid2(r)));
  const f2 w = one_minus_square2(d), p = exp_of2(g), q = f2_add(p, f2_all(1.f));
  *a = d.lambda;
  *b = f2_mul(f2_mul(f2_mul(w, x), p), rsqrt2(f2_mul(positive2(w), f2_mul(q, q))));
}

template <typename E, bool kTma, Mode kMode>
struct Forward {
  using S = Shape<E, false, kTma, kMode>;
  static constexpr int K = S::kRows;
  f2 a[K], b[K];

  // The warp's rows composed.  kEdges: some row begins or ends a sequence or belongs to none.
  // `ask` runs when most rows are done.
  template <bool kEdges, bool kSmall, typename F>
  __device__ __forceinline__ Run first(const Params<E>& p, const char* stage, int low, f2 slope, const Rows& rows,
                                       const Lane<kTma>& l, int lane, F ask) {
    const View<E, false, kTma, kMode> x(p, stage, 0, low, lane), r(p, stage, 1, low, lane), g(p, stage, 2, low, lane);
    if constexpr (kEdges) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        b[k] = f2_all(0.f);
        if (rows.begin >> k & 1u) b[k] = load_state(p.start, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l);
      }
    }
    Run run{f2_all(1.f), f2_all(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k == S::kAsk) ask();
      f2 in;
      step2<kSmall>(slope, x.get(k), r.get(k), g.gate(k), &a[k], &in);
      if constexpr (kEdges) {
        b[k] = f2_fma(a[k], b[k], in);
        if (rows.begin >> k & 1u) run = {f2_all(-0.f), f2_all(0.f)};
      } else {
        b[k] = in;
      }
      run.h = f2_fma(a[k], run.h, b[k]);
      run.a = f2_mul(run.a, a[k]);
    }
    return run;
  }

  template <bool kEdges>
  __device__ __forceinline__ void second(const Params<E>& p, int low, f2 h, const Rows& rows, const Lane<kTma>& l) {
    E* o = p.out[0] + static_cast<int64_t>(low) * p.ld_out[0] + l.c[0];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (kEdges) {
        if (rows.begin >> k & 1u) h = f2_all(0.f);
      }
      h = f2_fma(a[k], h, b[k]);
      if (!kEdges || (rows.live >> k & 1u)) store2(o, l, h);
      o += p.ld_out[0];
      if constexpr (kEdges) {
        if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l, h);
      }
    }
  }
};

// ---------------------------------------------------------------- the gradients' scan

template <typename E, bool kTma, Mode kMode>
struct Backward {
  using S = Shape<E, true, kTma, kMode>;
  static constexpr int K = S::kRows;
  f2 er[K], kept[K];  // exp(-r) and the decay, folded; row k in walking order is row K - 1 - k of the stage

  template <bool kEdges, bool kSmall, typename F>
  __device__ __forceinline__ Run first(const Params<E>& p, const char* stage, int low, f2 slope, const Rows& rows,
                                       const Lane<kTma>& l, int lane, F ask) {
    const View<E, true, kTma, kMode> r(p, stage, 1, low, lane), d(p, stage, 3, low, lane);
    Run run{f2_all(1.f), f2_all(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k == S::kAsk) ask();
      er[k] = exp_minus2(r.get(K - 1 - k));
      const f2 u = f2_mul(slope, sigmoid_of2(er[k]));
      const Decay decay = decay2<kSmall>(u);
      const f2 a = decay.lambda;
      kept[k] = fold2<kSmall>(u, decay);
      if constexpr (kEdges) {
        if (rows.begin >> k & 1u)
          run = {f2_all(-0.f), load_state(p.start, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l)};
      }
      run.h = f2_mul(a, f2_add(d.get(K - 1 - k), run.h));
      run.a = f2_mul(run.a, a);
    }
    return run;
  }

  // Writes dx, dr, dg; returns the rows' terms of dslopes.  w = lambda_{t+1} G_{t+1} on entry.
  template <bool kEdges>
  __device__ __forceinline__ f2 second(const Params<E>& p, const char* stage, int low, f2 slope, f2 w, const Rows& rows,
                                       const Lane<kTma>& l, int lane) {
    const View<E, true, kTma, kMode> x(p, stage, 0, low, lane), g(p, stage, 2, low, lane), d(p, stage, 3, low, lane),
        h(p, stage, 4, low, lane);
    E* out[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) out[i] = p.out[i] + static_cast<int64_t>(low + K) * p.ld_out[i] + l.c[0];
    f2 sum = f2_all(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = K - 1 - k;
      f2 before = h.get(at);
#pragma unroll
      for (int i = 0; i < 3; ++i) out[i] -= p.ld_out[i];
      if constexpr (kEdges) {
        if (!(rows.live >> k & 1u)) continue;
        const int slot = __shfl_sync(0xFFFFFFFFu, rows.slot, k);
        if (rows.begin >> k & 1u) w = load_state(p.start, slot, p.C, l);
        if (rows.end >> k & 1u) before = load_state(p.h0, slot, p.C, l);
      }
      const f2 G = f2_add(d.get(at), w), vx = x.get(at);
      const Gate in = gate_of2(exp_minus2(g.get(at))), out_of = gate_of2(er[k]);
      const Decay decay = unfold2(kept[k]);
      const f2 lambda = decay.lambda, beta2 = one_minus_square2(decay);
      // 1 / beta, and beta, are 0 where u = 0 (or beta^2 is under the smallest normal number)
      const float2 vb = f2_unpack(beta2), vi = f2_unpack(rsqrt2(beta2));
      const f2 inv = f2_pack(vb.x >= kLeast ? vi.x : 0.f, vb.y >= kLeast ? vi.y : 0.f), beta = f2_mul(beta2, inv);
      const f2 gs = f2_mul(G, in.open), dx = f2_mul(gs, beta);
      store2(out[0], l, dx);
      store2(out[2], l, f2_mul(f2_mul(dx, vx), in.rest));
      // du = lambda (gs x lambda / beta - G h_{t-1}); ds = du sig(r); with u = slope sig(r), dr = ds slope (1 - sig(r))
      const f2 t = f2_mul(f2_mul(gs, vx), f2_mul(lambda, inv));
      const f2 ds = f2_mul(f2_mul(lambda, f2_sub(t, f2_mul(G, before))), out_of.open);
      store2(out[1], l, f2_mul(ds, f2_mul(slope, out_of.rest)));
      sum = f2_add(sum, ds);
      w = f2_mul(lambda, G);
      if constexpr (kEdges) {
        if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l, w);
      }
    }
    return sum;
  }
};

// ---------------------------------------------------------------- the scan kernel

// Blocks are persistent and take tiles one after another.
// By tiles (long scans over few channels), and packed batches of short sequences: by tickets in
// walking order, all channels of a place before the next, the sequences of a fixed-length batch
// (or of a packed batch's table) side by side; the states pass from block to block.
// By chains: all tiles of a sequence's channels in order, the state passing in shared memory and no
// block waiting for another; chains in turn, or by tickets the longest first (packed).
// Tiles of several whole sequences: in turn.
template <typename E, bool kBack, bool kTma, Mode kMode>
__global__ void __launch_bounds__(Shape<E, kBack, kTma, kMode>::kThreads, Shape<E, kBack, kTma, kMode>::kBlocks)
    gated_scan_kernel(const __grid_constant__ Params<E> p, const __grid_constant__ Maps maps) {
  using S = Shape<E, kBack, kTma, kMode>;
  constexpr int K = S::kRows, kWarps = S::kWarps;
  const bool waits = kMode == kByTiles || (kMode == kMixed && p.runs);  // states pass from block to block
  extern __shared__ __align__(128) char shared[];
  auto& sm = *reinterpret_cast<ScanSmem<kMode, kWarps>*>(shared + kStages * S::kStageBytes);
  // uniform in the warp, and known to be
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int mine = (kBack ? kWarps - 1 - warp : warp) * K;  // the warp's first row in a stage

  if (threadIdx.x == 0) {
    sm.abort = 0;
    if constexpr (kTma) {
      for (int i = 0; i < kWarps * kStages; ++i) lap::mbar_init(&sm.bar[0][0] + i, 1);
      lap::fence_mbar_init();
    }
  }
  if (threadIdx.x < 2) {
    for (int w = 0; w < 8; ++w) sm.turn[threadIdx.x].late[w] = sm.turn[threadIdx.x].begins[w] = 0;
  }
  lap::griddep_wait();
  lap::griddep_launch_dependents();

  // Thread 0's: the number of the next tile or chain (asked for early, looked at late), and the tile.
  const int total = (p.order || p.table ? p.ticket[2] : p.tiles) * p.columns;
  const int part0 = kBack && kMode == kByChains && p.table ? p.ticket[kTicket + 2] : 0;  // sums of dslopes before the chains'
  constexpr Tile kNone{-1, 0, 0, 0, 0, 0, 0, 0};
  Tile chain{0, 0, 0, 0, 0, 0, 0, 0};
  int step = 0, steps = 0, turns = static_cast<int>(blockIdx.x);
  auto next_id = [&] {
    if (waits || (kMode == kByChains && p.order && step == steps)) return atomicAdd(p.ticket, 1);
    return 0;
  };
  auto tile_of = [&](int id) -> Tile {
    if constexpr (kMode == kByChains) {
      if (step == steps) {  // the next chain
        if (!p.order) {
          id = turns;
          turns += static_cast<int>(gridDim.x);
        }
        const int place = id / p.columns;
        if (p.order ? id >= total : place >= p.N) return kNone;
        chain.column = id - place * p.columns;
        chain.t = part0 + place;
        chain.n = p.order ? p.order[place] : place;
        chain.row = p.order ? p.cu_seqlens[chain.n] : place * p.T;  // of the sequence
        chain.left = p.order ? p.cu_seqlens[chain.n + 1] - chain.row : p.T;
        step = 0;
        steps = chain.left <= p.stride ? 1 : (chain.left + p.stride - 1) / p.stride;
      }
      Tile q = chain;
      q.i = step;
      q.left -= step * p.stride;
      q.row += kBack ? q.left - p.stride : step * p.stride;
      ++step;
      return q;
    } else {
      if (!waits) {
        id = turns;
        turns += static_cast<int>(gridDim.x);
      }
      if (id >= total) return kNone;
      const int place = id / p.columns, column = id - place * p.columns;
      if constexpr (kMode == kByTiles) {
        if (p.table) {
          Tile q = p.table[place];
          q.column = column;
          return q;
        }
        const int i = place / p.N, n = place - i * p.N, left = p.T - i * p.stride;
        return {n * p.per + i, column, n, i, i % p.group, n * p.groups + i / p.group,
                n * p.T + (kBack ? left - p.stride : i * p.stride), left};
      } else {
        const int at = waits && kBack ? p.tiles - 1 - place : place, i = waits ? place : 0;
        return {at, column, 0, i, i % p.group, i / p.group, at * p.stride, -1};
      }
    }
  };
  int loaded = -1;  // the last turn whose tile has been asked for
  auto load = [&](int turn) {
    const Tile& q = sm.tile[turn & 3];
    if (q.t >= 0) {
      if (!kTma || lane == 0)
        fetch<kMode, kBack, kTma>(p, maps, shared + turn % kStages * S::kStageBytes, &sm.bar[warp][turn % kStages],
                           q.row + (kBack ? p.stride - S::kTileRows : 0), q.column, mine, lane);
      loaded = turn;
    } else if constexpr (!kTma) {
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  // What has_edges wants to know of a tile, a turn ahead of its use.
  auto look_up = [&](const Tile& q) {
    if (q.t < 0) return 0;
    if constexpr (kMode == kMixed) return p.places ? p.places[q.t].y : 0;
    return p.state_indices ? p.state_indices[q.n] : q.n;
  };

  if (threadIdx.x == 0) {
    sm.tile[0] = tile_of(next_id());
    // blocks that have one tile each take no second one ahead of a block that starts later
    sm.tile[1] = waits && total <= static_cast<int>(gridDim.x) ? kNone : tile_of(next_id());
  }
  __syncthreads();
  load(0);
  load(1);
  int inside = look_up(sm.tile[0]);
  f2 slope = load_state(p.slopes, 0, p.C, Lane<kTma>(sm.tile[0].column, lane, p.C));
  f2 ds = f2_all(0.f);

  for (int turn = 0;; ++turn) {
    Tile q = sm.tile[turn & 3];  // uniform, and known to be
    q.t = __shfl_sync(0xFFFFFFFFu, q.t, 0);
    q.column = __shfl_sync(0xFFFFFFFFu, q.column, 0);
    q.i = __shfl_sync(0xFFFFFFFFu, q.i, 0);
    q.row = __shfl_sync(0xFFFFFFFFu, q.row, 0);
    if constexpr (kMode != kMixed) {
      q.n = __shfl_sync(0xFFFFFFFFu, q.n, 0);
      q.left = __shfl_sync(0xFFFFFFFFu, q.left, 0);
    }
    if constexpr (kMode != kByChains) {
      q.j = __shfl_sync(0xFFFFFFFFu, q.j, 0);
      q.g = __shfl_sync(0xFFFFFFFFu, q.g, 0);
    }
    if (q.t < 0) break;
    auto& ex = sm.turn[turn & 1];
    const Tile& then = sm.tile[(turn + 1) & 3];
    const bool more = threadIdx.x == 0 && then.t >= 0;
    const int ahead = more ? next_id() : 0;
    const int next_inside = look_up(then);
    const f2 next_slope = load_state(p.slopes, 0, p.C, Lane<kTma>(then.column, lane, p.C));
    const bool edges = __any_sync(0xFFFFFFFFu, has_edges<kMode, K>(p, q, inside, warp));
    auto start_state = [&] {
      if (kMode == kMixed || inside < 0 || inside >= p.pool_size) return f2_all(0.f);
      return load_state(p.start, inside, p.C, Lane<kTma>(q.column, lane, p.C));
    };
    const f2 start = kMode == kByChains && q.i == 0 ? start_state() : f2_all(0.f);
    const int low = q.row + (kBack ? p.stride - S::kTileRows : 0) + mine;
    const char* stage = shared + turn % kStages * S::kStageBytes + mine * S::kPitch;
    // thread 0: whether the next tile but one is copied from the table, with the words
    const auto listed = [&] { return kMode == kByTiles && p.table && more && ahead < total; };
    auto ask = [&] {
      if (listed()) {
        const Tile* from = p.table + ahead / p.columns;
        Tile* to = &sm.tile[(turn + 2) & 3];
        copy16(lap::smem_u32(to), from);
        copy16(lap::smem_u32(to) + 16, reinterpret_cast<const char*>(from) + 16);
      }
      if (waits) Needs<kMode, kWarps>(p, q, warp).ask(p, ex, q, warp, lane);
    };
    unsigned begins = 0u;
    auto close = [&](const Run& run) {  // the warp's rows are composed
      ex.own[warp][lane] = run;
      if (kMode == kMixed && lane == 0) ex.begins[warp] = begins != 0u;
      if (threadIdx.x == 0) {
        if (!listed()) sm.tile[(turn + 2) & 3] = more ? tile_of(ahead) : kNone;
        if (kMode == kMixed) ex.fresh = begins & 1u;
      }
      if (waits) {
        // the first group's; before the barrier, so read before any block may write a final state there
        if (warp == kWarps - 1 && q.i == q.j) ex.base[lane] = start_state();
        Needs<kMode, kWarps>(p, q, warp).look(ex, q, warp, lane);
        if (listed()) sm.tile[(turn + 2) & 3].column = ahead % p.columns;
      }
    };
    const bool here = arrived<kTma>(&sm.bar[warp][turn % kStages], turn / kStages, &sm.abort);
    if constexpr (!kBack) {
      Forward<E, kTma, kMode> f;
      // u <= slope: where all of the tile's slopes are small, so is every u
      const float2 s = f2_unpack(slope);
      const bool small = __all_sync(0xFFFFFFFFu, s.x < kNear && s.y < kNear);
      Run run;
      if (kMode == kMixed && edges) {
        const Rows rows = rows_of<kMode, kBack, K>(p, q, warp, lane);
        begins = rows.begin;
        run = f.template first<true, false>(p, stage, low, slope, rows, Lane<kTma>(q.column, lane, p.C), lane, ask);
      } else if (small) {
        run = f.template first<false, true>(p, stage, low, slope, Rows{}, Lane<kTma>(q.column, lane, p.C), lane, ask);
      } else {
        run = f.template first<false, false>(p, stage, low, slope, Rows{}, Lane<kTma>(q.column, lane, p.C), lane, ask);
      }
      close(run);
      if (__syncthreads_or(!here)) break;
      load(turn + kStages);  // every warp has this tile's rows in registers: its stage takes the tile after next
      const f2 h = state_before<kMode>(p, ex, sm.turn[(turn + 1) & 1], q, run, start, warp, lane);
      if (edges)
        f.template second<true>(p, low, h, rows_of<kMode, kBack, K>(p, q, warp, lane), Lane<kTma>(q.column, lane, p.C));
      else
        f.template second<false>(p, low, h, Rows{}, Lane<kTma>(q.column, lane, p.C));
    } else {
      Backward<E, kTma, kMode> f;
      const Lane<kTma> l(q.column, lane, p.C);
      Run run;
      if (kMode == kMixed && edges) {
        const Rows rows = rows_of<kMode, kBack, K>(p, q, warp, lane);
        begins = rows.begin;
        run = f.template first<true, false>(p, stage, low, slope, rows, l, lane, ask);
      } else {
        // as forward; 600 sequences of up to 128 tokens, 2048 channels: 314 us, 321 without (2 x 8192
        // tokens of 8192 channels 388 and 383, 32768 of 4096 450 and 453)
        const float2 s = f2_unpack(slope);
        if (kMode != kMixed && __all_sync(0xFFFFFFFFu, s.x < kNear && s.y < kNear))
          run = f.template first<false, true>(p, stage, low, slope, Rows{}, l, lane, ask);
        else
          run = f.template first<false, false>(p, stage, low, slope, Rows{}, l, lane, ask);
      }
      close(run);
      if (__syncthreads_or(!here)) break;
      const f2 w = state_before<kMode>(p, ex, sm.turn[(turn + 1) & 1], q, run, start, warp, lane);
      const f2 sum = edges ? f.template second<true>(p, stage, low, slope, w, rows_of<kMode, kBack, K>(p, q, warp, lane), l, lane)
                           : f.template second<false>(p, stage, low, slope, w, Rows{}, l, lane);
      ds = f2_add(ds, sum);
      __syncthreads();
      load(turn + kStages);
      if (kMode != kByChains || q.left <= p.stride) {  // the end of a tile or chain: its terms of dslopes, warps in order
        ex.own[warp][lane].h = ds;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int i = 1; i < kWarps; ++i) ds = f2_add(ds, ex.own[i][lane].h);
          store_state(p.part, q.t, p.C, l, ds);
        }
        ds = f2_all(0.f);
      }
    }
    if (edges) empty_sequences<kMode, kWarps>(p, q, Lane<kTma>(q.column, lane, p.C), warp);
    inside = next_inside;
    slope = next_slope;
  }
  if constexpr (kTma) {
    if (sm.abort && lane == 0) {  // a load did not arrive in time: tell the others, outlive the copies in flight
      report(p.dev_error, kErrTimeout);
      if (p.ticket) atomicExch(p.ticket + 1, 1);
      for (int turn = loaded; turn >= 0 && turn > loaded - kStages; --turn)
        lap::mbar_wait_drain(&sm.bar[warp][turn % kStages], turn / kStages & 1);
    }
  }
}

// out[c] = sum over rows of part[rows][C] (0 rows: 0; `count`: a packed scan's tiles and chains), unless
// the scan was skipped: 32 channels a block, each warp every 32nd row, the warps' sums in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int rows, int C, const int* ticket,
                                                          bool count, float* out) {
  __shared__ float sums[32][33];
  lap::griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  if (ticket && *ticket >= 1 << 30) return;  // cu_seqlens was refused
  if (count) rows = ticket[2] + ticket[kTicket + 2];
  float s = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int i = warp; i < rows; i += 32) s += part[static_cast<size_t>(i) * C + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sums[i][lane];
    out[c] = s;
  }
}

// ---------------------------------------------------------------- decode, verify, commit

// kVec = 4: four neighbouring channels per thread, 8- or 16-byte loads; kVec = 1: two channels, a
// block's width apart, element by element.  Either way the same arithmetic per channel.
template <typename E, int kVec>
struct Chunk;  // as loaded
template <>
struct Chunk<float, 4> {
  float4 w;
  __device__ __forceinline__ f2 get(int i) const { return i == 0 ? f2_pack(w.x, w.y) : f2_pack(w.z, w.w); }
};
template <>
struct Chunk<__nv_bfloat16, 4> {
  uint2 w;
  __device__ __forceinline__ f2 get(int i) const { return lap::bf16x2_to_f2(i == 0 ? w.x : w.y); }
};
template <typename E>
struct Chunk<E, 1> {
  E a, b;
  __device__ __forceinline__ f2 get(int) const { return f2_pack(to_f32(a), to_f32(b)); }
};
template <typename E, int kVec>
__device__ __forceinline__ Chunk<E, kVec> load_chunk(const E* row, int c, bool second) {
  Chunk<E, kVec> q;
  if constexpr (kVec == 4) {
    q.w = *reinterpret_cast<const decltype(q.w)*>(row + c);
  } else {
    q.a = row[c];
    q.b = second ? row[c + kThreads] : row[c];
  }
  return q;
}
template <int kVec, typename E>
__device__ __forceinline__ void store_chunk(E* row, int c, bool second, const f2 (&v)[2]) {
  const float2 a = f2_unpack(v[0]), b = f2_unpack(v[1]);
  if constexpr (kVec == 4 && sizeof(E) == 4) {
    *reinterpret_cast<float4*>(row + c) = make_float4(a.x, a.y, b.x, b.y);
  } else if constexpr (kVec == 4) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(b.x, b.y);
    *reinterpret_cast<uint2*>(row + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    row[c] = from_f32<E>(a.x);
    if (second) row[c + kThreads] = from_f32<E>(a.y);
  }
}

// Each thread walks a request's tokens for its channels.  The states are read and written once; many
// threads with the loads of kAhead tokens in flight each keep the memory busy.  The next tokens' loads
// are issued once these are computed, so where few requests leave the memory idle (128 x 8: 0.77 of the
// copy rate) it is their latency that bounds.  BF16 requests of 8192 channels, 128 x 1 token 4.8 us,
// 128 x 8 14.5 (verify 14.5; commit of 0 to 8 tokens 10.0), 4096 x 8 of 4096 channels 188 (0.95); with 4
// tokens ahead and 8 blocks per SM 5.1, 13.8, 189; with 8 ahead (registers spill) 20, 40, 487.
template <typename E, int kVec>
__global__ void __launch_bounds__(kThreads, 12) gated_decode_kernel(const Params<E> p) {
  using Q = Chunk<E, kVec>;
  constexpr int kPairs = kVec == 4 ? 2 : 1, kAhead = sizeof(E) == 2 ? 2 : 1, kSpan = kThreads * (kVec == 4 ? 4 : 2);
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int tiles = (p.C + kSpan - 1) / kSpan;
  const int n = static_cast<int>(blockIdx.x) / tiles;
  const int c = (static_cast<int>(blockIdx.x) - n * tiles) * kSpan + static_cast<int>(threadIdx.x) * (kVec == 4 ? 4 : 1);
  const bool second = c + kThreads < p.C;  // kVec = 1
  const int slot = slot_of(p, n);
  if (slot < 0 || c >= p.C) return;
  int rows = p.T;
  if (p.accepted_len) {
    rows = min(max(p.accepted_len[n], 0), p.T);
    if (rows == 0) return;
  }
  const int64_t first = static_cast<int64_t>(n) * p.T;
  const size_t at = static_cast<size_t>(slot) * p.C;
  const auto slope = load_chunk<float, kVec>(p.slopes, c, second);
  f2 h[2];
  {
    const auto q = load_chunk<float, kVec>(p.start + at, c, second);
#pragma unroll
    for (int i = 0; i < 2; ++i) h[i] = q.get(i);
  }
  for (int t0 = 0; t0 < rows; t0 += kAhead) {
    Q x[kAhead], r[kAhead], g[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (t0 + k < rows) {
        const int64_t row = first + t0 + k;
        r[k] = load_chunk<E, kVec>(p.in[1] + row * p.ld_in[1], c, second);
        g[k] = load_chunk<E, kVec>(p.in[2] + row * p.ld_in[2], c, second);
        x[k] = load_chunk<E, kVec>(p.in[0] + row * p.ld_in[0], c, second);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (t0 + k >= rows) break;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        f2 a, b;
        step2<false>(slope.get(i), x[k].get(i), r[k].get(i), at_most_open2(g[k].get(i)), &a, &b);
        h[i] = f2_fma(a, h[i], b);
      }
      if (p.out[0]) store_chunk<kVec, E>(p.out[0] + (first + t0 + k) * p.ld_out[0], c, second, h);
    }
  }
  if (p.finish) store_chunk<kVec, float>(p.finish + at, c, second, h);
}

}  // namespace lag
