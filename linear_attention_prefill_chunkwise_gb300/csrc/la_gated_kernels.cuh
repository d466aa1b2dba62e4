// la_gated_kernels.cuh -- kernels of the gated linear recurrence (include/la_gated.h).
//
// The scan.  With a_t = lambda_t and b_t the token's input (beta_t sig(g_t) x_t forward; lambda_t
// dout_t backward, where the state is w_t = lambda_t G_t and tokens are walked from the end), a
// run of tokens maps the state before it to A h + H, A the product of its a's and H its own scan
// from zero; two runs compose as (A2 A1, A2 H1 + H2).  So the rows of the whole batch, sequence
// after sequence, are one scan whose state is replaced where a sequence begins: the rows are cut
// into tiles whatever the sequences' lengths, which balances packed batches by construction.
//
// A tile is kWarps x kRows rows of 64 channels, two channels per lane, kRows rows per warp.  Blocks
// are persistent, and each warp has two stages of shared memory for its rows of the inputs: while
// one tile is computed the loads of the next are in flight, each warp's own TMA boxes (or, where
// rows are not 16-byte aligned, its own asynchronous 4-byte copies), so no warp waits for another's
// loads.  A warp composes its rows, the block its warps, and the tile's (A, H) is published in the
// workspace.  Once the state before the tile is known, each warp walks its rows again (forward:
// from a and b in registers) and writes the outputs: every input is read once and every output
// written once.
// The state before a tile: tiles are taken in order (by a ticket, so that whatever a block waits
// for is already running), in groups of `group` along the rows.  A tile composes the published
// (A, H) of the tiles before it in its group, in order, onto the state that the previous group's
// last tile published; a long scan is thus a chain of one step per group, not per tile.  The
// order of every sum is fixed, so results repeat bitwise.
// A published word carries its own readiness: the workspace is filled with all-ones before the
// scan (a NaN pattern that no arithmetic produces), a tile's (A, H) is one 64-bit store, and a
// reader polls the word itself: no fence and no second flag on the way from block to block.
// Where a sequence begins, A becomes -0: products of decays are >= +0, so the sign marks "what
// came before does not matter", and composition then selects H instead of multiplying, which keeps
// infinities and NaN of one sequence out of the next.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "la_gated_math.cuh"
#include "sm103_ptx.cuh"

namespace lag {

constexpr unsigned kErrBadSeqlens = 1u, kErrBadIndex = 2u, kErrTimeout = 4u;
constexpr int kCols = 64;       // channels of a tile: two per lane
constexpr int kWarps = 8;       // warps of a scan block
constexpr int kScanThreads = kWarps * 32;
constexpr int kThreads = 128;   // threads of the small kernels
constexpr int kMaxInputs = 5;   // x, r, g; backward: dout and o (one row up: h_{t-1}) too
constexpr int kStages = 2;

// Shape of a scan kernel: rows per warp, blocks per SM and the stages' layout.  kTma: rows arrive
// by TMA boxes of kRows x 64 channels; else by 4-byte copies, and a BF16 row takes one word more
// where it begins in the middle of a word.
template <typename E, bool kBack, bool kTma>
struct Shape {
  static constexpr int kRows = sizeof(E) == 2 ? 8 : 4;
  static constexpr int kBlocks = kBack ? 2 : 3;
  static constexpr int kTileRows = kWarps * kRows;
  static constexpr int kInputs = kBack ? 5 : 3;
  static constexpr int kPitch = kCols * sizeof(E) + (kTma || sizeof(E) == 4 ? 0 : 4);  // bytes of a row
  static constexpr int kInputBytes = kRows * kPitch;                                 // one input, one warp
  static constexpr int kStageBytes = (kInputs * kInputBytes + 127) / 128 * 128;
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
  float* part;         // backward: [tiles, C] sums of each tile's terms of dslopes
  const int32_t* state_indices;
  const int32_t* cu_seqlens;
  const int32_t* accepted_len;  // commit
  int* dev_error;
  // the workspace of a scan
  int* ticket;         // next tile, then an abort flag; null: blocks take tiles in turn, nothing is waited for
  int32_t* first_seq;  // [tiles + 1] (packed) first sequence that begins at or after the tile's first row
  float2* runs;        // [tiles][padded C] published (A, H)
  float* before;       // [groups][padded C] published states after each group
  int T, N, C, pool_size, rows;
  int tiles, columns, stride, group;  // tiles along the rows, of `stride` rows; along the channels; per group
};

struct Maps {
  CUtensorMap of[kMaxInputs];
};

__device__ __forceinline__ void report(int* dev_error, unsigned bit) {
  if (dev_error) atomicOr(reinterpret_cast<unsigned*>(dev_error), bit);
}

// ---------------------------------------------------------------- before a scan

// Fills the published words, sets the ticket and, for a packed batch, checks cu_seqlens
// (non-decreasing inside [0, T]; if not, the ticket starts past the last tile, so that the scan
// does nothing) and finds the sequences of each tile.
template <typename E>
__global__ void __launch_bounds__(kThreads) scan_plan_kernel(const Params<E> p, size_t words) {
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const size_t id = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x;
  const size_t all = static_cast<size_t>(gridDim.x) * kThreads;
  uint4* w = reinterpret_cast<uint4*>(p.runs);  // runs and before lie together, 16-byte multiples
  for (size_t i = id; i < words / 4; i += all) w[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  if (p.cu_seqlens) {
    for (size_t i = id; i <= static_cast<size_t>(p.tiles); i += all) {
      const int64_t row = static_cast<int64_t>(i) * p.stride;
      int a = 0, b = p.N;  // the first n with cu[n] >= row; the last tile owns the rest
      while (a < b) {
        const int m = (a + b) / 2;
        if (p.cu_seqlens[m] >= row) b = m; else a = m + 1;
      }
      p.first_seq[i] = i == static_cast<size_t>(p.tiles) ? p.N : a;
    }
  }
  if (blockIdx.x == 0) {
    int wrong = 0;
    if (p.cu_seqlens)
      for (int n = threadIdx.x; n < p.N; n += kThreads)
        wrong |= p.cu_seqlens[n] < 0 || p.cu_seqlens[n] > p.cu_seqlens[n + 1] || p.cu_seqlens[n + 1] > p.T;
    wrong = __syncthreads_or(wrong);
    if (threadIdx.x == 0) {
      p.ticket[0] = wrong ? 1 << 30 : 0;
      p.ticket[1] = 0;
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
__device__ __forceinline__ int slot_of(const Params<E>& p, int n) {
  const int slot = p.state_indices ? p.state_indices[n] : n;
  if (slot >= p.pool_size) {
    report(p.dev_error, kErrBadIndex);
    return -1;
  }
  return slot;
}

template <bool kBack, int K, typename E>
__device__ __forceinline__ Rows rows_of(const Params<E>& p, int tile, int warp, int lane) {
  Rows q{0u, 0u, 0u, -1};
  const int place = warp * K + lane;  // in walking order
  const int at = kBack ? p.stride - 1 - place : place;
  const int64_t row = static_cast<int64_t>(tile) * p.stride + at;
  bool first = false, last = false;
  if (lane < K && place < p.stride && row < p.rows) {
    if (p.cu_seqlens) {
      int a = p.first_seq[tile], b = p.first_seq[tile + 1];
      while (a < b) {  // the number of sequences that begin at or before the row
        const int m = (a + b) / 2;
        if (p.cu_seqlens[m] <= row) a = m + 1; else b = m;
      }
      if (a > 0) {
        const int lo = p.cu_seqlens[a - 1], hi = p.cu_seqlens[a];
        if (row < hi) {
          q.slot = slot_of(p, a - 1);
          first = row == lo;
          last = row == hi - 1;
        }
      }
    } else {
      const int n = static_cast<int>(row) / p.T, t = static_cast<int>(row) - n * p.T;
      q.slot = slot_of(p, n);
      first = t == 0;
      last = t == p.T - 1;
    }
  }
  q.live = __ballot_sync(0xFFFFFFFFu, q.slot >= 0);
  q.begin = __ballot_sync(0xFFFFFFFFu, q.slot >= 0 && (kBack ? last : first));
  q.end = __ballot_sync(0xFFFFFFFFu, q.slot >= 0 && (kBack ? first : last));
  return q;
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

// Output rows: the lane's two channels (a TMA kernel's rows hold an even number of channels).
template <bool kTma>
__device__ __forceinline__ void store2(float* row, const Lane<kTma>& l, f2 v) {
  const float2 t = f2_unpack(v);
  if constexpr (kTma) {
    if (l.ok[0]) __stcs(reinterpret_cast<float2*>(row + l.c[0]), t);
  } else {
    if (l.ok[0]) __stcs(row + l.c[0], t.x);
    if (l.ok[1]) __stcs(row + l.c[1], t.y);
  }
}
template <bool kTma>
__device__ __forceinline__ void store2(__nv_bfloat16* row, const Lane<kTma>& l, f2 v) {
  const float2 t = f2_unpack(v);
  const __nv_bfloat162 b = __floats2bfloat162_rn(t.x, t.y);
  const unsigned w = *reinterpret_cast<const unsigned*>(&b);
  unsigned short* s = reinterpret_cast<unsigned short*>(row);
  if constexpr (kTma) {
    if (l.ok[0]) __stcs(reinterpret_cast<unsigned*>(s + l.c[0]), w);
  } else {
    if (l.ok[0]) __stcs(s + l.c[0], static_cast<unsigned short>(w));
    if (l.ok[1]) __stcs(s + l.c[1], static_cast<unsigned short>(w >> 16));
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

__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Starts the loads of a warp's kRows rows (the lowest is row `low`) of every input into `stage`.
template <bool kBack, bool kTma, typename E>
__device__ __forceinline__ void fetch(const Params<E>& p, const Maps& maps, char* stage, uint64_t* bar, int low,
                                      int column, int lane) {
  using S = Shape<E, kBack, kTma>;
  if constexpr (kTma) {
    if (lane == 0) {
      lap::mbar_arrive_expect_tx(bar, S::kInputs * S::kInputBytes);
#pragma unroll
      for (int i = 0; i < S::kInputs; ++i)  // o one row up; rows outside the matrix arrive as zeros
        lap::tma_load_2d(stage + i * S::kInputBytes, &maps.of[i], bar, column * kCols, low - (i == 4));
    }
  } else {
    const uint32_t to = lap::smem_u32(stage);
    const int64_t last = static_cast<int64_t>(p.rows) - 1;
#pragma unroll
    for (int i = 0; i < S::kInputs; ++i) {
#pragma unroll
      for (int k = 0; k < S::kRows; ++k) {
        const int64_t row = static_cast<int64_t>(low) + k - (i == 4);
        if (row < 0 || row > last) continue;
        const int64_t first = row * p.ld_in[i] + column * kCols;  // element of the matrix
        const uint32_t dst = to + i * S::kInputBytes + k * S::kPitch;
        const E* src = p.in[i] + first;
        if constexpr (sizeof(E) == 4) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (column * kCols + lane + 32 * j < p.C) copy4(dst + 4 * (lane + 32 * j), src + lane + 32 * j);
        } else {
          // whole words that hold a channel of this tile; a word's other half may be a neighbour
          // inside the matrix, but nothing outside it is read
          const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(src) >> 1 & 1u);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int w = lane + 32 * j;
            if (j == 1 && (lane > 0 || !odd)) break;
            const int e = 2 * w - odd, c = column * kCols + e;
            if (c + (e < 0) >= p.C) continue;
            if (first + e >= 0 && first + e + 1 <= last * p.ld_in[i] + p.C - 1) {
              copy4(dst + 4 * w, src + e);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (e + h >= 0 && c + h < p.C)
                  asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + 4 * w + 2 * h),
                               "h"(reinterpret_cast<const unsigned short*>(src)[e + h])
                               : "memory");
            }
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
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    return true;
  }
}

// A lane's view of one input's rows in a stage.
template <typename E, bool kBack, bool kTma>
struct View {
  using S = Shape<E, kBack, kTma>;
  const char* at[2];  // of even and odd rows of the stage: they may begin at different half words
  __device__ __forceinline__ View(const Params<E>& p, const char* stage, int i, int low, int lane) {
    const char* s = stage + i * S::kInputBytes;
    if constexpr (kTma) {
      at[0] = at[1] = s + lane * 2 * sizeof(E);
    } else if constexpr (sizeof(E) == 4) {
      at[0] = at[1] = s + lane * 4;
    } else {
      const unsigned base = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p.in[i]) >> 1);
      const unsigned row = static_cast<unsigned>(low - (i == 4)), ld = static_cast<unsigned>(p.ld_in[i]);
      at[0] = s + 2 * (lane + ((base + row * ld) & 1u));
      at[1] = s + 2 * (lane + ((base + (row + 1) * ld) & 1u));
    }
  }
  __device__ __forceinline__ f2 get(int k) const {
    const char* s = at[k & 1] + k * S::kPitch;
    if constexpr (sizeof(E) == 4) {
      if constexpr (kTma) return *reinterpret_cast<const f2*>(s);
      return f2_pack(*reinterpret_cast<const float*>(s), *reinterpret_cast<const float*>(s + 128));
    } else {
      if constexpr (kTma) return lap::bf16x2_to_f2(*reinterpret_cast<const uint32_t*>(s));
      const unsigned lo = *reinterpret_cast<const unsigned short*>(s);
      const unsigned hi = *reinterpret_cast<const unsigned short*>(s + 64);
      return f2_pack(__uint_as_float(lo << 16), __uint_as_float(hi << 16));
    }
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

constexpr unsigned long long kUnset = ~0ull;

__device__ __forceinline__ void publish_run(float2* at, const Run& r) {
  const float2 a = f2_unpack(r.a), h = f2_unpack(r.h);
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(at), "l"(f2_pack(a.x, h.x)), "l"(f2_pack(a.y, h.y))
               : "memory");
}
__device__ __forceinline__ unsigned ready_bits(float v) {
  const unsigned u = __float_as_uint(v);
  return u == ~0u ? 0x7FFFFFFFu : u;  // a NaN that looks unset becomes another NaN
}
__device__ __forceinline__ void publish_state(float* at, f2 state) {
  const float2 h = f2_unpack(state);
  asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(at), "r"(ready_bits(h.x)), "r"(ready_bits(h.y))
               : "memory");
}

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

__device__ __forceinline__ Run await_run(const float2* at, int* ticket, int* dev_error) {
  unsigned long long u, v;
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(u), "=l"(v) : "l"(at) : "memory");
    if (u != kUnset && v != kUnset) break;
    if (i == 0) t0 = lap::globaltimer_ns();
    if ((i & 15u) == 15u && !keep_polling(ticket, dev_error, t0)) break;
  }
  const float2 x = f2_unpack(u), y = f2_unpack(v);
  return {f2_pack(x.x, y.x), f2_pack(x.y, y.y)};
}

__device__ __forceinline__ f2 await_state(const float* at, int* ticket, int* dev_error) {
  unsigned u, v;
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(u), "=r"(v) : "l"(at) : "memory");
    if (u != ~0u && v != ~0u) break;
    if (i == 0) t0 = lap::globaltimer_ns();
    if ((i & 15u) == 15u && !keep_polling(ticket, dev_error, t0)) break;
  }
  return f2_pack(__uint_as_float(u), __uint_as_float(v));
}

// What a tile shares between its warps; two of them in turn, so that a warp may begin the next
// tile while another still reads this one's.
struct Exchange {
  Run own[kWarps][32];  // each warp's rows
  int next;             // the tile to load next
  int fresh;            // the tile's first row begins a sequence
};
struct ScanSmem {
  Exchange turn[2];
  Run earlier[kWarps][32];  // pieces of the group's earlier tiles, in order
  f2 base[32];              // the state before the group
  uint64_t bar[kWarps][kStages];
  int first;                // the block's first tile
  int abort;                // a load did not arrive
};

template <typename E, bool kBack, bool kTma>
__host__ __device__ constexpr int scan_smem_bytes() {
  return kStages * kWarps * Shape<E, kBack, kTma>::kStageBytes + static_cast<int>(sizeof(ScanSmem));
}

// The state before this warp's rows.  `mine` (in ex.own already) is the composition of the warp's
// rows; t the tile in walking order.  Publishes the tile for those that follow.
template <typename E>
__device__ __forceinline__ f2 state_before(const Params<E>& p, ScanSmem& sm, Exchange& ex, const Run& mine, int t,
                                           int column, int warp, int lane) {
  f2 before = f2_all(0.f);
  if (p.ticket) {
    const size_t width = static_cast<size_t>(p.columns) * kCols;
    const size_t at = static_cast<size_t>(column) * kCols + 2 * lane;
    const int group = t / p.group, j = t - group * p.group;
    const bool last = j == p.group - 1;
    Run whole;
    if (warp == 0) {
      whole = mine;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) whole = compose(whole, ex.own[w][lane]);
      if (!last) publish_run(p.runs + t * width + at, whole);
    }
    if (!ex.fresh) {
      // this warp's piece of the earlier tiles
      const int per = (j + kWarps - 1) / kWarps, lo = min(j, warp * per), hi = min(j, lo + per);
      const size_t g0 = static_cast<size_t>(group) * p.group;
      if (lo < hi) {
        Run q = await_run(p.runs + (g0 + lo) * width + at, p.ticket, p.dev_error);
#pragma unroll 1
        for (int i = lo + 1; i < hi; ++i) q = compose(q, await_run(p.runs + (g0 + i) * width + at, p.ticket, p.dev_error));
        sm.earlier[warp][lane] = q;
      }
      if (warp == kWarps - 1)
        sm.base[lane] = group == 0 ? before : await_state(p.before + (group - 1) * width + at, p.ticket, p.dev_error);
      __syncthreads();
      before = sm.base[lane];
      const int pieces = j == 0 ? 0 : (j + per - 1) / per;
#pragma unroll 1
      for (int i = 0; i < pieces; ++i) before = apply(sm.earlier[i][lane], before);
    }
    if (warp == 0 && last) publish_state(p.before + group * width + at, apply(whole, before));
  }
#pragma unroll 1
  for (int w = 0; w < warp; ++w) before = apply(ex.own[w][lane], before);
  return before;
}

// The final states of the empty sequences that lie in this tile: their initial ones.
template <typename E, bool kTma>
__device__ __forceinline__ void empty_sequences(const Params<E>& p, int tile, const Lane<kTma>& l, int warp) {
  if (!p.finish || (!p.cu_seqlens && p.T > 0)) return;
  const int lo = p.cu_seqlens ? p.first_seq[tile] : 0, hi = p.cu_seqlens ? p.first_seq[tile + 1] : p.N;
  for (int n = lo + warp; n < hi; n += kWarps) {
    if (p.cu_seqlens && p.cu_seqlens[n] != p.cu_seqlens[n + 1]) continue;
    const int slot = slot_of(p, n);
    if (slot >= 0) store_state(p.finish, slot, p.C, l, load_state(p.start, slot, p.C, l));
  }
}

// ---------------------------------------------------------------- the forward scan

// a = lambda and b = beta sig(g) x of one token.
__device__ __forceinline__ void step2(f2 slope, f2 x, f2 r, f2 g, f2* a, f2* b) {
  const f2 m = one_minus_lambda2(f2_mul(slope, sigmoid2(r)));
  f2 w;
  const f2 inv = inverse_beta2(m, &w);
  *a = f2_sub(f2_all(1.f), m);
  *b = f2_mul(f2_mul(f2_mul(w, inv), sigmoid2(g)), x);
}

template <typename E, bool kTma>
struct Forward {
  using S = Shape<E, false, kTma>;
  static constexpr int K = S::kRows;
  f2 a[K], b[K];

  // The warp's rows composed.  kEdges: some row begins or ends a sequence or belongs to none.
  template <bool kEdges>
  __device__ __forceinline__ Run first(const Params<E>& p, const char* stage, int low, f2 slope, const Rows& rows,
                                       const Lane<kTma>& l, int lane) {
    const View<E, false, kTma> x(p, stage, 0, low, lane), r(p, stage, 1, low, lane), g(p, stage, 2, low, lane);
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
      f2 in;
      step2(slope, x.get(k), r.get(k), g.get(k), &a[k], &in);
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
    E* o = p.out[0] + static_cast<int64_t>(low) * p.ld_out[0];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (kEdges) {
        if (rows.begin >> k & 1u) h = f2_all(0.f);
      }
      h = f2_fma(a[k], h, b[k]);
      if (!kEdges || (rows.live >> k & 1u)) store2(o + k * p.ld_out[0], l, h);
      if constexpr (kEdges) {
        if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l, h);
      }
    }
  }
};

// ---------------------------------------------------------------- the gradients' scan

template <typename E, bool kTma>
struct Backward {
  using S = Shape<E, true, kTma>;
  static constexpr int K = S::kRows;
  f2 sr[K], m[K];  // sig(r) and 1 - lambda; row k in walking order is row K - 1 - k of the stage

  template <bool kEdges>
  __device__ __forceinline__ Run first(const Params<E>& p, const char* stage, int low, f2 slope, const Rows& rows,
                                       const Lane<kTma>& l, int lane) {
    const View<E, true, kTma> r(p, stage, 1, low, lane), d(p, stage, 3, low, lane);
    Run run{f2_all(1.f), f2_all(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      sr[k] = sigmoid2(r.get(K - 1 - k));
      m[k] = one_minus_lambda2(f2_mul(slope, sr[k]));
      const f2 a = f2_sub(f2_all(1.f), m[k]);
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
    const View<E, true, kTma> x(p, stage, 0, low, lane), g(p, stage, 2, low, lane), d(p, stage, 3, low, lane),
        h(p, stage, 4, low, lane);
    E* out[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) out[i] = p.out[i] + static_cast<int64_t>(low) * p.ld_out[i];
    f2 sum = f2_all(0.f);
    const f2 one = f2_all(1.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int at = K - 1 - k;
      f2 before = h.get(at);
      if constexpr (kEdges) {
        if (!(rows.live >> k & 1u)) continue;
        const int slot = __shfl_sync(0xFFFFFFFFu, rows.slot, k);
        if (rows.begin >> k & 1u) w = load_state(p.start, slot, p.C, l);
        if (rows.end >> k & 1u) before = load_state(p.h0, slot, p.C, l);
      }
      const f2 G = f2_add(d.get(at), w), vx = x.get(at), sg = sigmoid2(g.get(at)), u = f2_mul(slope, sr[k]);
      f2 beta;
      f2 inv = inverse_beta2(m[k], &beta);
      beta = f2_mul(beta, inv);
      const float2 vu = f2_unpack(u), vi = f2_unpack(inv);
      inv = f2_pack(vu.x > 0.f ? vi.x : 0.f, vu.y > 0.f ? vi.y : 0.f);
      const f2 lambda = f2_sub(one, m[k]);
      const f2 gs = f2_mul(G, sg), dx = f2_mul(gs, beta);
      store2(out[0] + at * p.ld_out[0], l, dx);
      store2(out[2] + at * p.ld_out[2], l, f2_mul(f2_mul(dx, vx), f2_sub(one, sg)));
      // du = lambda (gs x lambda / beta - G h_{t-1})
      const f2 t = f2_mul(f2_mul(gs, vx), f2_mul(lambda, inv));
      const f2 du = f2_mul(lambda, f2_sub(t, f2_mul(G, before)));
      store2(out[1] + at * p.ld_out[1], l, f2_mul(f2_mul(du, u), f2_sub(one, sr[k])));
      sum = f2_fma(du, sr[k], sum);
      w = f2_mul(lambda, G);
      if constexpr (kEdges) {
        if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l, w);
      }
    }
    return sum;
  }
};

// ---------------------------------------------------------------- the scan kernel

template <typename E, bool kBack, bool kTma>
__global__ void __launch_bounds__(kScanThreads, Shape<E, kBack, kTma>::kBlocks)
    gated_scan_kernel(const __grid_constant__ Params<E> p, const __grid_constant__ Maps maps) {
  using S = Shape<E, kBack, kTma>;
  constexpr int K = S::kRows;
  extern __shared__ __align__(128) char shared[];
  ScanSmem& sm = *reinterpret_cast<ScanSmem*>(shared + kStages * kWarps * S::kStageBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  char* stages = shared + warp * kStages * S::kStageBytes;
  const int total = p.tiles * p.columns;
  // Blocks that have one tile each take no second one ahead of a block that starts later.
  const bool several = total > static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    sm.abort = 0;
    if constexpr (kTma) {
      for (int i = 0; i < kWarps * kStages; ++i) lap::mbar_init(&sm.bar[0][0] + i, 1);
      lap::fence_mbar_init();
    }
  }
  lap::griddep_wait();
  lap::griddep_launch_dependents();

  // a tile's number is its place in walking order times `columns`, plus its column; -1: none
  auto take = [&](int turn) {
    const int id = p.ticket ? atomicAdd(p.ticket, 1) : static_cast<int>(blockIdx.x) + turn * static_cast<int>(gridDim.x);
    return id < total ? id : -1;
  };
  auto lowest = [&](int id) {  // the warp's lowest row of a tile
    const int t = id / p.columns;
    return kBack ? (p.tiles - 1 - t) * p.stride + p.stride - 1 - warp * K - (K - 1) : t * p.stride + warp * K;
  };
  int loaded = -1;  // the last turn whose tile has been asked for
  auto load = [&](int id, int turn) {
    if (id >= 0) {
      fetch<kBack, kTma>(p, maps, stages + turn % kStages * S::kStageBytes, &sm.bar[warp][turn % kStages], lowest(id),
                         id % p.columns, lane);
      loaded = turn;
    } else if constexpr (!kTma) {
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };

  if (threadIdx.x == 0) sm.first = take(0);
  __syncthreads();
  int id = sm.first, id1 = -1;
  load(id, 0);
  if (several) {
    if (threadIdx.x == 0) sm.turn[1].next = take(1);
    __syncthreads();
    id1 = sm.turn[1].next;
  }
  load(id1, 1);

  for (int turn = 0; id >= 0; ++turn) {
    Exchange& ex = sm.turn[turn & 1];
    const int t = id / p.columns, column = id - t * p.columns, tile = kBack ? p.tiles - 1 - t : t;
    const int low = lowest(id);
    char* stage = stages + (turn % kStages) * S::kStageBytes;
    int ahead = -1;
    if (threadIdx.x == 0 && id1 >= 0) ahead = take(turn + 2);
    const Lane<kTma> l(column, lane, p.C);
    const Rows rows = rows_of<kBack, K>(p, tile, warp, lane);
    constexpr unsigned kFull = (1u << K) - 1u;
    const bool edges = rows.live != kFull || rows.begin || rows.end;
    const f2 slope = load_state(p.slopes, 0, p.C, l);
    const bool here = arrived<kTma>(&sm.bar[warp][turn % kStages], turn / kStages, &sm.abort);
    if (threadIdx.x == 0) {
      ex.next = ahead;
      ex.fresh = rows.begin & 1u;
    }
    int id2 = -1;
    if constexpr (!kBack) {
      Forward<E, kTma> f;
      const Run run = edges ? f.template first<true>(p, stage, low, slope, rows, l, lane)
                            : f.template first<false>(p, stage, low, slope, rows, l, lane);
      ex.own[warp][lane] = run;
      if (__syncthreads_or(!here)) break;
      id2 = ex.next;
      load(id2, turn + kStages);  // this tile's rows are in registers: their stage takes the tile after next
      const f2 h = state_before(p, sm, ex, run, t, column, warp, lane);
      if (edges) f.template second<true>(p, low, h, rows, l);
      else f.template second<false>(p, low, h, rows, l);
    } else {
      Backward<E, kTma> f;
      const Run run = edges ? f.template first<true>(p, stage, low, slope, rows, l, lane)
                            : f.template first<false>(p, stage, low, slope, rows, l, lane);
      ex.own[warp][lane] = run;
      if (__syncthreads_or(!here)) break;
      id2 = ex.next;
      const f2 w = state_before(p, sm, ex, run, t, column, warp, lane);
      const f2 ds = edges ? f.template second<true>(p, stage, low, slope, w, rows, l, lane)
                          : f.template second<false>(p, stage, low, slope, w, rows, l, lane);
      __syncwarp();
      load(id2, turn + kStages);
      // the tile's terms of dslopes, warps in order
      __syncthreads();
      ex.own[warp][lane].h = ds;
      __syncthreads();
      if (warp == 0) {
        f2 sum = ds;
#pragma unroll
        for (int i = 1; i < kWarps; ++i) sum = f2_add(sum, ex.own[i][lane].h);
        store_state(p.part, tile, p.C, l, sum);
      }
    }
    empty_sequences(p, tile, l, warp);
    id = id1;
    id1 = id2;
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

// out[c] = sum over rows of part[rows][C] (0 rows: 0), unless the scan was skipped: 32 channels a
// block, each warp every 32nd row, the warps' sums in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int rows, int C, const int* ticket,
                                                          float* out) {
  __shared__ float sums[32][33];
  lap::griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  if (ticket && *ticket >= 1 << 30) return;  // cu_seqlens was refused
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

// One thread per (request, channel) walks the request's tokens; neighbouring threads hold
// neighbouring channels.
template <typename E>
__global__ void __launch_bounds__(kThreads) gated_decode_kernel(const Params<E> p) {
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int tiles = (p.C + kThreads - 1) / kThreads;
  const int n = static_cast<int>(blockIdx.x / tiles);
  const int c = static_cast<int>(blockIdx.x % tiles) * kThreads + static_cast<int>(threadIdx.x);
  const int slot = slot_of(p, n);
  if (slot < 0 || c >= p.C) return;
  int rows = p.T;
  if (p.accepted_len) {
    rows = min(max(p.accepted_len[n], 0), p.T);
    if (rows == 0) return;
  }
  const float slope = p.slopes[c];
  const size_t at = static_cast<size_t>(slot) * p.C + c;
  float h = p.start[at];
  const int64_t first = static_cast<int64_t>(n) * p.T;
  for (int64_t t = first; t < first + rows; ++t) {
    const float x = to_f32(p.in[0][t * p.ld_in[0] + c]);
    const Decay d = decay_of(slope * sigmoid(to_f32(p.in[1][t * p.ld_in[1] + c])));
    h = fmaf(d.lambda, h, d.beta * sigmoid(to_f32(p.in[2][t * p.ld_in[2] + c])) * x);
    if (p.out[0]) p.out[0][t * p.ld_out[0] + c] = from_f32<E>(h);
  }
  if (p.finish) p.finish[at] = h;
}

}  // namespace lag
