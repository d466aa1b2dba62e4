// la_gated_kernels.cuh -- kernels of the gated linear recurrence (include/la_gated.h).
//
// The scan.  With a_t = lambda_t and b_t the token's input (beta_t sig(g_t) x_t forward; lambda_t
// dout_t backward, where the state is w_t = lambda_t G_t and tokens are walked from the end), a
// run of tokens maps the state before it to A h + H, A the product of its a's and H its own scan
// from zero; two runs compose as (A2 A1, A2 H1 + H2).  So the rows of the whole batch, sequence
// after sequence, are one scan whose state is replaced where a sequence begins: the rows are cut
// into tiles whatever the sequences' lengths, which balances packed batches by construction.
//
// A tile is kWarps x K rows of 64 channels.  Each lane holds two channels of its warp's K rows in
// registers: the warp composes its rows, the block its warps, and the tile's (A, H) is published
// in the workspace.  Once the state before the tile is known, each warp walks its rows again from
// registers and writes the outputs, so every input is read once and every output written once.
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

#include <cuda_bf16.h>
#include <cstdint>

#include "la_gated_math.cuh"
#include "sm103_ptx.cuh"

namespace lag {

constexpr unsigned kErrBadSeqlens = 1u, kErrBadIndex = 2u, kErrTimeout = 4u;
constexpr int kCols = 64;       // channels of a tile: two per lane
constexpr int kWarps = 16;      // warps of a scan block
constexpr int kScanThreads = kWarps * 32;
constexpr int kThreads = 128;   // threads of the small kernels

// Rows per warp: FP32 activations take twice the registers, the gradients five inputs.
template <typename E, bool kBack>
__host__ __device__ constexpr int rows_per_warp() { return (sizeof(E) == 2 ? 8 : 4); }
template <typename E, bool kBack>
__host__ __device__ constexpr int tile_rows() { return kWarps * rows_per_warp<E, kBack>(); }

template <typename E>
struct Params {
  const E *x, *r, *g;
  const E *o_in, *dout;  // backward
  E *o, *dx, *dr, *dg;
  int64_t ldx, ldr, ldg, ldo, lddout, lddx, lddr, lddg;
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
  int* ticket;         // next tile, then an abort flag; null: block b takes tile b, nothing is waited for
  int32_t* first_seq;  // [tiles + 1] (packed) first sequence that begins at or after the tile's first row
  float2* runs;        // [tiles][padded C] published (A, H)
  float* before;       // [groups][padded C] published states after each group
  int T, N, C, pool_size, rows;
  int tiles, columns, stride, group;  // tiles along the rows, of `stride` rows; along the channels; per group
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

template <typename E, bool kBack, int K>
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

// A lane's two channels: neighbours where the rows allow paired loads, else a warp's width apart.
template <bool kPair>
struct Lane {
  int c[2];
  bool ok[2];
  __device__ __forceinline__ Lane(int column, int lane, int C) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = column * kCols + (kPair ? 2 * lane + j : lane + 32 * j);
      ok[j] = c[j] < C;
    }
  }
};

// Two activations as loaded.
template <typename E>
struct Raw;
template <>
struct Raw<float> {
  float a, b;
  __device__ __forceinline__ float2 get() const { return make_float2(a, b); }
};
template <>
struct Raw<__nv_bfloat16> {
  uint32_t w;
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};

template <bool kPair>
__device__ __forceinline__ Raw<float> load2(const float* row, const Lane<kPair>& l) {
  Raw<float> v{0.f, 0.f};
  if constexpr (kPair) {
    if (l.ok[0]) {
      const float2 t = __ldcs(reinterpret_cast<const float2*>(row + l.c[0]));
      v.a = t.x;
      v.b = t.y;
    }
  } else {
    if (l.ok[0]) v.a = __ldcs(row + l.c[0]);
    if (l.ok[1]) v.b = __ldcs(row + l.c[1]);
  }
  return v;
}
template <bool kPair>
__device__ __forceinline__ Raw<__nv_bfloat16> load2(const __nv_bfloat16* row, const Lane<kPair>& l) {
  Raw<__nv_bfloat16> v{0u};
  const unsigned short* s = reinterpret_cast<const unsigned short*>(row);
  if constexpr (kPair) {
    if (l.ok[0]) v.w = __ldcs(reinterpret_cast<const unsigned*>(s + l.c[0]));
  } else {
    unsigned a = 0, b = 0;
    if (l.ok[0]) a = __ldcs(s + l.c[0]);
    if (l.ok[1]) b = __ldcs(s + l.c[1]);
    v.w = a | b << 16;
  }
  return v;
}

template <bool kPair>
__device__ __forceinline__ void store2(float* row, const Lane<kPair>& l, float a, float b) {
  if constexpr (kPair) {
    if (l.ok[0]) __stcs(reinterpret_cast<float2*>(row + l.c[0]), make_float2(a, b));
  } else {
    if (l.ok[0]) __stcs(row + l.c[0], a);
    if (l.ok[1]) __stcs(row + l.c[1], b);
  }
}
template <bool kPair>
__device__ __forceinline__ void store2(__nv_bfloat16* row, const Lane<kPair>& l, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  const unsigned w = *reinterpret_cast<const unsigned*>(&v);
  unsigned short* s = reinterpret_cast<unsigned short*>(row);
  if constexpr (kPair) {
    if (l.ok[0]) __stcs(reinterpret_cast<unsigned*>(s + l.c[0]), w);
  } else {
    if (l.ok[0]) __stcs(s + l.c[0], static_cast<unsigned short>(w));
    if (l.ok[1]) __stcs(s + l.c[1], static_cast<unsigned short>(w >> 16));
  }
}

// A state [P, C] of one slot, the lane's channels; 0 without a pool.
template <bool kPair>
__device__ __forceinline__ float2 load_state(const float* pool, int slot, int C, const Lane<kPair>& l) {
  float2 v = make_float2(0.f, 0.f);
  if (pool) {
    const float* s = pool + static_cast<size_t>(slot) * C;
    if (l.ok[0]) v.x = s[l.c[0]];
    if (l.ok[1]) v.y = s[l.c[1]];
  }
  return v;
}
template <bool kPair>
__device__ __forceinline__ void store_state(float* pool, int slot, int C, const Lane<kPair>& l, float2 v) {
  float* s = pool + static_cast<size_t>(slot) * C;
  if (l.ok[0]) s[l.c[0]] = v.x;
  if (l.ok[1]) s[l.c[1]] = v.y;
}

// ---------------------------------------------------------------- composition and publication

// A run of rows of the lane's two channels: h -> a h + h0 per channel; a = -0 marks a beginning.
struct Run {
  float2 a, h;
};

__device__ __forceinline__ float apply(float a, float h, float before) {
  return signbit(a) ? h : fmaf(a, before, h);
}
__device__ __forceinline__ float2 apply(const Run& r, float2 before) {
  return make_float2(apply(r.a.x, r.h.x, before.x), apply(r.a.y, r.h.y, before.y));
}
// `first`, then `then`.
__device__ __forceinline__ Run compose(const Run& first, const Run& then) {
  Run q;
  q.h = apply(then, first.h);
  q.a.x = signbit(then.a.x) ? -0.f : first.a.x * then.a.x;
  q.a.y = signbit(then.a.y) ? -0.f : first.a.y * then.a.y;
  return q;
}

constexpr unsigned long long kUnset = ~0ull;

__device__ __forceinline__ unsigned long long word_of(float lo, float hi) {
  return static_cast<unsigned long long>(__float_as_uint(lo)) |
         static_cast<unsigned long long>(__float_as_uint(hi)) << 32;
}
__device__ __forceinline__ void publish_run(float2* at, const Run& r) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(at), "l"(word_of(r.a.x, r.h.x)),
               "l"(word_of(r.a.y, r.h.y))
               : "memory");
}
__device__ __forceinline__ unsigned ready_bits(float v) {
  const unsigned u = __float_as_uint(v);
  return u == ~0u ? 0x7FFFFFFFu : u;  // a NaN that looks unset becomes another NaN
}
__device__ __forceinline__ void publish_state(float* at, float2 h) {
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
  Run r;
  r.a = make_float2(__uint_as_float(static_cast<unsigned>(u)), __uint_as_float(static_cast<unsigned>(v)));
  r.h = make_float2(__uint_as_float(static_cast<unsigned>(u >> 32)), __uint_as_float(static_cast<unsigned>(v >> 32)));
  return r;
}

__device__ __forceinline__ float2 await_state(const float* at, int* ticket, int* dev_error) {
  unsigned u, v;
  uint64_t t0 = 0;
  for (unsigned i = 0;; ++i) {
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(u), "=r"(v) : "l"(at) : "memory");
    if (u != ~0u && v != ~0u) break;
    if (i == 0) t0 = lap::globaltimer_ns();
    if ((i & 15u) == 15u && !keep_polling(ticket, dev_error, t0)) break;
  }
  return make_float2(__uint_as_float(u), __uint_as_float(v));
}

struct ScanSmem {
  Run own[kWarps][32];     // each warp's rows
  Run earlier[kWarps][32]; // pieces of the group's earlier tiles, in order
  float2 base[32];         // the state before the group
  int ticket, fresh;       // fresh: the tile's first row begins a sequence
};

// The state before this warp's rows.  `mine` is the composition of the warp's rows; t the tile in
// walking order.  Publishes the tile for those that follow.
template <typename E>
__device__ __forceinline__ float2 state_before(const Params<E>& p, ScanSmem& sm, const Run& mine, const Rows& rows,
                                               int t, int column, int warp, int lane) {
  sm.own[warp][lane] = mine;
  if (warp == 0 && lane == 0) sm.fresh = rows.begin & 1u;
  __syncthreads();
  float2 before = make_float2(0.f, 0.f);
  if (p.ticket) {
    const size_t width = static_cast<size_t>(p.columns) * kCols;
    const size_t at = static_cast<size_t>(column) * kCols + 2 * lane;
    const int group = t / p.group, j = t - group * p.group;
    const bool last = j == p.group - 1;
    Run whole;
    if (warp == 0) {
      whole = mine;
#pragma unroll 1
      for (int w = 1; w < kWarps; ++w) whole = compose(whole, sm.own[w][lane]);
      if (!last) publish_run(p.runs + t * width + at, whole);
    }
    if (!sm.fresh) {
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
  for (int w = 0; w < warp; ++w) before = apply(sm.own[w][lane], before);
  return before;
}

// The tile this block takes: its number in walking order and its channels; false when none is left.
template <typename E>
__device__ __forceinline__ bool take_tile(const Params<E>& p, ScanSmem& sm, int* t, int* column) {
  int id = static_cast<int>(blockIdx.x);
  if (p.ticket) {
    if (threadIdx.x == 0) sm.ticket = atomicAdd(p.ticket, 1);
    __syncthreads();
    id = sm.ticket;
  }
  *t = id / p.columns;
  *column = id - *t * p.columns;
  return *t < p.tiles;
}

// The final states of the empty sequences that lie in this tile: their initial ones.
template <typename E, bool kPair>
__device__ __forceinline__ void empty_sequences(const Params<E>& p, int tile, const Lane<kPair>& l, int warp) {
  if (!p.finish || (!p.cu_seqlens && p.T > 0)) return;
  const int lo = p.cu_seqlens ? p.first_seq[tile] : 0, hi = p.cu_seqlens ? p.first_seq[tile + 1] : p.N;
  for (int n = lo + warp; n < hi; n += kWarps) {
    if (p.cu_seqlens && p.cu_seqlens[n] != p.cu_seqlens[n + 1]) continue;
    const int slot = slot_of(p, n);
    if (slot >= 0) store_state(p.finish, slot, p.C, l, load_state(p.start, slot, p.C, l));
  }
}

// ---------------------------------------------------------------- the forward scan

template <typename E, bool kPair>
__global__ void __launch_bounds__(kScanThreads, 2) gated_scan_fwd_kernel(const __grid_constant__ Params<E> p) {
  constexpr int K = rows_per_warp<E, false>();
  constexpr bool kPrecise = sizeof(E) == 4;
  __shared__ ScanSmem sm;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  int t, column;
  if (!take_tile(p, sm, &t, &column)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Lane<kPair> l(column, lane, p.C);
  const Rows rows = rows_of<E, false, K>(p, t, warp, lane);
  const int64_t row0 = static_cast<int64_t>(t) * p.stride + warp * K;

  Raw<E> x[K], r[K], g[K];
  {
    const E *px = p.x + row0 * p.ldx, *pr = p.r + row0 * p.ldr, *pg = p.g + row0 * p.ldg;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = r[k] = g[k] = Raw<E>{};
      if (rows.live >> k & 1u) {
        r[k] = load2(pr + k * p.ldr, l);
        g[k] = load2(pg + k * p.ldg, l);
        x[k] = load2(px + k * p.ldx, l);
      }
    }
  }
  const float2 slope = load_state(p.slopes, 0, p.C, l);
  float2 a[K], b[K];
  Run run{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float2 vr = r[k].get(), vg = g[k].get(), vx = x[k].get();
    const Decay d0 = decay_of<kPrecise>(slope.x * sigmoid<kPrecise>(vr.x));
    const Decay d1 = decay_of<kPrecise>(slope.y * sigmoid<kPrecise>(vr.y));
    a[k] = make_float2(d0.lambda, d1.lambda);
    b[k] = make_float2(d0.beta * sigmoid<kPrecise>(vg.x) * vx.x, d1.beta * sigmoid<kPrecise>(vg.y) * vx.y);
    if (rows.begin >> k & 1u) {
      const float2 h = load_state(p.start, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l);
      b[k].x = fmaf(a[k].x, h.x, b[k].x);
      b[k].y = fmaf(a[k].y, h.y, b[k].y);
      run.a = make_float2(-0.f, -0.f);
      run.h = make_float2(0.f, 0.f);
    }
    run.a.x *= a[k].x;
    run.a.y *= a[k].y;
    const bool begin = rows.begin >> k & 1u;
    run.h.x = begin ? b[k].x : fmaf(a[k].x, run.h.x, b[k].x);
    run.h.y = begin ? b[k].y : fmaf(a[k].y, run.h.y, b[k].y);
  }
  float2 h = state_before(p, sm, run, rows, t, column, warp, lane);
  E* po = p.o + row0 * p.ldo;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const bool begin = rows.begin >> k & 1u;
    h.x = begin ? b[k].x : fmaf(a[k].x, h.x, b[k].x);
    h.y = begin ? b[k].y : fmaf(a[k].y, h.y, b[k].y);
    if (rows.live >> k & 1u) store2(po + k * p.ldo, l, h.x, h.y);
    if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l, h);
  }
  empty_sequences(p, t, l, warp);
}

// ---------------------------------------------------------------- the gradients' scan

template <typename E, bool kPair>
__global__ void __launch_bounds__(kScanThreads, 1) gated_scan_bwd_kernel(const __grid_constant__ Params<E> p) {
  constexpr int K = rows_per_warp<E, true>();
  constexpr bool kPrecise = sizeof(E) == 4;
  __shared__ ScanSmem sm;
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  int t, column;
  if (!take_tile(p, sm, &t, &column)) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Lane<kPair> l(column, lane, p.C);
  const int tile = p.tiles - 1 - t;
  const Rows rows = rows_of<E, true, K>(p, tile, warp, lane);
  const int64_t row0 = static_cast<int64_t>(tile + 1) * p.stride - 1 - warp * K;  // row k is row0 - k

  Raw<E> x[K], r[K], g[K], before[K], dout[K];
  {
    const E *px = p.x + row0 * p.ldx, *pr = p.r + row0 * p.ldr, *pg = p.g + row0 * p.ldg;
    const E *po = p.o_in + (row0 - 1) * p.ldo, *pd = p.dout + row0 * p.lddout;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = r[k] = g[k] = before[k] = dout[k] = Raw<E>{};
      if (rows.live >> k & 1u) {
        r[k] = load2(pr - k * p.ldr, l);
        dout[k] = load2(pd - k * p.lddout, l);
        x[k] = load2(px - k * p.ldx, l);
        g[k] = load2(pg - k * p.ldg, l);
        if (!(rows.end >> k & 1u)) before[k] = load2(po - k * p.ldo, l);
      }
    }
  }
  const float2 slope = load_state(p.slopes, 0, p.C, l);
  Run run{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float2 vr = r[k].get();
    float2 vd = dout[k].get();
    const float a0 = decay_of<kPrecise>(slope.x * sigmoid<kPrecise>(vr.x)).lambda;
    const float a1 = decay_of<kPrecise>(slope.y * sigmoid<kPrecise>(vr.y)).lambda;
    if (rows.begin >> k & 1u) {
      const float2 h = load_state(p.start, __shfl_sync(0xFFFFFFFFu, rows.slot, k), p.C, l);
      run.a = make_float2(-0.f, -0.f);
      run.h = h;
    }
    run.a.x *= a0;
    run.a.y *= a1;
    run.h.x = a0 * (vd.x + run.h.x);
    run.h.y = a1 * (vd.y + run.h.y);
  }
  float2 w = state_before(p, sm, run, rows, t, column, warp, lane);
  float2 ds = make_float2(0.f, 0.f);
  E *px = p.dx + row0 * p.lddx, *pr = p.dr + row0 * p.lddr, *pg = p.dg + row0 * p.lddg;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!(rows.live >> k & 1u)) continue;
    const float2 vx = x[k].get(), vr = r[k].get(), vg = g[k].get(), vd = dout[k].get();
    float2 vb = before[k].get();
    const int slot = __shfl_sync(0xFFFFFFFFu, rows.slot, k);
    if (rows.begin >> k & 1u) w = load_state(p.start, slot, p.C, l);
    if (rows.end >> k & 1u) vb = load_state(p.h0, slot, p.C, l);
    const float2 G = make_float2(vd.x + w.x, vd.y + w.y);
    const Grads d0 = grads_of<kPrecise>(vx.x, vr.x, vg.x, slope.x, G.x, vb.x);
    const Grads d1 = grads_of<kPrecise>(vx.y, vr.y, vg.y, slope.y, G.y, vb.y);
    store2(px - k * p.lddx, l, d0.dx, d1.dx);
    store2(pr - k * p.lddr, l, d0.dr, d1.dr);
    store2(pg - k * p.lddg, l, d0.dg, d1.dg);
    ds.x += d0.ds;
    ds.y += d1.ds;
    w = make_float2(d0.lambda * G.x, d1.lambda * G.y);
    if (p.finish && (rows.end >> k & 1u)) store_state(p.finish, slot, p.C, l, w);
  }
  // the tile's terms of dslopes, warps in order
  __syncthreads();
  sm.own[warp][lane].h = ds;
  __syncthreads();
  if (warp == 0) {
#pragma unroll 1
    for (int i = 1; i < kWarps; ++i) {
      ds.x += sm.own[i][lane].h.x;
      ds.y += sm.own[i][lane].h.y;
    }
    store_state(p.part, tile, p.C, l, ds);
  }
  empty_sequences(p, tile, l, warp);
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
  constexpr bool kPrecise = sizeof(E) == 4;
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
    const float x = to_f32(p.x[t * p.ldx + c]);
    const Decay d = decay_of<kPrecise>(slope * sigmoid<kPrecise>(to_f32(p.r[t * p.ldr + c])));
    h = fmaf(d.lambda, h, d.beta * sigmoid<kPrecise>(to_f32(p.g[t * p.ldg + c])) * x);
    if (p.o) p.o[t * p.ldo + c] = from_f32<E>(h);
  }
  if (p.finish) p.finish[at] = h;
}

}  // namespace lag
