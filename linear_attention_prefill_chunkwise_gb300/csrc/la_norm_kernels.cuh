// la_norm_kernels.cuh -- kernels of the root-mean-square norm (include/la_norm.h).
//
// A row is shared out among `share` threads, from eight up to a whole block (a block of narrow rows
// takes several at once).  Its sum of squares and, for the 8-bit output, its largest |y| are reduced
// over those threads; every input is read once and every output written once, and the work is bound
// by those bytes.
//
// Two forms.  The direct kernels load a row into registers; many small blocks keep the memory busy.
// The ring kernels (gradients, which keep sums over rows, and the 8-bit output, whose two
// reductions follow one another) are persistent: a ring of stages in shared memory is filled by
// bulk copies, one per row and input, as many turns ahead as there are stages, so that the copies
// of the next rows run while a row is reduced and written.  A bulk copy moves whole 16-byte chunks;
// a row that begins or ends inside one is read from its own offset in the stage, so any row stride
// and alignment takes the same path.
// Measured, of the bytes at the copy rate: forward with a residual 16384 x 8192 BF16 169 us (0.94),
// FP32 8192 x 8192 155 (1.02), 2^20 x 128 BF16 158 (1.0), 128 x 8192 3.7 (0.34: launch and latency);
// 8-bit output 16384 x 8192 145 (0.95); gradients with dres 16384 x 4096 91 (0.87), 16384 x 8192 175
// (0.90), 4099 x 1001 18 (0.2: element by element, where rows are not 16-byte aligned).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "la_vec.cuh"
#include "sm103_ptx.cuh"

namespace lan {

constexpr int kGroup = 128;       // columns per scale of the grouped 8-bit output
constexpr int kMaxThreads = 512;
constexpr int kMaxColumns = 16384;
constexpr int kMaxStages = 8;

template <typename E>
struct FwdParams {
  const E *x, *res;
  E *y, *res_out;
  uint8_t* y8;
  float* scales;
  const float* weight;
  int64_t ldx, ldres, ldy, ldres_out;
  int* dev_error;
  float eps;
  int rows, C, group, share;
};

template <typename E>
struct BwdParams {
  const E *s, *dy, *dres;
  E* dx;
  const float* weight;
  float* part;  // [blocks, C] sums of each block's rows
  int64_t lds, lddy, lddres, lddx;
  int* dev_error;
  float eps;
  int rows, C, share;
};

// e4m3, rounded to nearest even, finite values clamped to +-448.
template <int kVec>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[kVec / 4];
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    if constexpr (kVec == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}
// kVec weights (4-byte aligned, so wide loads only where the pointer allows them).
template <int kVec>
__device__ __forceinline__ void load_weight(const float* p, float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    v[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p) + i);
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  }
}

// Sum (maximum) of kN values each over the `share` threads of a row, in a fixed order, returned to
// all of them.  `share` is a power of two; every thread of the block calls it.  Each call of a turn
// uses its own smem, so that one barrier each is enough.
template <bool kMax, int kN>
__device__ __forceinline__ void warp_reduce(float (&v)[kN], int lanes) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < lanes)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
        v[i] = kMax ? fmaxf(v[i], o) : v[i] + o;
      }
}
template <bool kMax, int kN>
__device__ __forceinline__ void reduce(float (&v)[kN], float (*smem)[kN], int share) {
  warp_reduce<kMax>(v, share);
  if (share <= 32) return;
  const int warp = threadIdx.x / 32, warps = share / 32, first = warp / warps * warps;
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int i = 0; i < kN; ++i) smem[warp][i] = v[i];
  __syncthreads();
  // the row's warps' values, one per lane (in turn, again and again), and the same tree
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = smem[first + threadIdx.x % 32 % warps][i];
  warp_reduce<kMax>(v, warps);
}

// Group maxima of |y| where a group of 128 columns lies with several warps or loads: by shared
// memory (bits of non-negative floats order as integers do).
__device__ __forceinline__ void raise(int* top, float v) { atomicMax(top, __float_as_int(v)); }

// The 8-bit output of a row's y (in s), with its scales.  Called by every thread of the block.
template <int kVec, int kLoads>
__device__ __forceinline__ void write_e4m3(float (&s)[kLoads][kVec], uint8_t* out, float* scales, int C, int group,
                                           int share, int tid, int sub, bool live, float (*tops)[1], int* groups) {
  if (group == 0) {
    float top[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e) top[0] = fmaxf(top[0], fabsf(s[i][e]));
    reduce<true>(top, tops, share);
    const float m = fmaxf(top[0], 0x1p-40f), inv = 448.f / m;
    if (live && tid == 0) *scales = m / 448.f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * share + tid) * kVec;
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] *= inv;
      if (live && c < C) store_e4m3<kVec>(out + c, s[i]);
    }
    return;
  }
  const int count = (C + kGroup - 1) / kGroup;
  int* mine = groups + sub * count;
  if constexpr (kVec == 1) {
    for (int k = tid; k < count; k += share) mine[k] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = i * share + tid;
      if (c < C) raise(mine + c / kGroup, fmaxf(fabsf(s[i][0]), 0.f));
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * share + tid) * kVec;
    float m[1] = {0.f};
    if constexpr (kVec == 1) {
      if (c < C) m[0] = __int_as_float(mine[c / kGroup]);
    } else {  // kGroup / kVec neighbouring lanes hold one group
#pragma unroll
      for (int e = 0; e < kVec; ++e) m[0] = fmaxf(m[0], fabsf(s[i][e]));
      warp_reduce<true>(m, min(share, kGroup / kVec));
    }
    const float top = fmaxf(m[0], 0x1p-40f), inv = 448.f / top;
    if (live && c < C) {
      if (c % kGroup == 0) scales[c / kGroup] = top / 448.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] *= inv;
      store_e4m3<kVec>(out + c, s[i]);
    }
  }
}

// kLoads loads of kVec elements per thread (8, 16 or 32 elements); C <= kLoads * kVec * share.
template <typename E, bool kFp8, int kVec, int kLoads>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const FwdParams<E> p) {
  __shared__ float sums[kMaxThreads / 32][1], tops[kMaxThreads / 32][1];
  __shared__ int groups[kFp8 && kVec == 1 ? kMaxColumns / kGroup : 1];  // of a block's rows together
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  const int tid = threadIdx.x % p.share, sub = threadIdx.x / p.share;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.share) + sub;
  const bool live = row < p.rows;
  float s[kLoads][kVec];
  float ss[1] = {0.f};
  const E* x = p.x + row * p.ldx;
  const E* res = p.res ? p.res + row * p.ldres : nullptr;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * p.share + tid) * kVec;
    if (live && c < p.C) {
      load<kVec>(x + c, s[i]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] = 0.f;
    }
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec;
      if (live && c < p.C) {
        float r[kVec];
        load<kVec>(res + c, r);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s[i][e] += r[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
#pragma unroll
    for (int e = 0; e < kVec; ++e) ss[0] = fmaf(s[i][e], s[i][e], ss[0]);
  reduce<false>(ss, sums, p.share);
  const float rstd = rsqrtf(ss[0] / static_cast<float>(p.C) + p.eps);
  if (p.res_out && live) {
    E* out = p.res_out + row * p.ldres_out;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec;
      if (c < p.C) store<kVec>(out + c, s[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * p.share + tid) * kVec;
    if (c < p.C) {  // beyond it s is 0
      float w[kVec];
      load_weight<kVec>(p.weight + c, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] *= rstd * w[e];
    }
  }
  if constexpr (kFp8) {
    const int count = p.group ? (p.C + kGroup - 1) / kGroup : 1;
    write_e4m3<kVec, kLoads>(s, p.y8 + row * p.ldy, p.scales + row * count, p.C, p.group, p.share, tid, sub, live, tops,
                             groups);
  } else {
    E* out = p.y + row * p.ldy;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec;
      if (live && c < p.C) store<kVec>(out + c, s[i]);
    }
  }
}

// ---------------------------------------------------------------- the ring

// Bytes of a row in a stage: whole chunks wherever the row begins in its first one.
template <typename E>
__host__ __device__ constexpr int row_pitch(int C) { return (C * static_cast<int>(sizeof(E)) + 15) / 16 * 16 + 16; }

// One row of a matrix into shared memory at `dst` (its first element at dst + (address mod 16)),
// by one thread: whole chunks by a bulk copy, and what begins or ends inside a chunk at the
// matrix's own ends (beyond them nothing is read) element by element.  Arrives on `bar`.
template <typename E>
__device__ __forceinline__ void fetch_row(char* dst, const E* matrix, int64_t ld, int64_t row, int rows, int C,
                                          uint64_t* bar) {
  const char* begin = reinterpret_cast<const char*>(matrix);
  const char* end = begin + ((rows - 1) * ld + C) * static_cast<int64_t>(sizeof(E));
  const char* src = begin + row * ld * static_cast<int64_t>(sizeof(E));
  const char* stop = src + C * sizeof(E);
  const char* lo = src - (reinterpret_cast<uintptr_t>(src) & 15u);
  const char* origin = lo;
  const char* hi = stop + (-reinterpret_cast<uintptr_t>(stop) & 15u);
  if (lo < begin) lo += 16;
  if (hi > end) hi -= 16;
  const uint32_t bytes = hi > lo ? static_cast<uint32_t>(hi - lo) : 0u;
  for (const char* e = src; e < lo && e < stop; e += sizeof(E))
    *reinterpret_cast<E*>(dst + (e - origin)) = *reinterpret_cast<const E*>(e);
  const char* tail = lo > src ? lo : src;
  for (const char* e = hi > tail ? hi : tail; e < stop; e += sizeof(E))
    *reinterpret_cast<E*>(dst + (e - origin)) = *reinterpret_cast<const E*>(e);
  if (bytes) {
    lap::mbar_arrive_expect_tx(bar, bytes);
    lap::bulk_copy_g2s(dst + (lo - origin), lo, bytes, bar);
  } else {
    lap::mbar_arrive(bar);
  }
}

template <typename E>
__device__ __forceinline__ int row_offset(const E* matrix, int64_t ld, int64_t row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(matrix + row * ld) & 15u);
}

// The ring of a persistent block: turn t is rows (blockIdx.x + t gridDim.x) at_once .. + at_once - 1,
// in stage t mod stages.  kInputs matrices (null ones are not loaded).
template <typename E, int kInputs>
struct Ring {
  const E* in[kInputs];
  int64_t ld[kInputs];
  char* stage0;
  uint64_t* bar;
  int pitch, at_once, stages, rows, C;

  __device__ __forceinline__ int64_t first_row(int turn) const {
    return (static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(turn) * gridDim.x) * at_once;
  }
  __device__ __forceinline__ char* at(int turn, int i, int sub) const {
    return stage0 + (static_cast<size_t>(turn % stages * kInputs + i) * at_once + sub) * pitch;
  }
  __device__ __forceinline__ void init() const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) lap::mbar_init(bar + s, kInputs * at_once);
      lap::fence_mbar_init();
    }
  }
  // Starts a turn's copies: one thread per row and input.
  __device__ __forceinline__ void load(int turn) const {
    const int64_t row0 = first_row(turn);
    if (row0 >= rows) return;
    for (int k = threadIdx.x; k < kInputs * at_once; k += blockDim.x) {
      const int i = k / at_once, sub = k - i * at_once;
      uint64_t* b = bar + turn % stages;
      const E* m = in[0];
      int64_t l = ld[0];
#pragma unroll
      for (int j = 1; j < kInputs; ++j)
        if (i == j) m = in[j], l = ld[j];
      if (m && row0 + sub < rows) fetch_row(at(turn, i, sub), m, l, row0 + sub, rows, C, b);
      else lap::mbar_arrive(b);
    }
  }
  // A copy did not arrive in time: says so, and outlives the copies in flight.
  __device__ __forceinline__ void give_up(int turn, int* dev_error) const {
    if (threadIdx.x != 0) return;
    if (dev_error) atomicOr(reinterpret_cast<unsigned*>(dev_error), 4u);  // LA_DEV_ERR_TIMEOUT
    for (int t = turn; t < turn + stages - 1 && first_row(t) < rows; ++t)
      lap::mbar_wait_drain(bar + t % stages, t / stages & 1);
  }
};

// kVec elements of a row in a stage.
template <int kVec, typename E>
__device__ __forceinline__ void stage_load(const char* row, int c, float (&v)[kVec]) {
  load<kVec>(reinterpret_cast<const E*>(row) + c, v);
}

// The forward with an 8-bit output.
template <typename E, int kVec, int kLoads>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_ring_kernel(const FwdParams<E> p, int stages) {
  __shared__ float sums[2][kMaxThreads / 32][1], tops[2][kMaxThreads / 32][1];
  __shared__ int groups[kVec == 1 ? kMaxColumns / kGroup : 1];
  __shared__ uint64_t bar[kMaxStages];
  __shared__ int abort;
  extern __shared__ __align__(128) char shared[];
  const int tid = threadIdx.x % p.share, sub = threadIdx.x / p.share, at_once = blockDim.x / p.share;
  const Ring<E, 2> ring{{p.x, p.res}, {p.ldx, p.ldres}, shared, bar, row_pitch<E>(p.C), at_once, stages, p.rows, p.C};
  if (threadIdx.x == 0) abort = 0;
  ring.init();
  __syncthreads();
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  for (int t = 0; t < stages - 1; ++t) ring.load(t);
  float w[kLoads][kVec];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * p.share + tid) * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[i][e] = 0.f;
    if (c < p.C) load_weight<kVec>(p.weight + c, w[i]);
  }
  for (int turn = 0;; ++turn) {
    const int64_t row0 = ring.first_row(turn), row = row0 + sub;
    if (row0 >= p.rows) break;
    const bool live = row < p.rows;
    const bool here = lap::mbar_wait(bar + turn % stages, turn / stages & 1, &abort);
    // everyone has left the turn before: its stage takes the turn stages - 1 ahead
    if (__syncthreads_or(!here)) {
      ring.give_up(turn, p.dev_error);
      break;
    }
    ring.load(turn + stages - 1);
    float s[kLoads][kVec];
    float ss[1] = {0.f};
    const char* x = ring.at(turn, 0, sub) + row_offset(p.x, p.ldx, row);
    const char* res = ring.at(turn, 1, sub) + (p.res ? row_offset(p.res, p.ldres, row) : 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec;
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] = 0.f;
      if (live && c < p.C) {
        stage_load<kVec, E>(x, c, s[i]);
        if (p.res) {
          float r[kVec];
          stage_load<kVec, E>(res, c, r);
#pragma unroll
          for (int e = 0; e < kVec; ++e) s[i][e] += r[e];
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) ss[0] = fmaf(s[i][e], s[i][e], ss[0]);
      }
    }
    if (p.res_out && live) {
      E* out = p.res_out + row * p.ldres_out;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int c = (i * p.share + tid) * kVec;
        if (c < p.C) store<kVec>(out + c, s[i]);
      }
    }
    reduce<false>(ss, sums[turn & 1], p.share);
    const float rstd = rsqrtf(ss[0] / static_cast<float>(p.C) + p.eps);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[i][e] *= rstd * w[i][e];
    const int count = p.group ? (p.C + kGroup - 1) / kGroup : 1;
    write_e4m3<kVec, kLoads>(s, p.y8 + row * p.ldy, p.scales + row * count, p.C, p.group, p.share, tid, sub, live,
                             tops[turn & 1], groups);
  }
}

// ---------------------------------------------------------------- gradients

// A block's sums of dy n over its rows, one row of p.part: where it takes several rows at once,
// their sums are added in order through `add` [rows at once, C].
template <int kVec, int kLoads, typename E>
__device__ __forceinline__ void write_part(const BwdParams<E>& p, const float (&dw)[kLoads][kVec], float* add, int tid,
                                           int sub, int at_once) {
  float* part = p.part + static_cast<size_t>(blockIdx.x) * p.C;
  float* to = at_once == 1 ? part : add + sub * p.C;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * p.share + tid) * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (c < p.C) to[c + e] = dw[i][e];
  }
  if (at_once == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
    float t = add[c];
    for (int k = 1; k < at_once; ++k) t += add[k * p.C + c];
    part[c] = t;
  }
}

// Blocks walk rows; each thread keeps its columns' sums of dy n over its rows in registers.  A
// block's sums go to `part`, whose rows are then added in order.  kRing: rows come through the
// ring, and s and dy are read from it twice; else they are held in registers.
template <typename E, bool kRing, int kVec, int kLoads>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const BwdParams<E> p, int stages) {
  __shared__ float sums[2][kMaxThreads / 32][2];
  __shared__ uint64_t bar[kMaxStages];
  __shared__ int abort;
  extern __shared__ __align__(128) char shared[];
  const int tid = threadIdx.x % p.share, sub = threadIdx.x / p.share, at_once = blockDim.x / p.share;
  const Ring<E, 3> ring{{p.s, p.dy, p.dres}, {p.lds, p.lddy, p.lddres}, shared, bar, row_pitch<E>(p.C), at_once, stages,
                        p.rows, p.C};
  if constexpr (kRing) {
    if (threadIdx.x == 0) abort = 0;
    ring.init();
    __syncthreads();
  }
  lap::griddep_wait();
  lap::griddep_launch_dependents();
  if constexpr (kRing)
    for (int t = 0; t < stages - 1; ++t) ring.load(t);
  float dw[kLoads][kVec], w[kRing ? kLoads : 1][kVec];  // the weights, or those of one load
  auto weights = [&](int i) -> const float (&)[kVec] {
    if constexpr (!kRing) {
      const int c = (i * p.share + tid) * kVec;
      if (c < p.C) load_weight<kVec>(p.weight + c, w[0]);
    }
    return w[kRing ? i : 0];
  };
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = (i * p.share + tid) * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) dw[i][e] = w[kRing ? i : 0][e] = 0.f;
    if (kRing && c < p.C) load_weight<kVec>(p.weight + c, w[i]);
  }
  for (int turn = 0;; ++turn) {
    const int64_t row0 = ring.first_row(turn), row = row0 + sub;
    if (row0 >= p.rows) break;
    const bool live = row < p.rows;
    const char *at_s = nullptr, *at_dy = nullptr, *at_dres = nullptr;
    if constexpr (kRing) {
      const bool here = lap::mbar_wait(bar + turn % stages, turn / stages & 1, &abort);
      // everyone has left the turn before: its stage takes the turn stages - 1 ahead
      if (__syncthreads_or(!here)) {
        ring.give_up(turn, p.dev_error);
        break;
      }
      ring.load(turn + stages - 1);
      at_s = ring.at(turn, 0, sub) + row_offset(p.s, p.lds, row);
      at_dy = ring.at(turn, 1, sub) + row_offset(p.dy, p.lddy, row);
      at_dres = ring.at(turn, 2, sub) + (p.dres ? row_offset(p.dres, p.lddres, row) : 0);
    }
    float s[kRing ? 1 : kLoads][kVec], dy[kRing ? 1 : kLoads][kVec];
    float r[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec, k = kRing ? 0 : i;
#pragma unroll
      for (int e = 0; e < kVec; ++e) s[k][e] = dy[k][e] = 0.f;
      if (live && c < p.C) {
        if constexpr (kRing) {
          stage_load<kVec, E>(at_s, c, s[0]);
          stage_load<kVec, E>(at_dy, c, dy[0]);
        } else {
          load<kVec>(p.s + row * p.lds + c, s[k]);
          load<kVec>(p.dy + row * p.lddy + c, dy[k]);
        }
      }
      if constexpr (kRing) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          r[0] = fmaf(s[0][e], s[0][e], r[0]);
          r[1] = fmaf(dy[0][e] * weights(i)[e], s[0][e], r[1]);
        }
      }
    }
    if constexpr (!kRing) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const float(&v)[kVec] = weights(i);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          r[0] = fmaf(s[i][e], s[i][e], r[0]);
          r[1] = fmaf(dy[i][e] * v[e], s[i][e], r[1]);
        }
      }
    }
    reduce<false>(r, sums[turn & 1], p.share);
    const float rstd = rsqrtf(r[0] / static_cast<float>(p.C) + p.eps);
    const float m = r[1] * rstd / static_cast<float>(p.C);  // mean(w dy n)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int c = (i * p.share + tid) * kVec, k = kRing ? 0 : i;
      if (live && c < p.C) {
        float extra[kVec], out[kVec];
        const float(&v)[kVec] = weights(i);
        if constexpr (kRing) {
          stage_load<kVec, E>(at_s, c, s[0]);
          stage_load<kVec, E>(at_dy, c, dy[0]);
          if (p.dres) stage_load<kVec, E>(at_dres, c, extra);
        } else {
          if (p.dres) load<kVec>(p.dres + row * p.lddres + c, extra);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float n = s[k][e] * rstd;
          out[e] = rstd * (v[e] * dy[k][e] - n * m);
          if (p.dres) out[e] += extra[e];
          dw[i][e] = fmaf(dy[k][e], n, dw[i][e]);
        }
        store<kVec>(p.dx + row * p.lddx + c, out);
      }
    }
  }
  __syncthreads();  // the ring's memory is free
  write_part(p, dw, reinterpret_cast<float*>(shared), tid, sub, at_once);
}

// out[c] = sum over rows of part[rows][C] (0 rows: 0): 32 channels a block, each warp every 32nd
// row, the warps' sums in order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int rows, int C, float* out) {
  __shared__ float sums[32][33];
  lap::griddep_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < C) {
#pragma unroll 8
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

}  // namespace lan
