// la_gated_api.cu -- host side of the C ABI declared in include/la_gated.h: argument validation,
// the workspace layout and the launches.  Nothing here allocates device memory, reads device
// memory or synchronises with the host.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/la_gated.h"
#include "la_gated_kernels.cuh"
#include "la_host_common.h"
#include "la_rows_common.h"

namespace {

using la_host::fail;
using la_host::RowSpan;

la_host::DeviceState g_dev[la_host::kMaxDevices];

// How a scan is cut, and its device workspace: the ticket, the sequences of each tile (packed),
// the published runs and states, and for the gradients one row of partial sums of dslopes per tile.
struct Plan {
  int tiles = 0, columns = 0, stride = 0, group = 0;
  bool waits = false;  // tickets and published states are needed
  size_t first_seq = 0, runs = 0, words = 0, before = 0, part = 0, bytes = 0;
};

// Tiles of a group: each composes half a group of published runs on average, and a scan is a
// chain of one step per group.
constexpr int kGroup = 16;

Plan plan_of(int B, int T, int N, int C, bool packed, la_dtype dtype, bool backward) {
  Plan q;
  if (N == 0) return q;
  const int most = dtype == LA_DTYPE_BF16
                       ? (backward ? lag::tile_rows<__nv_bfloat16, true>() : lag::tile_rows<__nv_bfloat16, false>())
                       : (backward ? lag::tile_rows<float, true>() : lag::tile_rows<float, false>());
  const int64_t rows = static_cast<int64_t>(B) * T;
  // short sequences of one length: tiles of whole sequences wait for nothing
  const bool whole = !packed && T > 0 && T <= most;
  q.stride = whole ? most / T * T : most;
  q.waits = !whole;
  q.tiles = static_cast<int>((rows + q.stride - 1) / q.stride);
  if (q.tiles == 0) q.tiles = 1;  // empty sequences alone
  q.columns = (C + lag::kCols - 1) / lag::kCols;
  q.group = kGroup;
  if (q.waits) {
    const size_t width = static_cast<size_t>(q.columns) * lag::kCols;
    const size_t groups = (q.tiles + q.group - 1) / q.group;
    q.first_seq = 256;
    q.runs = q.first_seq + (packed ? la_host::align256((static_cast<size_t>(q.tiles) + 1) * 4) : 0);
    q.before = q.runs + q.tiles * width * 8;
    q.words = q.tiles * width * 2 + groups * width;
    q.bytes = q.runs + q.words * 4;
  }
  q.part = q.bytes;
  if (backward) q.bytes += la_host::align256(static_cast<size_t>(q.tiles) * C * 4);
  return q;
}

la_status check_sizes(int B, int T, int N, int C, bool packed, la_dtype dtype) {
  if (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32) return fail(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (C < 1) return fail(LA_ERR_INVALID_ARGUMENT, "C must be >= 1 (got %d)", C);
  if (B < 0 || T < 0 || N < 0) return fail(LA_ERR_INVALID_ARGUMENT, "B, T, N must be >= 0");
  if (packed) {
    if (B != 1) return fail(LA_ERR_INVALID_ARGUMENT, "packed mode (cu_seqlens given) needs B == 1 (got %d)", B);
  } else if (N != B) {
    return fail(LA_ERR_INVALID_ARGUMENT, "fixed-length mode needs N == B (got N=%d, B=%d)", N, B);
  }
  if (static_cast<int64_t>(B) * T > la_host::kMaxRows)
    return fail(LA_ERR_UNSUPPORTED, "B*T too large (%lld)", (long long)B * T);
  // tiles of at least 32 rows and 64 channels, numbered below 2^30 (more than any memory holds)
  if ((static_cast<int64_t>(B) * T / 32 + 1) * ((C + 63) / 64) >= int64_t(1) << 30)
    return fail(LA_ERR_UNSUPPORTED, "B*T*C too large");
  if (static_cast<int64_t>(N) * ((C + 63) / 64) > INT32_MAX) return fail(LA_ERR_UNSUPPORTED, "N*C too large");
  return LA_OK;
}

// Checks of the state pool and the per-sequence arrays; `states` = some state buffer is given.
la_status check_pool(bool states, const int32_t* state_indices, int pool_size, int N) {
  if (!states) return LA_OK;
  if (state_indices) {
    if (pool_size <= 0) return fail(LA_ERR_INVALID_ARGUMENT, "pool_size must be positive with state_indices");
  } else if (pool_size < N) {
    return fail(LA_ERR_INVALID_ARGUMENT, "pool_size (%d) must be >= N (%d) without state_indices", pool_size, N);
  }
  return LA_OK;
}

// A pool as an address range: P slots with state_indices, else one per sequence.
RowSpan pool_span(const void* p, const char* name, const int32_t* state_indices, int pool_size, int N, int C) {
  return la_host::flat(p, static_cast<uint64_t>(state_indices ? pool_size : N) * C * 4, name);
}

la_status device(la_host::DeviceState** ds) {
  return la_host::current_device(g_dev, ds, [] { return cudaSuccess; });
}

template <typename E>
void set_plan(lag::Params<E>* p, const Plan& q, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  p->tiles = q.tiles;
  p->columns = q.columns;
  p->stride = q.stride;
  p->group = q.group;
  if (q.waits) {
    p->ticket = reinterpret_cast<int*>(ws);
    p->first_seq = reinterpret_cast<int32_t*>(ws + q.first_seq);
    p->runs = reinterpret_cast<float2*>(ws + q.runs);
    p->before = reinterpret_cast<float*>(ws + q.before);
  }
  p->part = reinterpret_cast<float*>(ws + q.part);
}

// Whether a lane may load two neighbouring elements at once from rows of this stride.
template <typename E>
bool paired(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % (2 * sizeof(E)) == 0 && ld % 2 == 0;
}

template <typename E>
cudaError_t launch_plan(const lag::Params<E>& p, const Plan& q, int sms, cudaStream_t s) {
  const size_t want = (q.words / 4 + lag::kThreads - 1) / lag::kThreads;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want < size_t(sms) * 8 ? want : size_t(sms) * 8);
  return la_host::launch_pdl(lag::scan_plan_kernel<E>, grid, lag::kThreads, 0, s, p, q.words);
}

template <typename E>
la_status launch_scan(const lag::Params<E>& p, const Plan& q, bool backward, float* dslopes, int sms, cudaStream_t s) {
  cudaError_t ce = q.waits ? launch_plan(p, q, sms, s) : cudaSuccess;
  const unsigned grid = static_cast<unsigned>(q.tiles) * q.columns;
  const bool pair = p.C % 2 == 0 && paired<E>(p.x, p.ldx) && paired<E>(p.r, p.ldr) && paired<E>(p.g, p.ldg) &&
                    (backward ? paired<E>(p.o_in, p.ldo) && paired<E>(p.dout, p.lddout) && paired<E>(p.dx, p.lddx) &&
                                    paired<E>(p.dr, p.lddr) && paired<E>(p.dg, p.lddg)
                              : paired<E>(p.o, p.ldo));
  if (ce == cudaSuccess && q.tiles > 0) {
    auto kernel = backward ? (pair ? lag::gated_scan_bwd_kernel<E, true> : lag::gated_scan_bwd_kernel<E, false>)
                           : (pair ? lag::gated_scan_fwd_kernel<E, true> : lag::gated_scan_fwd_kernel<E, false>);
    ce = la_host::launch_pdl(kernel, grid, lag::kScanThreads, 0, s, p);
  }
  if (ce == cudaSuccess && backward)
    ce = la_host::launch_pdl(lag::column_sum_kernel, (p.C + 31) / 32, 1024, 0, s, static_cast<const float*>(p.part),
                             q.tiles, p.C, static_cast<const int*>(p.cu_seqlens ? p.ticket : nullptr), dslopes);
  if (ce == cudaSuccess) ce = cudaGetLastError();
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

template <typename E>
lag::Params<E> params_of(const void* x, const void* r, const void* g, const float* slopes, int64_t ldx, int64_t ldr,
                         int64_t ldg, const int32_t* state_indices, int* dev_error, int T, int N, int C,
                         int pool_size) {
  lag::Params<E> p{};
  p.x = static_cast<const E*>(x);
  p.r = static_cast<const E*>(r);
  p.g = static_cast<const E*>(g);
  p.slopes = slopes;
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldg = ldg;
  p.state_indices = state_indices;
  p.dev_error = dev_error;
  p.T = T;
  p.N = N;
  p.C = C;
  p.pool_size = pool_size;
  return p;
}

// Checks, then one launch, of the three speculative-decoding entry points.
la_status decode_call(const void* x, const void* r, const void* g, const float* slopes, const float* state,
                      float* state_out, const int32_t* state_indices, const int32_t* accepted_len, void* o, bool outputs,
                      int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo, int B, int T, int C, int pool_size,
                      la_dtype dtype, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(B, T, B, C, false, dtype);
  if (st != LA_OK) return st;
  if (T < 1) return fail(LA_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if ((st = check_pool(true, state_indices, pool_size, B)) != LA_OK) return st;
  if (B == 0) return LA_OK;
  if (!x || !r || !g || !slopes || !state || (outputs && !o) || (!outputs && !accepted_len))
    return fail(LA_ERR_INVALID_ARGUMENT, "x, r, g, slopes, state and %s must be non-null",
                outputs ? "o" : "accepted_len");
  const uint64_t es = la_host::element_size(dtype), rows = static_cast<uint64_t>(B) * T;
  const RowSpan ins[] = {la_host::rows_of(x, ldx, rows, C, es, "x"),
                         la_host::rows_of(r, ldr, rows, C, es, "r"),
                         la_host::rows_of(g, ldg, rows, C, es, "g"),
                         la_host::flat(slopes, static_cast<uint64_t>(C) * 4, "slopes"),
                         la_host::flat(state_indices, static_cast<uint64_t>(B) * 4, "state_indices"),
                         la_host::flat(accepted_len, static_cast<uint64_t>(B) * 4, "accepted_len"),
                         pool_span(state_out ? nullptr : state, "state", state_indices, pool_size, B, C)};
  const RowSpan outs[] = {la_host::rows_of(o, ldo, rows, C, es, "o"),
                          pool_span(state_out, "state", state_indices, pool_size, B, C),
                          la_host::flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 7, outs, 3)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    auto p = params_of<E>(x, r, g, slopes, ldx, ldr, ldg, state_indices, dev_error, T, B, C, pool_size);
    p.o = static_cast<E*>(o);
    p.ldo = ldo;
    p.start = state;
    p.finish = state_out;
    p.accepted_len = accepted_len;
    const unsigned grid = static_cast<unsigned>(B) * ((C + lag::kThreads - 1) / lag::kThreads);
    cudaError_t ce = la_host::launch_pdl(lag::gated_decode_kernel<E>, grid, lag::kThreads, 0,
                                         static_cast<cudaStream_t>(stream), p);
    if (ce == cudaSuccess) ce = cudaGetLastError();
    return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // namespace

extern "C" {

la_status la_gated_scan_workspace(int B, int T, int N, int C, int packed, la_dtype dtype, int backward,
                                  size_t* bytes) {
  la_host::g_last_error[0] = '\0';
  if (!bytes) return fail(LA_ERR_INVALID_ARGUMENT, "bytes is null");
  const la_status st = check_sizes(B, T, N, C, packed != 0, dtype);
  if (st != LA_OK) return st;
  *bytes = plan_of(B, T, N, C, packed != 0, dtype, backward != 0).bytes;
  return LA_OK;
}

la_status la_gated_scan_fwd(const void* x, const void* r, const void* g, const float* slopes, const float* h0,
                            const int32_t* state_indices, const int32_t* cu_seqlens, void* o, float* h_final,
                            int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo, int B, int T, int N, int C,
                            int pool_size, la_dtype dtype, void* workspace, size_t workspace_bytes, int* dev_error,
                            void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(B, T, N, C, cu_seqlens != nullptr, dtype);
  if (st != LA_OK) return st;
  if ((st = check_pool(h0 || h_final, state_indices, pool_size, N)) != LA_OK) return st;
  if (N == 0) return LA_OK;
  const uint64_t es = la_host::element_size(dtype), rows = static_cast<uint64_t>(B) * T;
  if (!slopes || (rows > 0 && (!x || !r || !g || !o)))
    return fail(LA_ERR_INVALID_ARGUMENT, "x, r, g, slopes and o must be non-null");
  const Plan w = plan_of(B, T, N, C, cu_seqlens != nullptr, dtype, false);
  if ((st = la_host::check_workspace(workspace, workspace_bytes, w.bytes)) != LA_OK) return st;
  const RowSpan ins[] = {la_host::rows_of(x, ldx, rows, C, es, "x"),
                         la_host::rows_of(r, ldr, rows, C, es, "r"),
                         la_host::rows_of(g, ldg, rows, C, es, "g"),
                         la_host::flat(slopes, static_cast<uint64_t>(C) * 4, "slopes"),
                         pool_span(h0 == h_final ? nullptr : h0, "h0", state_indices, pool_size, N, C),
                         la_host::flat(state_indices, static_cast<uint64_t>(N) * 4, "state_indices"),
                         la_host::flat(cu_seqlens, static_cast<uint64_t>(N) * 4 + 4, "cu_seqlens")};
  const RowSpan outs[] = {la_host::rows_of(o, ldo, rows, C, es, "o"),
                          pool_span(h_final, "h_final", state_indices, pool_size, N, C),
                          la_host::flat(workspace, w.bytes, "workspace"),
                          la_host::flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 7, outs, 4)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    auto p = params_of<E>(x, r, g, slopes, ldx, ldr, ldg, state_indices, dev_error, T, N, C,
                          la_host::effective_pool_size(h0, h_final, state_indices, pool_size, N));
    p.o = static_cast<E*>(o);
    p.ldo = ldo;
    p.start = h0;
    p.finish = h_final;
    p.cu_seqlens = cu_seqlens;
    p.rows = static_cast<int>(rows);
    set_plan(&p, w, workspace);
    return launch_scan<E>(p, w, false, nullptr, ds->sms, static_cast<cudaStream_t>(stream));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

la_status la_gated_scan_bwd(const void* x, const void* r, const void* g, const float* slopes, const float* h0,
                            const void* o, const void* dout, const float* dh_final, const int32_t* state_indices,
                            const int32_t* cu_seqlens, void* dx, void* dr, void* dg, float* dslopes, float* dh0,
                            int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo, int64_t lddout, int64_t lddx,
                            int64_t lddr, int64_t lddg, int B, int T, int N, int C, int pool_size, la_dtype dtype,
                            void* workspace, size_t workspace_bytes, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(B, T, N, C, cu_seqlens != nullptr, dtype);
  if (st != LA_OK) return st;
  const bool states = h0 || dh_final || dh0;
  if ((st = check_pool(states, state_indices, pool_size, N)) != LA_OK) return st;
  const uint64_t es = la_host::element_size(dtype), rows = static_cast<uint64_t>(B) * T;
  if (!slopes || !dslopes || (rows > 0 && (!x || !r || !g || !o || !dout || !dx || !dr || !dg)))
    return fail(LA_ERR_INVALID_ARGUMENT, "x, r, g, slopes, o, dout, dx, dr, dg and dslopes must be non-null");
  const Plan w = plan_of(B, T, N, C, cu_seqlens != nullptr, dtype, true);
  if ((st = la_host::check_workspace(workspace, workspace_bytes, w.bytes)) != LA_OK) return st;
  const RowSpan ins[] = {la_host::rows_of(x, ldx, rows, C, es, "x"),
                         la_host::rows_of(r, ldr, rows, C, es, "r"),
                         la_host::rows_of(g, ldg, rows, C, es, "g"),
                         la_host::rows_of(o, ldo, rows, C, es, "o"),
                         la_host::rows_of(dout, lddout, rows, C, es, "dout"),
                         la_host::flat(slopes, static_cast<uint64_t>(C) * 4, "slopes"),
                         pool_span(h0, "h0", state_indices, pool_size, N, C),
                         pool_span(dh_final, "dh_final", state_indices, pool_size, N, C),
                         la_host::flat(state_indices, static_cast<uint64_t>(N) * 4, "state_indices"),
                         la_host::flat(cu_seqlens, static_cast<uint64_t>(N) * 4 + 4, "cu_seqlens")};
  const RowSpan outs[] = {la_host::rows_of(dx, lddx, rows, C, es, "dx"),
                          la_host::rows_of(dr, lddr, rows, C, es, "dr"),
                          la_host::rows_of(dg, lddg, rows, C, es, "dg"),
                          la_host::flat(dslopes, static_cast<uint64_t>(C) * 4, "dslopes"),
                          pool_span(dh0, "dh0", state_indices, pool_size, N, C),
                          la_host::flat(workspace, w.bytes, "workspace"),
                          la_host::flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 10, outs, 7)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    const int pool = states ? pool_size : state_indices ? INT32_MAX : N;
    auto p = params_of<E>(x, r, g, slopes, ldx, ldr, ldg, state_indices, dev_error, T, N, C, pool);
    p.o_in = static_cast<const E*>(o);
    p.ldo = ldo;
    p.dout = static_cast<const E*>(dout);
    p.lddout = lddout;
    p.dx = static_cast<E*>(dx);
    p.lddx = lddx;
    p.dr = static_cast<E*>(dr);
    p.lddr = lddr;
    p.dg = static_cast<E*>(dg);
    p.lddg = lddg;
    p.start = dh_final;
    p.finish = dh0;
    p.h0 = h0;
    p.cu_seqlens = cu_seqlens;
    p.rows = static_cast<int>(rows);
    set_plan(&p, w, workspace);
    return launch_scan<E>(p, w, true, dslopes, ds->sms, static_cast<cudaStream_t>(stream));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

la_status la_gated_decode(const void* x, const void* r, const void* g, const float* slopes, float* state,
                          const int32_t* state_indices, void* o, int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo,
                          int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error, void* stream) {
  return decode_call(x, r, g, slopes, state, state, state_indices, nullptr, o, true, ldx, ldr, ldg, ldo, B, T, C,
                     pool_size, dtype, dev_error, stream);
}

la_status la_gated_verify(const void* x, const void* r, const void* g, const float* slopes, const float* state,
                          const int32_t* state_indices, void* o, int64_t ldx, int64_t ldr, int64_t ldg, int64_t ldo,
                          int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error, void* stream) {
  return decode_call(x, r, g, slopes, state, nullptr, state_indices, nullptr, o, true, ldx, ldr, ldg, ldo, B, T, C,
                     pool_size, dtype, dev_error, stream);
}

la_status la_gated_commit(const void* x, const void* r, const void* g, const float* slopes, float* state,
                          const int32_t* state_indices, const int32_t* accepted_len, int64_t ldx, int64_t ldr,
                          int64_t ldg, int B, int T, int C, int pool_size, la_dtype dtype, int* dev_error,
                          void* stream) {
  return decode_call(x, r, g, slopes, state, state, state_indices, accepted_len, nullptr, false, ldx, ldr, ldg, 0, B,
                     T, C, pool_size, dtype, dev_error, stream);
}

}  // extern "C"
