// la_norm_api.cu -- host side of the C ABI declared in include/la_norm.h: argument validation and
// the launches.  Nothing here allocates device memory, reads device memory or synchronises with
// the host.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/la_norm.h"
#include "la_host_common.h"
#include "la_norm_kernels.cuh"
#include "la_rows_common.h"

namespace {

using la_host::fail;
using la_host::flat;
using la_host::rows_of;
using la_host::RowSpan;

la_host::DeviceState g_dev[la_host::kMaxDevices];
using lan::kMaxColumns;

la_status check_sizes(int rows, int C, la_dtype dtype) {
  if (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32) return fail(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (C < 1 || rows < 0) return fail(LA_ERR_INVALID_ARGUMENT, "C must be >= 1 and rows >= 0 (got %d, %d)", C, rows);
  if (C > kMaxColumns) return fail(LA_ERR_UNSUPPORTED, "C up to %d is implemented (got %d)", kMaxColumns, C);
  if (rows > la_host::kMaxRows) return fail(LA_ERR_UNSUPPORTED, "rows too large (%d)", rows);
  return LA_OK;
}

// How a row is shared out: threads per row and per block, and elements per thread (8, 16 or 32,
// a template parameter of the kernels), `most` of them if the threads suffice; `least` threads.
struct Split {
  int share, threads, elements;
};
Split split_of(int C, int vec, int most, int least = 8) {
  Split q;
  q.share = least;
  while (q.share < lan::kMaxThreads && C > q.share * most) q.share *= 2;
  q.threads = q.share < 256 ? 256 : q.share;
  const int loads = ((C + vec - 1) / vec + q.share - 1) / q.share;
  q.elements = loads * vec <= 8 ? 8 : loads * vec <= 16 ? 16 : 32;
  return q;
}

// Elements per thread, where rows allow it: 64 bytes of each input.  Measured against 16 elements:
// gradients of 16384 x 4096 BF16 92 and 115 us, of 8192 x 4096 FP32 87 (32 elements) and 82; single
// elements 26 (32 elements) and 18 us for 4099 x 1001.
template <typename E>
int most_of(bool vec) { return vec ? 64 / static_cast<int>(sizeof(E)) : 16; }

// The ring of a persistent block: as many stages as fit beside `blocks` blocks per SM (one block
// per 512 threads at least), none if there is no room for two.
int stages_of(size_t stage, int threads) {
  constexpr size_t kShared = 227 * 1024;
  for (int blocks = 1024 / threads; blocks >= 1; blocks /= 2) {
    const size_t room = kShared / blocks - 2048;
    const size_t n = room / stage;
    if (n >= 2) return n < lan::kMaxStages ? static_cast<int>(n) : lan::kMaxStages;
  }
  return 0;
}

// Whether rows can be read and written 16 bytes at a time.
template <typename E>
bool wide(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(E) % 16 == 0;
}
template <typename E>
constexpr int vec_of() { return 16 / static_cast<int>(sizeof(E)); }

// Calls f(std::integral_constant<int, kVec>, std::integral_constant<int, kLoads>).
template <typename E, typename F>
cudaError_t with_split(bool vec, int elements, F f) {
  constexpr int kVec = vec_of<E>();
  using std::integral_constant;
  if (vec) {
    if (elements == 8) return f(integral_constant<int, kVec>{}, integral_constant<int, 8 / kVec>{});
    if (elements == 16) return f(integral_constant<int, kVec>{}, integral_constant<int, 16 / kVec>{});
    return f(integral_constant<int, kVec>{}, integral_constant<int, 32 / kVec>{});
  }
  if (elements == 8) return f(integral_constant<int, 1>{}, integral_constant<int, 8>{});
  if (elements == 16) return f(integral_constant<int, 1>{}, integral_constant<int, 16>{});
  return f(integral_constant<int, 1>{}, integral_constant<int, 32>{});
}

// One-time setup per device: the rings exceed the default shared memory.
template <typename E>
cudaError_t setup_type() {
  cudaError_t e = cudaSuccess;
  for (int vec = 0; vec < 2; ++vec)
    for (int elements = 8; elements <= 32; elements *= 2)
      if (e == cudaSuccess)
        e = with_split<E>(vec != 0, elements, [](auto v, auto l) {
          constexpr int kVec = decltype(v)::value, kLoads = decltype(l)::value, most = 226 * 1024;
          const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
          cudaError_t r = cudaFuncSetAttribute(lan::norm_fwd_ring_kernel<E, kVec, kLoads>, attr, most);
          if (r == cudaSuccess) r = cudaFuncSetAttribute(lan::norm_bwd_kernel<E, true, kVec, kLoads>, attr, most);
          return r;
        });
  return e;
}

la_status device(la_host::DeviceState** ds) {
  return la_host::current_device(g_dev, ds, [] {
    const cudaError_t e = setup_type<__nv_bfloat16>();
    return e == cudaSuccess ? setup_type<float>() : e;
  });
}

// Launches a persistent kernel with as many blocks as the device holds at once, `most` at most.
template <typename... Params, typename... Args>
cudaError_t launch_resident(void (*kernel)(Params...), int sms, int most, int threads, int shared, cudaStream_t s,
                            int* blocks, Args... args) {
  // the last answers, by kernel and block (the query costs as much as a launch)
  struct Known {
    const void* kernel = nullptr;
    int threads = 0, shared = 0, sms = 0, per_sm = 0;
  };
  thread_local Known known[16];
  const void* id = reinterpret_cast<const void*>(kernel);
  Known& k = known[(reinterpret_cast<uintptr_t>(id) / 16 + static_cast<uintptr_t>(shared) / 1024) % 16];
  if (k.kernel != id || k.threads != threads || k.shared != shared || k.sms != sms) {
    int n = 0;
    const cudaError_t ce = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, shared);
    if (ce != cudaSuccess) return ce;
    k = {id, threads, shared, sms, n};
  }
  const int per_sm = k.per_sm;
  *blocks = per_sm * sms < most ? (per_sm < 1 ? 1 : per_sm * sms) : most;
  return la_host::launch_pdl(kernel, *blocks, threads, shared, s, args...);
}

// Most blocks of the gradient kernel (rows of partial sums): eight per SM of the largest part.
constexpr int kMostBlocks = 8 * 152;
int bwd_blocks(int rows) { return rows < kMostBlocks ? rows : kMostBlocks; }
size_t bwd_bytes(int rows, int C) { return la_host::align256(static_cast<size_t>(bwd_blocks(rows)) * C * 4); }

la_status forward(const void* x, const void* residual, const float* weight, float eps, void* y, float* scales,
                  void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy, int64_t ldres_out, int rows, int C,
                  bool fp8, int group, la_dtype dtype, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(rows, C, dtype);
  if (st != LA_OK) return st;
  if (fp8 && group != 0 && group != lan::kGroup)
    return fail(LA_ERR_UNSUPPORTED, "group must be 0 or %d (got %d)", lan::kGroup, group);
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (residual_out && !residual) return fail(LA_ERR_INVALID_ARGUMENT, "residual_out needs a residual");
  if (rows == 0) return LA_OK;
  if (!x || !weight || !y || (fp8 && !scales))
    return fail(LA_ERR_INVALID_ARGUMENT, "x, weight, y%s must be non-null", fp8 ? " and scales" : "");
  const uint64_t es = la_host::element_size(dtype);
  const bool in_place = residual_out && residual_out == residual && ldres_out == ldres;
  const uint64_t groups = group ? (C + group - 1) / group : 1;
  const RowSpan ins[] = {rows_of(x, ldx, rows, C, es, "x"),
                         rows_of(in_place ? nullptr : residual, ldres, rows, C, es, "residual"),
                         flat(weight, static_cast<uint64_t>(C) * 4, "weight")};
  const RowSpan outs[] = {rows_of(y, ldy, rows, C, fp8 ? 1 : es, "y"),
                          rows_of(residual_out, ldres_out, rows, C, es, "residual_out"),
                          flat(scales, fp8 ? rows * groups * 4 : 0, "scales"), flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 3, outs, 4)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = [&](auto tag) {
    using E = decltype(tag);
    lan::FwdParams<E> p{};
    p.x = static_cast<const E*>(x);
    p.res = static_cast<const E*>(residual);
    p.res_out = static_cast<E*>(residual_out);
    p.weight = weight;
    p.ldx = ldx;
    p.ldres = ldres;
    p.ldy = ldy;
    p.ldres_out = ldres_out;
    p.eps = eps;
    p.rows = rows;
    p.C = C;
    p.group = group;
    p.scales = scales;
    p.y = fp8 ? nullptr : static_cast<E*>(y);
    p.y8 = static_cast<uint8_t*>(y);
    const bool vec = C % vec_of<E>() == 0 && wide<E>(x, ldx) && (!residual || wide<E>(residual, ldres)) &&
                     (!residual_out || wide<E>(residual_out, ldres_out)) &&
                     reinterpret_cast<uintptr_t>(weight) % 16 == 0 &&
                     (fp8 ? reinterpret_cast<uintptr_t>(y) % vec_of<E>() == 0 && ldy % vec_of<E>() == 0 : wide<E>(y, ldy));
    p.dev_error = dev_error;
    const int v1 = vec ? vec_of<E>() : 1;
    // one load of a row's threads covers a group of columns, or the row
    const int least = group && vec && C > 8 * v1 ? group / v1 : 8;
    Split q = split_of(C, v1, most_of<E>(vec), least);
    const int at_once = q.threads / q.share;
    p.share = q.share;
    const size_t stage = 2 * static_cast<size_t>(at_once) * lan::row_pitch<E>(C);
    const int stages = stages_of(stage, q.threads);
    cudaError_t ce;
    // 8-bit rows are reduced twice, one after the other, and gain from the ring where blocks have
    // several turns (16384 x 8192 BF16: 146 us with it, 167 without); the others do not (186 and
    // 168; FP32 8192 x 8192 182 and 155)
    if (fp8 && stages > 0 && rows / at_once >= 8 * ds->sms) {
      int blocks;
      ce = with_split<E>(vec, q.elements, [&](auto v, auto l) {
        return launch_resident(lan::norm_fwd_ring_kernel<E, decltype(v)::value, decltype(l)::value>, ds->sms,
                               (rows + at_once - 1) / at_once, q.threads, static_cast<int>(stage * stages), s, &blocks,
                               p, stages);
      });
    } else {
      ce = with_split<E>(vec, q.elements, [&](auto v, auto l) {
        constexpr int kVec = decltype(v)::value, kLoads = decltype(l)::value;
        auto kernel = fp8 ? lan::norm_fwd_kernel<E, true, kVec, kLoads> : lan::norm_fwd_kernel<E, false, kVec, kLoads>;
        return la_host::launch_pdl(kernel, static_cast<unsigned>((rows + at_once - 1) / at_once), q.threads, 0, s, p);
      });
    }
    return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // namespace

extern "C" {

la_status la_rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps, void* y,
                          void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy, int64_t ldres_out, int rows,
                          int C, la_dtype dtype, int* dev_error, void* stream) {
  return forward(x, residual, weight, eps, y, nullptr, residual_out, ldx, ldres, ldy, ldres_out, rows, C, false, 0,
                 dtype, dev_error, stream);
}

la_status la_rms_norm_fwd_fp8(const void* x, const void* residual, const float* weight, float eps, void* y,
                              float* scales, void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy,
                              int64_t ldres_out, int rows, int C, int group, la_dtype dtype, int* dev_error,
                              void* stream) {
  return forward(x, residual, weight, eps, y, scales, residual_out, ldx, ldres, ldy, ldres_out, rows, C, true, group,
                 dtype, dev_error, stream);
}

la_status la_rms_norm_bwd_workspace(int rows, int C, size_t* bytes) {
  la_host::g_last_error[0] = '\0';
  if (!bytes) return fail(LA_ERR_INVALID_ARGUMENT, "bytes is null");
  const la_status st = check_sizes(rows, C, LA_DTYPE_BF16);
  if (st != LA_OK) return st;
  *bytes = bwd_bytes(rows, C);
  return LA_OK;
}

la_status la_rms_norm_bwd(const void* s, const float* weight, float eps, const void* dy, const void* dres, void* dx,
                          float* dweight, int64_t lds, int64_t lddy, int64_t lddres, int64_t lddx, int rows, int C,
                          la_dtype dtype, void* workspace, size_t workspace_bytes, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(rows, C, dtype);
  if (st != LA_OK) return st;
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (!dweight || !weight || (rows > 0 && (!s || !dy || !dx)))
    return fail(LA_ERR_INVALID_ARGUMENT, "s, weight, dy, dx and dweight must be non-null");
  const size_t need = bwd_bytes(rows, C);
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  const uint64_t es = la_host::element_size(dtype);
  const RowSpan ins[] = {rows_of(s, lds, rows, C, es, "s"), rows_of(dy, lddy, rows, C, es, "dy"),
                         rows_of(dres, lddres, rows, C, es, "dres"),
                         flat(weight, static_cast<uint64_t>(C) * 4, "weight")};
  const RowSpan outs[] = {rows_of(dx, lddx, rows, C, es, "dx"), flat(dweight, static_cast<uint64_t>(C) * 4, "dweight"),
                          flat(workspace, need, "workspace"), flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 4, outs, 4)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  auto run = [&](auto tag) {
    using E = decltype(tag);
    lan::BwdParams<E> p{};
    p.s = static_cast<const E*>(s);
    p.dy = static_cast<const E*>(dy);
    p.dres = static_cast<const E*>(dres);
    p.dx = static_cast<E*>(dx);
    p.weight = weight;
    p.part = static_cast<float*>(workspace);
    p.lds = lds;
    p.lddy = lddy;
    p.lddres = lddres;
    p.lddx = lddx;
    p.eps = eps;
    p.rows = rows;
    p.C = C;
    const bool vec = C % vec_of<E>() == 0 && wide<E>(s, lds) && wide<E>(dy, lddy) && (!dres || wide<E>(dres, lddres)) &&
                     wide<E>(dx, lddx) && reinterpret_cast<uintptr_t>(weight) % 16 == 0;
    p.dev_error = dev_error;
    const Split q = split_of(C, vec ? vec_of<E>() : 1, most_of<E>(vec));
    p.share = q.share;
    const int at_once = q.threads / q.share;
    const size_t stage = 3 * static_cast<size_t>(at_once) * lan::row_pitch<E>(C);
    const int stages = stages_of(stage, q.threads);
    const int add = at_once > 1 ? at_once * C * static_cast<int>(sizeof(float)) : 0;
    const int most = (rows + at_once - 1) / at_once < bwd_blocks(rows) ? (rows + at_once - 1) / at_once : bwd_blocks(rows);
    int blocks = 0;
    cudaError_t ce = cudaSuccess;
    if (rows > 0)
      ce = with_split<E>(vec, q.elements, [&](auto v, auto l) {
        constexpr int kVec = decltype(v)::value, kLoads = decltype(l)::value;
        if (stages > 0) {
          const int ring = static_cast<int>(stage * stages);
          return launch_resident(lan::norm_bwd_kernel<E, true, kVec, kLoads>, ds->sms, most, q.threads,
                                 ring > add ? ring : add, cs, &blocks, p, stages);
        }
        // FP32 rows of more than about 9600 columns: two stages do not fit
        if constexpr (sizeof(E) == 4 && kVec * kLoads == 32)
          return launch_resident(lan::norm_bwd_kernel<E, false, kVec, kLoads>, ds->sms, most, q.threads, add, cs,
                                 &blocks, p, 0);
        return cudaErrorInvalidConfiguration;
      });
    if (ce == cudaSuccess)
      ce = la_host::launch_pdl(lan::column_sum_kernel, (C + 31) / 32, 1024, 0, cs, static_cast<const float*>(p.part),
                               blocks, C, dweight);
    return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // extern "C"
