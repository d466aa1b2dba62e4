// la_norm_api.cu -- host side of the C ABI declared in include/la_norm.h: argument validation and
// the launches.  Nothing here allocates device memory, reads device memory or synchronises with
// the host.
#include <cuda_runtime.h>

#include <cstdint>

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
constexpr int kMaxColumns = 16384;

la_status check_sizes(int rows, int C, la_dtype dtype) {
  if (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32) return fail(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (C < 1 || rows < 0) return fail(LA_ERR_INVALID_ARGUMENT, "C must be >= 1 and rows >= 0 (got %d, %d)", C, rows);
  if (C > kMaxColumns) return fail(LA_ERR_UNSUPPORTED, "C up to %d is implemented (got %d)", kMaxColumns, C);
  if (rows > la_host::kMaxRows) return fail(LA_ERR_UNSUPPORTED, "rows too large (%d)", rows);
  return LA_OK;
}

la_status device() {
  la_host::DeviceState* ds = nullptr;
  return la_host::current_device(g_dev, &ds, [] { return cudaSuccess; });
}

la_status launched() {
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

int bwd_blocks(int rows) { return rows < lan::kBlocks ? rows : lan::kBlocks; }
size_t bwd_bytes(int rows, int C) { return la_host::align256(static_cast<size_t>(bwd_blocks(rows)) * C * 4); }

la_status forward(const void* x, const void* residual, const float* weight, float eps, void* y, float* scales,
                  void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy, int64_t ldres_out, int rows, int C,
                  bool fp8, int group, la_dtype dtype, void* stream) {
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
                          flat(scales, fp8 ? rows * groups * 4 : 0, "scales")};
  if ((st = la_host::check_rows(ins, 3, outs, 3)) != LA_OK) return st;
  if ((st = device()) != LA_OK) return st;
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
    if (fp8) {
      p.y8 = static_cast<uint8_t*>(y);
      lan::norm_fwd_kernel<E, true><<<rows, lan::kThreads, 0, s>>>(p);
    } else {
      p.y = static_cast<E*>(y);
      lan::norm_fwd_kernel<E, false><<<rows, lan::kThreads, 0, s>>>(p);
    }
    return launched();
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // namespace

extern "C" {

la_status la_rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps, void* y,
                          void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy, int64_t ldres_out, int rows,
                          int C, la_dtype dtype, void* stream) {
  return forward(x, residual, weight, eps, y, nullptr, residual_out, ldx, ldres, ldy, ldres_out, rows, C, false, 0,
                 dtype, stream);
}

la_status la_rms_norm_fwd_fp8(const void* x, const void* residual, const float* weight, float eps, void* y,
                              float* scales, void* residual_out, int64_t ldx, int64_t ldres, int64_t ldy,
                              int64_t ldres_out, int rows, int C, int group, la_dtype dtype, void* stream) {
  return forward(x, residual, weight, eps, y, scales, residual_out, ldx, ldres, ldy, ldres_out, rows, C, true, group,
                 dtype, stream);
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
                          la_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
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
                          flat(workspace, need, "workspace")};
  if ((st = la_host::check_rows(ins, 4, outs, 3)) != LA_OK) return st;
  if ((st = device()) != LA_OK) return st;
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
    p.dweight = dweight;
    p.lds = lds;
    p.lddy = lddy;
    p.lddres = lddres;
    p.lddx = lddx;
    p.eps = eps;
    p.rows = rows;
    p.C = C;
    if (rows > 0) lan::norm_bwd_kernel<E><<<bwd_blocks(rows), lan::kThreads, 0, cs>>>(p);
    lan::column_sum_kernel<<<(C + lan::kThreads - 1) / lan::kThreads, lan::kThreads, 0, cs>>>(
        p.part, bwd_blocks(rows), C, dweight);
    return launched();
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // extern "C"
