// la_rows_common.h -- host-side checks shared by the entry points that work on rows of channels
// with row strides of their own (la_gated.h, la_norm.h).
#pragma once

#include <cstdint>

#include "../../include/la_gated.h"
#include "la_host_common.h"

namespace la_host {

constexpr int64_t kMaxRows = INT32_MAX - 1024;  // row numbers and tile ends stay within int32

inline uint64_t element_size(la_dtype t) { return t == LA_DTYPE_FP32 ? 4 : 2; }
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// A buffer as rows of `width` bytes, `stride` bytes apart; a contiguous one is a single row.
struct RowSpan {
  const void* p;
  uint64_t width, stride, rows, align;
  int64_t ld, columns;  // as the caller gave them (0 for a contiguous buffer)
  const char* name;
};

inline RowSpan flat(const void* p, uint64_t bytes, const char* name) { return {p, bytes, bytes, 1, 4, 0, 0, name}; }

inline RowSpan rows_of(const void* p, int64_t ld, uint64_t rows, int64_t columns, uint64_t element, const char* name) {
  return {p,    static_cast<uint64_t>(columns) * element, static_cast<uint64_t>(ld) * element, rows, element, ld,
          columns, name};
}

// Whether two buffers share a byte.  Rows of one stride that interleave (column ranges of one
// matrix) share none; otherwise the whole address ranges count.
inline bool share(const RowSpan& a, const RowSpan& b) {
  if (!a.p || !b.p || a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
  const uint64_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t ex = x + (a.rows - 1) * a.stride + a.width, ey = y + (b.rows - 1) * b.stride + b.width;
  if (x >= ey || y >= ex) return false;
  if (a.stride != b.stride || (a.rows == 1 && b.rows == 1)) return true;
  const uint64_t s = a.stride, d = y >= x ? (y - x) % s : (s - (x - y) % s) % s;  // b's column, from a's
  return d < a.width || d + b.width > s;
}

// Row strides and alignment of every buffer, then outs against ins and against each other.
inline la_status check_rows(const RowSpan* ins, int n_in, const RowSpan* outs, int n_out) {
  for (int i = 0; i < n_in + n_out; ++i) {
    const RowSpan& s = i < n_in ? ins[i] : outs[i - n_in];
    if (!s.p) continue;
    if (s.columns > 0 && (s.ld < s.columns || s.ld > (int64_t(1) << 40)))
      return fail(LA_ERR_INVALID_ARGUMENT, "the row stride of %s (%lld) must be at least C (%lld)", s.name,
                  (long long)s.ld, (long long)s.columns);
    if (reinterpret_cast<uintptr_t>(s.p) % s.align != 0)
      return fail(LA_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", s.name, (int)s.align);
  }
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (share(outs[i], ins[j]))
        return fail(LA_ERR_INVALID_ARGUMENT, "%s overlaps %s (an output may share no memory with an input)",
                    outs[i].name, ins[j].name);
    for (int j = 0; j < i; ++j)
      if (share(outs[i], outs[j]))
        return fail(LA_ERR_INVALID_ARGUMENT, "%s overlaps %s (outputs may share no memory)", outs[i].name,
                    outs[j].name);
  }
  return LA_OK;
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
  return launch_pdl(kernel, *blocks, threads, shared, s, args...);
}

inline la_status check_workspace(const void* workspace, size_t given, size_t needed) {
  if (needed == 0) return LA_OK;
  if (!workspace || given < needed)
    return fail(LA_ERR_INVALID_ARGUMENT, "workspace of %zu bytes given, %zu needed", workspace ? given : size_t(0),
                needed);
  if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return fail(LA_ERR_INVALID_ARGUMENT, "workspace must be 256-byte aligned");
  return LA_OK;
}

}  // namespace la_host
