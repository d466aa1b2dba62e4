// la_rotary_api.cu -- host side of the C ABI declared in include/la_rotary.h: argument validation and
// the launches.  Nothing here allocates device memory, reads device memory or synchronises with
// the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/la_rotary.h"
#include "la_heads_common.h"
#include "la_host_common.h"
#include "la_rotary_kernels.cuh"

namespace {

using la_host::fail;
using la_host::flat;
using la_host::heads_arg;
using la_host::HeadsArg;
using la_host::RowSpan;

la_host::DeviceState g_dev[la_host::kMaxDevices];

// Most blocks of the gradient kernel (rows of partial sums): eight per SM of the largest part.
constexpr int kMostBlocks = 8 * 152;

la_status check_sizes(int tokens, int H, int HK, int D, int R, la_dtype dtype) {
  if (dtype != LA_DTYPE_BF16 && dtype != LA_DTYPE_FP32) return fail(LA_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (D != 64 && D != 128 && D != 256) return fail(LA_ERR_UNSUPPORTED, "only D = 64, 128 and 256 are implemented (got %d)", D);
  if (H < 1 || HK < 1 || tokens < 0)
    return fail(LA_ERR_INVALID_ARGUMENT, "H and HK must be >= 1 and tokens >= 0 (got %d, %d, %d)", H, HK, tokens);
  if (R < 0 || R > D || R % 2) return fail(LA_ERR_INVALID_ARGUMENT, "R must be even and within 0 .. D (got %d)", R);
  if (tokens > la_host::kMaxRows || H > (1 << 16) || HK > (1 << 16))
    return fail(LA_ERR_UNSUPPORTED, "tokens or heads too large (%d, %d, %d)", tokens, H, HK);
  return LA_OK;
}

// Dynamic shared memory: the rows read ahead, then the angles of the block's tokens.
template <typename E, int kVec, int D>
constexpr int rows_bytes(bool backward) {
  constexpr int kChunks = lar::Layout<E, kVec, D>::kChunks;
  return backward ? lar::Ahead<E, kVec, 4 * kChunks>::kBytes : lar::Ahead<E, kVec, 2 * kChunks>::kBytes;
}
int angle_bytes(int tokens, int R) { return tokens * (R / 2) * static_cast<int>(sizeof(float2)); }

// Tokens whose angles a block holds at once, at most; in bytes for the gradients, whose two blocks per SM
// leave that much beside the rows read ahead and the sums.
constexpr int kAngleTokens = 32, kAngleBytes = 28 * 1024;

// Tokens of a block of the forward kernel: enough for eight turns of its groups of threads, as long as
// the grid still holds the three blocks that run at once on each SM.  Measured, BF16, D = 128, us for 1, 2,
// 4, 8, 16, 32 tokens a block: 128 tokens of 72 heads 3.5, 4.4, 6, 9.9, 17; 1024 of 72 (in L2) 12, 10.2, 11.3,
// 9.9, 17; 4096 of 18 (in L2) 31, 18, 12.3, 10.9, 12.6; 16384 of 72 166, 118, 95, 92, 98; 65536 of 9 474, 249,
// 140, 96, 73, 63.
int tokens_per_block(int tokens, int heads, int groups, int sms) {
  int n = 1;
  while (n < kAngleTokens && n * heads < 8 * groups && tokens / (2 * n) >= 3 * sms) n *= 2;
  return n;
}

// Tokens that a block of the gradients takes at a time, by the bytes of a token's queries.  Reading ahead begins
// anew with each such part, which costs most where a token's rows are few; where they are many, the start of
// a part brings the block's threads together, so that they write neighbouring rows at the same time.
// Measured, D = 128, us for 8, 16, 32, 56 tokens: 16384 of 64 + 8 heads BF16 149, 158, 164, 165; of 32 + 4
// 88, 82.4, 82.2, 82; of 16 + 2 61, 54, 50, 45; of 16 + 4 FP32 83.4, 82.4, 84.3, 88.9; 65536 of 8 + 1 BF16
// 159, 132, 116, 113.
int part_tokens(int64_t bytes) { return bytes >= 12 * 1024 ? 8 : bytes >= 6 * 1024 ? 16 : INT32_MAX; }

// Calls f(vector length, head size, whether neighbours rotate) as integral constants.
template <typename E, typename F>
cudaError_t with_layout(bool vec, int D, bool near, F f) {
  using std::integral_constant;
  constexpr int kVec = 16 / static_cast<int>(sizeof(E));
  auto at = [&](auto v, auto n) {
    if (D == 64) return f(v, integral_constant<int, 64>{}, n);
    if (D == 128) return f(v, integral_constant<int, 128>{}, n);
    return f(v, integral_constant<int, 256>{}, n);
  };
  auto of = [&](auto n) { return vec ? at(integral_constant<int, kVec>{}, n) : at(integral_constant<int, 1>{}, n); };
  return near ? of(std::true_type{}) : of(std::false_type{});
}

// One-time setup per device: the rows read ahead exceed the default shared memory.
template <typename E>
cudaError_t setup_type() {
  cudaError_t e = cudaSuccess;
  for (int x = 0; x < 6; ++x)
    if (e == cudaSuccess)
      e = with_layout<E>(true, 64 << x / 2, x % 2, [](auto v, auto d, auto near) {
        constexpr int kVec = decltype(v)::value, kD = decltype(d)::value;
        constexpr bool kNear = decltype(near)::value;
        const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
        const cudaError_t r = cudaFuncSetAttribute(lar::norm_rope_fwd_kernel<E, kVec, kD, kNear>, most,
                                                   rows_bytes<E, kVec, kD>(false) + angle_bytes(kAngleTokens, kD));
        return r != cudaSuccess ? r
                                : cudaFuncSetAttribute(lar::norm_rope_bwd_kernel<E, kVec, kD, kNear>, most,
                                                       rows_bytes<E, kVec, kD>(true) + kAngleBytes);
      });
  return e;
}

la_status device(la_host::DeviceState** ds) {
  return la_host::current_device(g_dev, ds, [] {
    const cudaError_t e = setup_type<__nv_bfloat16>();
    return e == cudaSuccess ? setup_type<float>() : e;
  });
}

// Whether the heads can be read and written 16 bytes at a time.  (With R a multiple of 16, FP32 8, so that no
// vector is cut by the end of the rotated part or of its half.)  Otherwise elements go one at a time, 2 or 4
// bytes an access and one row ahead in registers: 16384 tokens of 32 + 4 heads of 128, BF16, all rotated,
// forward 54 us against 140 with rows 8 bytes off, gradients 84 against 307; FP32 91 against 200 and 156
// against 352.  (R = 90: the same, neighbours forward 182.)
bool wide(const HeadsArg& h) {
  return !h.p || (reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.ld * h.element % 16 == 0 && h.hs * h.element % 16 == 0);
}

template <typename E>
lar::Heads<E> heads_of(const HeadsArg& h) {
  return {static_cast<E*>(const_cast<void*>(h.p)), h.ld, h.hs};
}

la_status launched(cudaError_t ce) {
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

bool same(const HeadsArg& a, const HeadsArg& b) { return a.p == b.p && a.ld == b.ld && a.hs == b.hs; }

la_status check_tables(const int32_t* positions, const float* inv_freq, const float* wq, const float* wk, float eps,
                       int tokens, int R) {
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARGUMENT, "eps must be >= 0");
  if (R > 0 && ((tokens > 0 && !positions) || !inv_freq))
    return fail(LA_ERR_INVALID_ARGUMENT, "positions and inv_freq must be non-null with R > 0");
  if (!la_host::aligned4(positions) || !la_host::aligned4(inv_freq) || !la_host::aligned4(wq) || !la_host::aligned4(wk))
    return fail(LA_ERR_INVALID_ARGUMENT, "positions, inv_freq and the weights must be 4-byte aligned");
  return LA_OK;
}

int bwd_blocks(int tokens) { return tokens < kMostBlocks ? tokens : kMostBlocks; }
size_t bwd_bytes(int tokens, int D) {
  return la_host::align256(static_cast<size_t>(2) * bwd_blocks(tokens) * D * sizeof(float));
}

}  // namespace

extern "C" {

la_status la_qk_norm_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight, float eps,
                              const int32_t* positions, const float* inv_freq, void* q_out, void* k_out, int64_t ldq,
                              int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldqo, int64_t hsqo, int64_t ldko,
                              int64_t hsko, int tokens, int H, int HK, int D, int R, int interleaved, la_dtype dtype,
                              void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(tokens, H, HK, D, R, dtype);
  if (st != LA_OK) return st;
  if ((st = check_tables(positions, inv_freq, q_weight, k_weight, eps, tokens, R)) != LA_OK) return st;
  if (tokens == 0) return LA_OK;
  if (!q || !k || !q_out || !k_out) return fail(LA_ERR_INVALID_ARGUMENT, "q, k, q_out and k_out must be non-null");
  const uint64_t es = la_host::element_size(dtype);
  const HeadsArg args[] = {heads_arg(q, ldq, hsq, tokens, H, D, es, es, "q"),
                           heads_arg(k, ldk, hsk, tokens, HK, D, es, es, "k"),
                           heads_arg(q_out, ldqo, hsqo, tokens, H, D, es, es, "q_out"),
                           heads_arg(k_out, ldko, hsko, tokens, HK, D, es, es, "k_out")};
  bool vec = R % (2 * (16 / static_cast<int>(es))) == 0;
  for (const HeadsArg& h : args) {
    if ((st = la_host::check_heads(h)) != LA_OK) return st;
    vec = vec && wide(h);
  }
  const RowSpan none{nullptr, 0, 0, 0, 1, 0, 0, ""};
  const uint64_t wb = static_cast<uint64_t>(D) * 4;
  const RowSpan ins[] = {same(args[0], args[2]) ? none : span_of(args[0]),
                         same(args[1], args[3]) ? none : span_of(args[1]),
                         flat(q_weight, wb, "q_weight"),
                         flat(k_weight, wb, "k_weight"),
                         flat(positions, static_cast<uint64_t>(tokens) * 4, "positions"),
                         flat(inv_freq, static_cast<uint64_t>(R) * 2, "inv_freq")};
  const RowSpan outs[] = {span_of(args[2]), span_of(args[3])};
  if ((st = la_host::check_apart(ins, 6, outs, 2)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    lar::FwdParams<E> p{};
    for (int i = 0; i < 2; ++i) {
      p.x[i] = heads_of<const E>(args[i]);
      p.y[i] = heads_of<E>(args[2 + i]);
    }
    p.weight[0] = q_weight;
    p.weight[1] = k_weight;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.eps = eps;
    p.tokens = tokens;
    p.heads[0] = H;
    p.heads[1] = HK;
    p.R = R;
    const int lanes = vec ? D * static_cast<int>(es) / 32 : 32;
    p.per_block = tokens_per_block(tokens, H + HK, lar::kThreads / lanes, ds->sms);
    const int blocks = (tokens + p.per_block - 1) / p.per_block;
    return launched(with_layout<E>(vec, D, interleaved != 0, [&](auto v, auto d, auto near) {
      constexpr int kVec = decltype(v)::value, kD = decltype(d)::value;
      constexpr bool kNear = decltype(near)::value;
      return la_host::launch_pdl(lar::norm_rope_fwd_kernel<E, kVec, kD, kNear>, blocks, lar::kThreads,
                                 rows_bytes<E, kVec, kD>(false) + angle_bytes(p.per_block, R),
                                 static_cast<cudaStream_t>(stream), p);
    }));
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

la_status la_qk_norm_rope_bwd_workspace(int tokens, int H, int HK, int D, size_t* bytes) {
  la_host::g_last_error[0] = '\0';
  if (!bytes) return fail(LA_ERR_INVALID_ARGUMENT, "bytes is null");
  const la_status st = check_sizes(tokens, H, HK, D, 0, LA_DTYPE_BF16);
  if (st != LA_OK) return st;
  *bytes = bwd_bytes(tokens, D);
  return LA_OK;
}

la_status la_qk_norm_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight, float eps,
                              const int32_t* positions, const float* inv_freq, const void* dq_out, const void* dk_out,
                              void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t ldq, int64_t hsq,
                              int64_t ldk, int64_t hsk, int64_t lddqo, int64_t hsdqo, int64_t lddko, int64_t hsdko,
                              int64_t lddq, int64_t hsdq, int64_t lddk, int64_t hsdk, int tokens, int H, int HK, int D,
                              int R, int interleaved, la_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_sizes(tokens, H, HK, D, R, dtype);
  if (st != LA_OK) return st;
  if ((st = check_tables(positions, inv_freq, q_weight, k_weight, eps, tokens, R)) != LA_OK) return st;
  if (tokens > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk))
    return fail(LA_ERR_INVALID_ARGUMENT, "q, k, dq_out, dk_out, dq and dk must be non-null");
  if (!la_host::aligned4(dq_weight) || !la_host::aligned4(dk_weight))
    return fail(LA_ERR_INVALID_ARGUMENT, "dq_weight and dk_weight must be 4-byte aligned");
  const bool sums = dq_weight || dk_weight;
  const size_t need = sums ? bwd_bytes(tokens, D) : 0;
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  const uint64_t es = la_host::element_size(dtype);
  const HeadsArg args[] = {heads_arg(q, ldq, hsq, tokens, H, D, es, es, "q"),
                           heads_arg(k, ldk, hsk, tokens, HK, D, es, es, "k"),
                           heads_arg(dq_out, lddqo, hsdqo, tokens, H, D, es, es, "dq_out"),
                           heads_arg(dk_out, lddko, hsdko, tokens, HK, D, es, es, "dk_out"),
                           heads_arg(dq, lddq, hsdq, tokens, H, D, es, es, "dq"),
                           heads_arg(dk, lddk, hsdk, tokens, HK, D, es, es, "dk")};
  bool vec = R % (2 * (16 / static_cast<int>(es))) == 0;
  for (const HeadsArg& h : args) {
    if ((st = la_host::check_heads(h)) != LA_OK) return st;
    vec = vec && wide(h);
  }
  const RowSpan none{nullptr, 0, 0, 0, 1, 0, 0, ""};
  const uint64_t wb = static_cast<uint64_t>(D) * 4;
  const RowSpan ins[] = {span_of(args[0]),
                         span_of(args[1]),
                         same(args[2], args[4]) ? none : span_of(args[2]),
                         same(args[3], args[5]) ? none : span_of(args[3]),
                         flat(q_weight, wb, "q_weight"),
                         flat(k_weight, wb, "k_weight"),
                         flat(positions, static_cast<uint64_t>(tokens) * 4, "positions"),
                         flat(inv_freq, static_cast<uint64_t>(R) * 2, "inv_freq")};
  const RowSpan outs[] = {span_of(args[4]), span_of(args[5]), flat(dq_weight, wb, "dq_weight"),
                          flat(dk_weight, wb, "dk_weight"), flat(workspace, need, "workspace")};
  if ((st = la_host::check_apart(ins, 8, outs, 5)) != LA_OK) return st;
  if (tokens == 0 && !sums) return LA_OK;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  auto run = [&](auto tag) {
    using E = decltype(tag);
    lar::BwdParams<E> p{};
    for (int i = 0; i < 2; ++i) {
      p.x[i] = heads_of<const E>(args[i]);
      p.dy[i] = heads_of<const E>(args[2 + i]);
      p.dx[i] = heads_of<E>(args[4 + i]);
    }
    p.weight[0] = q_weight;
    p.weight[1] = k_weight;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.part = sums ? static_cast<float*>(workspace) : nullptr;
    p.eps = eps;
    p.tokens = tokens;
    p.heads[0] = H;
    p.heads[1] = HK;
    p.R = R;
    const int each = (tokens + 2 * ds->sms - 1) / (2 * ds->sms);  // tokens of a block, about
    p.per_block = std::max(1, std::min({each, part_tokens(static_cast<int64_t>(H) * D * es), R > 0 ? kAngleBytes / angle_bytes(1, R) : each}));
    int blocks = 0;
    cudaError_t ce = cudaSuccess;
    if (tokens > 0)
      ce = with_layout<E>(vec, D, interleaved != 0, [&](auto v, auto d, auto near) {
        constexpr int kVec = decltype(v)::value, kD = decltype(d)::value;
        constexpr bool kNear = decltype(near)::value;
        return la_host::launch_resident(lar::norm_rope_bwd_kernel<E, kVec, kD, kNear>, ds->sms, bwd_blocks(tokens), lar::kThreads,
                                        rows_bytes<E, kVec, kD>(true) + angle_bytes(p.per_block, R), cs, &blocks, p);
      });
    if (ce == cudaSuccess && sums)
      ce = la_host::launch_pdl(lar::weight_sum_kernel, dim3(D / 32, 2), 1024, 0, cs,
                               static_cast<const float*>(p.part), blocks, D, dq_weight, dk_weight);
    return launched(ce);
  };
  return dtype == LA_DTYPE_BF16 ? run(__nv_bfloat16{}) : run(float{});
}

}  // extern "C"
