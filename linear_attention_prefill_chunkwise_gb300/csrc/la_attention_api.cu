// la_attention_api.cu -- host side of the C ABI declared in include/la_attention.h: argument
// validation and the launches.  Nothing here allocates device memory, reads device memory or
// synchronises with the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/la_attention.h"
#include "la_attention_bwd.cuh"
#include "la_attention_commit.cuh"
#include "la_attention_fwd.cuh"
#include "la_attention_verify.cuh"
#include "la_heads_common.h"
#include "la_host_common.h"

namespace {

using la_host::fail;
using la_host::flat;
using la_host::heads_arg;
using la_host::HeadsArg;
using la_host::RowSpan;
using laa::bf16;

la_host::DeviceState g_dev[la_host::kMaxDevices];

template <int D>
constexpr int fwd_shared() {
  static_assert(sizeof(laa::FwdShared<D>) <= 227 * 1024, "shared memory");
  return static_cast<int>(sizeof(laa::FwdShared<D>));
}

template <int D>
constexpr int bwd_shared() {
  static_assert(sizeof(laa::BwdShared<D>) <= 227 * 1024, "shared memory");
  return static_cast<int>(sizeof(laa::BwdShared<D>));
}
template <int D>
constexpr int verify_shared() { return static_cast<int>(sizeof(laa::VerifyShared<D>)) + 1024; }

la_status device(la_host::DeviceState** ds) {
  return la_host::current_device(g_dev, ds, [] {
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(laa::attn_fwd_kernel<64>, most, fwd_shared<64>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_fwd_kernel<128>, most, fwd_shared<128>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_bwd_kernel<64, false>, most, bwd_shared<64>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_bwd_kernel<64, true>, most, bwd_shared<64>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_bwd_kernel<128, false>, most, bwd_shared<128>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_bwd_kernel<128, true>, most, bwd_shared<128>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_verify_kernel<64>, most, verify_shared<64>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(laa::attn_verify_kernel<128>, most, verify_shared<128>());
    return e;
  });
}

la_status launched(cudaError_t ce) {
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

constexpr int kMostDrafts = 1 << 18;  // drafted tokens of a request: their tiles, of all query tiles, stay within int32
constexpr int64_t kMostTokens = INT32_MAX - 1024;  // row numbers and tile ends stay within int32
constexpr float kMostScale = 2.0e38f;  // the kernels multiply it by log2 e

HeadsArg rows(const void* p, int64_t ld, int64_t hs, int64_t tokens, int heads, int D, const char* name) {
  return heads_arg(p, ld, hs, tokens, heads, D, 2, 16, name);
}

struct CacheArg {
  const void* p;
  int64_t pages, tokens, heads;  // extents
  int64_t ps, ts, hs;            // strides
  const char* name;
};

// Map over a tensor of heads with boxes of `heads` heads x `tokens` tokens x 64 columns (a head's rows
// of 128 bytes, 128-byte swizzle).
la_status encode_heads(CUtensorMap* map, const HeadsArg& h, int heads, int tokens) {
  auto enc = la_host::tensor_map_encoder();
  if (!enc) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the CUDA driver");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(h.D), static_cast<cuuint64_t>(h.heads), static_cast<cuuint64_t>(h.tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(h.hs) * 2, static_cast<cuuint64_t>(h.ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(h.p), dims, strides, box, ones,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", h.name, (int)r);
  return LA_OK;
}

// Map over the cache with boxes of `rows` rows of one page and head x 64 columns.
la_status encode_cache(CUtensorMap* map, const CacheArg& c, int D, int rows) {
  auto enc = la_host::tensor_map_encoder();
  if (!enc) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the CUDA driver");
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.tokens),
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.hs) * 2, static_cast<cuuint64_t>(c.ts) * 2,
                                 static_cast<cuuint64_t>(c.ps) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(c.p), dims, strides, box, ones,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with CUresult %d", c.name, (int)r);
  return LA_OK;
}

// How a call's items are cut: see laa::VerifyShape.
laa::VerifyShape verify_shape(int T, int H, int HK, bool mask, int page_size, bool paged) {
  laa::VerifyShape v{};
  v.group = H / HK;
  v.per_tile = std::min(T, laa::kTile / v.group);
  v.rows = v.per_tile * v.group;
  v.q_tiles = (T + v.per_tile - 1) / v.per_tile;
  v.box = laa::kTile;
  if (paged)
    while (page_size % v.box) v.box /= 2;
  v.draft_box = std::min(laa::kTile, (T + 7) / 8 * 8);
  for (int i = 0; i < v.q_tiles; ++i)
    v.drafts += mask ? 1 : static_cast<int>((std::min<int64_t>(T, (i + int64_t(1)) * v.per_tile) + laa::kTile - 1) / laa::kTile);
  return v;
}

// Blocks for at most this many items of work, one per SM.
int blocks_for(int64_t items, int sms) { return static_cast<int>(std::min<int64_t>(items, sms)); }

laa::Heads<const bf16> in(const HeadsArg& h) { return {static_cast<const bf16*>(h.p), h.ld, h.hs}; }
laa::Heads<bf16> out(const HeadsArg& h) { return {static_cast<bf16*>(const_cast<void*>(h.p)), h.ld, h.hs}; }

la_status check_heads_of(int H, int HK, int D) {
  if (D != 64 && D != 128) return fail(LA_ERR_UNSUPPORTED, "only D = 64 and 128 are implemented (got %d)", D);
  if (H < 1 || HK < 1) return fail(LA_ERR_INVALID_ARGUMENT, "H and HK must be >= 1 (got %d, %d)", H, HK);
  if (H % HK != 0) return fail(LA_ERR_UNSUPPORTED, "H (%d) must be a multiple of HK (%d)", H, HK);
  if (H > (1 << 15)) return fail(LA_ERR_UNSUPPORTED, "H too large (%d)", H);
  return LA_OK;
}

// Shapes and batch mode of the prompt calls.
la_status check_prompt(const int32_t* cu_seqlens, int B, int T, int N, int H, int HK, int D) {
  const la_status st = check_heads_of(H, HK, D);
  if (st != LA_OK) return st;
  if (B < 0 || T < 0 || N < 0) return fail(LA_ERR_INVALID_ARGUMENT, "B, T, N must be >= 0");
  if (cu_seqlens) {
    if (B != 1) return fail(LA_ERR_INVALID_ARGUMENT, "packed mode (cu_seqlens given) needs B == 1 (got %d)", B);
    if (!la_host::aligned4(cu_seqlens)) return fail(LA_ERR_INVALID_ARGUMENT, "cu_seqlens must be 4-byte aligned");
  } else if (N != B) {
    return fail(LA_ERR_INVALID_ARGUMENT, "fixed-length mode needs N == B (got N=%d, B=%d)", N, B);
  }
  if (static_cast<int64_t>(B) * T + static_cast<int64_t>(N) * 128 > kMostTokens)
    return fail(LA_ERR_UNSUPPORTED, "B*T too large (%lld)", (long long)B * T);
  return LA_OK;
}

la_status check_scale(float scale) {
  // a scale of 0 is a plain mean; anything not finite has no meaning, nor what is not once log2 e multiplies it
  if (!(scale >= -kMostScale && scale <= kMostScale))
    return fail(LA_ERR_INVALID_ARGUMENT, "scale must be finite and at most %g in size (got %g)", kMostScale, scale);
  return LA_OK;
}

// Checks strides and alignment of every tensor, then outputs (the last n_out) against the others and
// against each other, and both against the flat buffers.
la_status check_tensors(const HeadsArg* args, int n, int n_out, const RowSpan* flat_in, int n_flat_in,
                        const RowSpan* flat_out, int n_flat_out) {
  RowSpan ins[16], outs[16];
  int ni = 0, no = 0;
  for (int i = 0; i < n; ++i) {
    if (!args[i].p) return fail(LA_ERR_INVALID_ARGUMENT, "%s must be non-null", args[i].name);
    const la_status st = la_host::check_heads(args[i]);
    if (st != LA_OK) return st;
    (i < n - n_out ? ins[ni++] : outs[no++]) = la_host::span_of(args[i]);
  }
  for (int i = 0; i < n_flat_in; ++i) ins[ni++] = flat_in[i];
  for (int i = 0; i < n_flat_out; ++i) outs[no++] = flat_out[i];
  return la_host::check_apart(ins, ni, outs, no);
}

// ---------------------------------------------------------------- the cache


// Strides that keep every row of the cache apart (its three outer axes in some order), and the
// cache as rows for the overlap checks: the outer axes that lie gaplessly within one another are
// one, so that key and value pages that interleave token by token share nothing.
la_status check_cache(CacheArg& c, int D, RowSpan* span) {
  if (c.heads == 1) c.hs = D;
  if (c.tokens == 1) c.ts = (c.heads - 1) * c.hs + D;
  if (c.pages == 1) c.ps = std::max((c.tokens - 1) * c.ts, (c.heads - 1) * c.hs) + std::max(c.ts, c.hs);
  struct Axis {
    int64_t n, s;
  } a[3] = {{c.pages, c.ps}, {c.tokens, c.ts}, {c.heads, c.hs}};
  std::sort(a, a + 3, [](const Axis& x, const Axis& y) { return x.s > y.s; });
  constexpr int64_t kMost = int64_t(1) << 38;
  int64_t width = D;
  for (int i = 2; i >= 0; --i) {
    if (a[i].s < width || a[i].s > kMost || a[i].n > kMost / (a[i].s > 0 ? a[i].s : 1))
      return fail(LA_ERR_INVALID_ARGUMENT, "the strides of %s (%lld between pages, %lld between tokens, %lld between heads) do not keep its rows apart",
                  c.name, (long long)c.ps, (long long)c.ts, (long long)c.hs);
    width += (a[i].n - 1) * a[i].s;
  }
  if (!la_host::aligned16(c.p)) return fail(LA_ERR_INVALID_ARGUMENT, "%s must be 16-byte aligned", c.name);
  if (c.ps % 8 || c.ts % 8 || c.hs % 8)
    return fail(LA_ERR_INVALID_ARGUMENT, "the strides of %s must be multiples of 8 elements", c.name);
  int64_t n = a[0].n, s = a[0].s, inner = (a[2].n - 1) * a[2].s + D;
  if (s == a[1].n * a[1].s) {
    n *= a[1].n;
    s = a[1].s;
  } else {
    inner += (a[1].n - 1) * a[1].s;
  }
  *span = {c.p, static_cast<uint64_t>(inner) * 2, static_cast<uint64_t>(s) * 2, static_cast<uint64_t>(n), 16, 0, 0, c.name};
  return LA_OK;
}

// What la_attn_verify and la_attn_commit share: the sizes of the cache.
la_status check_pages(const int32_t* cache_lens, const int32_t* page_table, int B, int T, int HK, int pages,
                      int page_size, int table_width, int64_t ld_table) {
  if (B < 0 || T < 0) return fail(LA_ERR_INVALID_ARGUMENT, "B and T must be >= 0 (got %d, %d)", B, T);
  if (pages < 1 || page_size < 1) return fail(LA_ERR_INVALID_ARGUMENT, "pages and page_size must be >= 1 (got %d, %d)", pages, page_size);
  if (page_size > kMostTokens) return fail(LA_ERR_UNSUPPORTED, "page_size too large (%d)", page_size);
  if (!cache_lens && B > 0) return fail(LA_ERR_INVALID_ARGUMENT, "cache_lens must be non-null");
  if (!la_host::aligned4(cache_lens) || !la_host::aligned4(page_table))
    return fail(LA_ERR_INVALID_ARGUMENT, "cache_lens and page_table must be 4-byte aligned");
  if (page_table) {
    if (page_size % 16 != 0) return fail(LA_ERR_UNSUPPORTED, "page_size must be a multiple of 16 with a page table (got %d)", page_size);
    if (table_width < 1 || (B > 1 && ld_table < table_width))
      return fail(LA_ERR_INVALID_ARGUMENT, "page_table's row stride (%lld) must be at least its width (%d >= 1)", (long long)ld_table, table_width);
    if (static_cast<int64_t>(table_width) * page_size > kMostTokens)
      return fail(LA_ERR_UNSUPPORTED, "table_width * page_size too large (%d, %d)", table_width, page_size);
  } else if (pages < B) {
    return fail(LA_ERR_INVALID_ARGUMENT, "pages (%d) must be >= B (%d) without a page table", pages, B);
  }
  return LA_OK;
}

uint64_t table_bytes(const int32_t* page_table, int B, int table_width, int64_t ld_table) {
  return page_table && B > 0 ? (static_cast<uint64_t>(B - 1) * ld_table + table_width) * 4 : 0;
}

// The gradients' workspace: delta, and, where a group's heads are shared out, the parts' sums and marks.
// Parts: as many as give each SM one item, with two tiles or more each, or two items, with eight or more (by the
// mean number of tiles that an item walks over, here of eight at least).  N sequences; a query for a packed
// batch does not know them and takes one, whose parts are not fewer.
// Measured, gradients, us with whole groups; by the rule (parts; others): one sequence of 8192, 8 heads of 128
// on 1 764; 307 (4; 8: 322); of 2048, 32 on 8 135; 114 (2; 4: 141); 2 x 512, 64 on 8 79; 68 (2; 8: 102); 512,
// 64 on 8 67; 47 (4; 8: 56); 16 x 64, 16 on 1 71; 37 (8; 16: 49); 128, 16 of 64 on 2 25; 20 (4; 8: 22);
// 4 x 2048, 32 on 4 stays whole: 353 (2: 381).
struct BwdWorkspace {
  int splits;
  size_t part, marks, bytes;
};
BwdWorkspace bwd_workspace(int64_t tokens, int N, int H, int HK, int D) {
  constexpr int64_t kSms = 152;
  const int group = H / HK;
  const int64_t tiles = std::max<int64_t>((tokens + laa::kTile - 1) / laa::kTile, N), items = tiles * HK;
  BwdWorkspace w{1, 0, 0, 0};
  const int64_t walk = (std::max<int64_t>(1, tiles / std::max(N, 1)) + 1) * group / 2;
  if (tiles > 0 && walk >= 8) {
    const int64_t one = std::min(kSms / items, walk / 2), two = std::min(2 * kSms / items, walk / 8);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(group, std::max(one, two)));
    const int each = static_cast<int>((group + want - 1) / want);  // heads of a part
    w.splits = (group + each - 1) / each;
  }
  w.part = la_host::align256(static_cast<size_t>(tokens) * H * sizeof(float));
  w.marks = w.part;
  if (w.splits > 1) w.marks += la_host::align256(static_cast<size_t>(w.splits) * 2 * HK * tokens * D * sizeof(float));
  w.bytes = w.marks + (w.splits > 1 ? la_host::align256(static_cast<size_t>(HK) * tokens) : 0);
  return w;
}

template <typename F>
cudaError_t with_dim(int D, F f) {
  if (D == 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

}  // namespace

extern "C" {

la_status la_attn_prefill_fwd(const void* q, const void* k, const void* v, float scale, const int32_t* cu_seqlens,
                              void* o, float* lse, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv,
                              int64_t hsv, int64_t ldo, int64_t hso, int B, int T, int N, int H, int HK, int D,
                              int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_prompt(cu_seqlens, B, T, N, H, HK, D);
  if (st != LA_OK) return st;
  if ((st = check_scale(scale)) != LA_OK) return st;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (tokens == 0 || N == 0) return LA_OK;
  if (!la_host::aligned4(lse) || !la_host::aligned4(dev_error))
    return fail(LA_ERR_INVALID_ARGUMENT, "lse and dev_error must be 4-byte aligned");
  const HeadsArg a[] = {rows(q, ldq, hsq, tokens, H, D, "q"), rows(k, ldk, hsk, tokens, HK, D, "k"),
                        rows(v, ldv, hsv, tokens, HK, D, "v"), rows(o, ldo, hso, tokens, H, D, "o")};
  const RowSpan fin[] = {flat(cu_seqlens, cu_seqlens ? (static_cast<uint64_t>(N) + 1) * 4 : 0, "cu_seqlens")};
  const RowSpan fout[] = {flat(lse, static_cast<uint64_t>(H) * tokens * 4, "lse"), flat(dev_error, 4, "dev_error")};
  if ((st = check_tensors(a, 4, 1, fin, 1, fout, 2)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  laa::PrefillParams p{};
  p.v = in(a[2]), p.o = out(a[3]);
  p.lse = lse;
  p.cu_seqlens = cu_seqlens;
  p.dev_error = dev_error;
  p.scale = scale;
  p.tokens = static_cast<int>(tokens), p.T = T, p.N = N, p.H = H, p.HK = HK;
  laa::FwdMaps maps;
  if ((st = encode_heads(&maps.q, a[0], 1, laa::kTile)) != LA_OK || (st = encode_heads(&maps.k, a[1], 1, laa::kTile)) != LA_OK ||
      (st = encode_heads(&maps.v, a[2], 1, laa::kTile)) != LA_OK)
    return st;
  // tiles of the queries: exact in fixed-length mode, at most in packed mode
  const int64_t tiles = cu_seqlens ? tokens / laa::kFwdRows + N : static_cast<int64_t>(N) * ((T + laa::kFwdRows - 1) / laa::kFwdRows);
  return launched(with_dim(D, [&](auto d) {
    constexpr int kD = decltype(d)::value;
    return la_host::launch_pdl(laa::attn_fwd_kernel<kD>, blocks_for(tiles * H, ds->sms), laa::kFwdThreads, fwd_shared<kD>(),
                               static_cast<cudaStream_t>(stream), maps, p);
  }));
}

la_status la_attn_prefill_bwd_workspace(int B, int T, int H, int HK, int D, size_t* bytes) {
  la_host::g_last_error[0] = '\0';
  if (!bytes) return fail(LA_ERR_INVALID_ARGUMENT, "bytes is null");
  const la_status st = check_heads_of(H, HK, D);
  if (st != LA_OK) return st;
  if (B < 0 || T < 0) return fail(LA_ERR_INVALID_ARGUMENT, "B and T must be >= 0 (got %d, %d)", B, T);
  if (static_cast<int64_t>(B) * T > kMostTokens) return fail(LA_ERR_UNSUPPORTED, "B*T too large (%lld)", (long long)B * T);
  *bytes = bwd_workspace(static_cast<int64_t>(B) * T, B, H, HK, D).bytes;
  return LA_OK;
}

la_status la_attn_prefill_bwd(const void* q, const void* k, const void* v, float scale, const void* o,
                              const float* lse, const void* dout, const int32_t* cu_seqlens, void* dq, void* dk,
                              void* dv, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv, int64_t hsv,
                              int64_t ldo, int64_t hso, int64_t lddo, int64_t hsdo, int64_t lddq, int64_t hsdq,
                              int64_t lddk, int64_t hsdk, int64_t lddv, int64_t hsdv, int B, int T, int N, int H,
                              int HK, int D, void* workspace, size_t workspace_bytes, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_prompt(cu_seqlens, B, T, N, H, HK, D);
  if (st != LA_OK) return st;
  if ((st = check_scale(scale)) != LA_OK) return st;
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (tokens == 0 || N == 0) return LA_OK;
  if (!lse) return fail(LA_ERR_INVALID_ARGUMENT, "lse must be non-null");
  if (!la_host::aligned4(lse) || !la_host::aligned4(dev_error))
    return fail(LA_ERR_INVALID_ARGUMENT, "lse and dev_error must be 4-byte aligned");
  size_t need = 0;
  if ((st = la_attn_prefill_bwd_workspace(B, T, H, HK, D, &need)) != LA_OK) return st;
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  const HeadsArg a[] = {rows(q, ldq, hsq, tokens, H, D, "q"),       rows(k, ldk, hsk, tokens, HK, D, "k"),
                        rows(v, ldv, hsv, tokens, HK, D, "v"),      rows(o, ldo, hso, tokens, H, D, "o"),
                        rows(dout, lddo, hsdo, tokens, H, D, "dout"), rows(dq, lddq, hsdq, tokens, H, D, "dq"),
                        rows(dk, lddk, hsdk, tokens, HK, D, "dk"),  rows(dv, lddv, hsdv, tokens, HK, D, "dv")};
  const RowSpan fin[] = {flat(cu_seqlens, cu_seqlens ? (static_cast<uint64_t>(N) + 1) * 4 : 0, "cu_seqlens"),
                         flat(lse, static_cast<uint64_t>(H) * tokens * 4, "lse")};
  const RowSpan fout[] = {flat(workspace, need, "workspace"), flat(dev_error, 4, "dev_error")};
  if ((st = check_tensors(a, 8, 3, fin, 2, fout, 2)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  laa::PrefillParams p{};
  p.o_in = in(a[3]), p.dout = in(a[4]);
  p.dq = out(a[5]), p.dk = out(a[6]), p.dv = out(a[7]);
  p.lse_in = lse;
  const BwdWorkspace w = bwd_workspace(tokens, N, H, HK, D);
  p.delta = static_cast<float*>(workspace);
  p.splits = w.splits;
  if (w.splits > 1) {
    p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.part);
    p.marks = static_cast<uint8_t*>(workspace) + w.marks;
  }
  p.cu_seqlens = cu_seqlens;
  p.dev_error = dev_error;
  p.scale = scale;
  p.tokens = static_cast<int>(tokens), p.T = T, p.N = N, p.H = H, p.HK = HK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  laa::BwdMaps maps;
  if ((st = encode_heads(&maps.q, a[0], 1, laa::kTile)) != LA_OK || (st = encode_heads(&maps.k, a[1], 1, laa::kTile)) != LA_OK ||
      (st = encode_heads(&maps.v, a[2], 1, laa::kTile)) != LA_OK || (st = encode_heads(&maps.dout, a[4], 1, laa::kTile)) != LA_OK)
    return st;
  const int64_t tiles = cu_seqlens ? tokens / laa::kTile + N : static_cast<int64_t>(N) * ((T + laa::kTile - 1) / laa::kTile);
  const int64_t delta_threads = tokens * H * (D / 8);
  if (delta_threads / laa::kDeltaThreads >= INT32_MAX) return fail(LA_ERR_UNSUPPORTED, "B*T*H too large (%lld)", (long long)(tokens * H));
  return launched(with_dim(D, [&](auto d) {
    constexpr int kD = decltype(d)::value;
    cudaError_t ce = la_host::launch_pdl(laa::attn_delta_kernel<kD>, static_cast<unsigned>((delta_threads + laa::kDeltaThreads - 1) / laa::kDeltaThreads),
                                         laa::kDeltaThreads, 0, s, p);
    if (ce == cudaSuccess)
      ce = la_host::launch_pdl(laa::attn_bwd_kernel<kD, false>, blocks_for(tiles * HK * p.splits, ds->sms), laa::kBwdThreads, bwd_shared<kD>(), s, maps, p);
    if (ce == cudaSuccess)
      ce = la_host::launch_pdl(laa::attn_bwd_kernel<kD, true>, blocks_for(tiles * H, ds->sms), laa::kBwdThreads, bwd_shared<kD>(), s, maps, p);
    if (ce == cudaSuccess && p.splits > 1)
      ce = la_host::launch_pdl(laa::attn_sum_kernel<kD>, static_cast<unsigned>((delta_threads / (H / HK) + laa::kDeltaThreads - 1) / laa::kDeltaThreads),
                               laa::kDeltaThreads, 0, s, p);
    return ce;
  }));
}

la_status la_attn_verify_workspace(int B, int T, int H, int HK, int D, size_t* bytes) {
  la_host::g_last_error[0] = '\0';
  if (!bytes) return fail(LA_ERR_INVALID_ARGUMENT, "bytes is null");
  const la_status st = check_heads_of(H, HK, D);
  if (st != LA_OK) return st;
  if (B < 0 || T < 1) return fail(LA_ERR_INVALID_ARGUMENT, "B must be >= 0 and T >= 1 (got %d, %d)", B, T);
  if (H / HK > laa::kTile) return fail(LA_ERR_UNSUPPORTED, "H / HK up to %d is implemented (got %d)", laa::kTile, H / HK);
  if (T > kMostDrafts) return fail(LA_ERR_UNSUPPORTED, "T up to %d is implemented (got %d)", kMostDrafts, T);
  *bytes = la_host::align256(laa::verify_part_bytes(verify_shape(T, H, HK, false, 16, false).rows, D));
  return LA_OK;
}

la_status la_attn_verify(const void* q, const void* k, const void* v, float scale, const void* k_cache,
                         const void* v_cache, const int32_t* cache_lens, const int32_t* page_table,
                         const int64_t* mask, void* o, int64_t ldq, int64_t hsq, int64_t ldk, int64_t hsk, int64_t ldv,
                         int64_t hsv, int64_t ldo, int64_t hso, int64_t kp, int64_t kt, int64_t kh, int64_t vp,
                         int64_t vt, int64_t vh, int64_t ld_table, int B, int T, int H, int HK, int D, int pages,
                         int page_size, int table_width, void* workspace, size_t workspace_bytes, int* dev_error,
                         void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_heads_of(H, HK, D);
  if (st != LA_OK) return st;
  if ((st = check_scale(scale)) != LA_OK) return st;
  if ((st = check_pages(cache_lens, page_table, B, T, HK, pages, page_size, table_width, ld_table)) != LA_OK) return st;
  if (T < 1) return fail(LA_ERR_INVALID_ARGUMENT, "T must be >= 1 (got %d)", T);
  if (mask && T > 64) return fail(LA_ERR_UNSUPPORTED, "a mask has at most 64 tokens (got %d)", T);
  if (H / HK > laa::kTile) return fail(LA_ERR_UNSUPPORTED, "H / HK up to %d is implemented (got %d)", laa::kTile, H / HK);
  if (T > kMostDrafts) return fail(LA_ERR_UNSUPPORTED, "T up to %d is implemented (got %d)", kMostDrafts, T);
  const int64_t tokens = static_cast<int64_t>(B) * T;
  if (tokens > kMostTokens) return fail(LA_ERR_UNSUPPORTED, "B*T too large (%lld)", (long long)tokens);
  if (B == 0) return LA_OK;
  if (!k_cache || !v_cache) return fail(LA_ERR_INVALID_ARGUMENT, "k_cache and v_cache must be non-null");
  if (!la_host::aligned4(dev_error) || reinterpret_cast<uintptr_t>(mask) % 8)
    return fail(LA_ERR_INVALID_ARGUMENT, "mask must be 8-byte and dev_error 4-byte aligned");
  size_t need = 0;
  if ((st = la_attn_verify_workspace(B, T, H, HK, D, &need)) != LA_OK) return st;
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  CacheArg kc{k_cache, pages, page_size, HK, kp, kt, kh, "k_cache"}, vc{v_cache, pages, page_size, HK, vp, vt, vh, "v_cache"};
  RowSpan fin[5];
  if ((st = check_cache(kc, D, &fin[0])) != LA_OK || (st = check_cache(vc, D, &fin[1])) != LA_OK) return st;
  fin[2] = flat(cache_lens, static_cast<uint64_t>(B) * 4, "cache_lens");
  fin[3] = flat(page_table, table_bytes(page_table, B, table_width, ld_table), "page_table");
  fin[4] = flat(mask, mask ? static_cast<uint64_t>(tokens) * 8 : 0, "mask");
  const HeadsArg a[] = {rows(q, ldq, hsq, tokens, H, D, "q"), rows(k, ldk, hsk, tokens, HK, D, "k"),
                        rows(v, ldv, hsv, tokens, HK, D, "v"), rows(o, ldo, hso, tokens, H, D, "o")};
  const RowSpan fout[] = {flat(workspace, need, "workspace"), flat(dev_error, 4, "dev_error")};
  if ((st = check_tensors(a, 4, 1, fin, 5, fout, 2)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  laa::CacheParams p{};
  p.v = in(a[2]), p.o = out(a[3]);
  p.ld_table = ld_table;
  p.cache_lens = cache_lens;
  p.page_table = page_table;
  p.mask = mask;
  p.dev_error = dev_error;
  p.scale = scale;
  p.B = B, p.T = T, p.HK = HK, p.pages = pages, p.page_size = page_size, p.table_width = table_width;
  p.part = workspace;
  const laa::VerifyShape shape = verify_shape(T, H, HK, mask != nullptr, page_size, page_table != nullptr);
  laa::VerifyMaps maps;
  if ((st = encode_heads(&maps.q, a[0], shape.group, shape.per_tile)) != LA_OK ||
      (st = encode_heads(&maps.k, a[1], 1, shape.draft_box)) != LA_OK ||
      (st = encode_heads(&maps.v, a[2], 1, shape.draft_box)) != LA_OK ||
      (st = encode_cache(&maps.k_cache, kc, D, shape.box)) != LA_OK || (st = encode_cache(&maps.v_cache, vc, D, shape.box)) != LA_OK)
    return st;
  const int64_t room = page_table ? static_cast<int64_t>(table_width) * page_size : page_size;
  const int64_t most = static_cast<int64_t>(B) * HK * (shape.q_tiles * ((room + laa::kTile - 1) / laa::kTile) + shape.drafts);
  // one block per SM, and a number that the heads divide where that leaves few SMs out (see laa::PieceWalk)
  int blocks = blocks_for(most, std::min(ds->sms, laa::kVerifyBlocks));
  if (blocks / HK * HK * 16 >= blocks * 15) blocks = blocks / HK * HK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launched(with_dim(D, [&](auto d) {
    constexpr int kD = decltype(d)::value;
    const cudaError_t ce = la_host::launch_pdl(laa::attn_verify_kernel<kD>, blocks, laa::kVerifyThreads, verify_shared<kD>(), s,
                                               maps, p, shape);
    if (ce != cudaSuccess) return ce;
    return la_host::launch_pdl(laa::attn_join_kernel<kD>, dim3(blocks, std::min(laa::kJoinShares, shape.rows)), laa::kJoinThreads,
                               0, s, p, shape);
  }));
}

la_status la_attn_commit(const void* k, const void* v, void* k_cache, void* v_cache, const int32_t* cache_lens,
                         const int32_t* cu_seqlens, const int32_t* accepted_len, const int32_t* path,
                         const int32_t* page_table, int64_t ldk, int64_t hsk, int64_t ldv, int64_t hsv, int64_t kp,
                         int64_t kt, int64_t kh, int64_t vp, int64_t vt, int64_t vh, int64_t ld_table, int B, int T,
                         int HK, int D, int pages, int page_size, int table_width, int* dev_error, void* stream) {
  la_host::g_last_error[0] = '\0';
  la_status st = check_heads_of(HK, HK, D);
  if (st != LA_OK) return st;
  if ((st = check_pages(cache_lens, page_table, B, T, HK, pages, page_size, table_width, ld_table)) != LA_OK) return st;
  if (cu_seqlens && (accepted_len || path))
    return fail(LA_ERR_INVALID_ARGUMENT, "accepted_len and path belong to the fixed-length mode (cu_seqlens null)");
  const int64_t tokens = cu_seqlens ? T : static_cast<int64_t>(B) * T;
  if (tokens > kMostTokens) return fail(LA_ERR_UNSUPPORTED, "B*T too large (%lld)", (long long)tokens);
  if (B == 0 || tokens == 0) return LA_OK;
  if (!k_cache || !v_cache) return fail(LA_ERR_INVALID_ARGUMENT, "k_cache and v_cache must be non-null");
  if (!la_host::aligned4(dev_error) || !la_host::aligned4(cu_seqlens) || !la_host::aligned4(accepted_len) || !la_host::aligned4(path))
    return fail(LA_ERR_INVALID_ARGUMENT, "cu_seqlens, accepted_len, path and dev_error must be 4-byte aligned");
  CacheArg kc{k_cache, pages, page_size, HK, kp, kt, kh, "k_cache"}, vc{v_cache, pages, page_size, HK, vp, vt, vh, "v_cache"};
  RowSpan fout[3];
  if ((st = check_cache(kc, D, &fout[0])) != LA_OK || (st = check_cache(vc, D, &fout[1])) != LA_OK) return st;
  fout[2] = flat(dev_error, 4, "dev_error");
  const RowSpan fin[] = {flat(cache_lens, static_cast<uint64_t>(B) * 4, "cache_lens"),
                         flat(cu_seqlens, cu_seqlens ? (static_cast<uint64_t>(B) + 1) * 4 : 0, "cu_seqlens"),
                         flat(accepted_len, accepted_len ? static_cast<uint64_t>(B) * 4 : 0, "accepted_len"),
                         flat(path, path ? static_cast<uint64_t>(tokens) * 4 : 0, "path"),
                         flat(page_table, table_bytes(page_table, B, table_width, ld_table), "page_table")};
  const HeadsArg a[] = {rows(k, ldk, hsk, tokens, HK, D, "k"), rows(v, ldv, hsv, tokens, HK, D, "v")};
  if ((st = check_tensors(a, 2, 0, fin, 5, fout, 3)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  laa::CacheParams p{};
  p.k = in(a[0]), p.v = in(a[1]);
  p.k_out = static_cast<bf16*>(k_cache);
  p.v_out = static_cast<bf16*>(v_cache);
  p.kp = kc.ps, p.kt = kc.ts, p.kh = kc.hs, p.vp = vc.ps, p.vt = vc.ts, p.vh = vc.hs;
  p.ld_table = ld_table;
  p.cache_lens = cache_lens, p.page_table = page_table, p.cu_seqlens = cu_seqlens, p.accepted_len = accepted_len, p.path = path;
  p.dev_error = dev_error;
  p.B = B, p.T = T, p.HK = HK, p.D = D, p.pages = pages, p.page_size = page_size, p.table_width = table_width;
  // blocks of a request: its tokens (packed: their number is on the device, so at most what a batch
  // of one would take, and few enough that the empty ones cost little)
  const int64_t most = (T + laa::kCommitTokens - 1) / laa::kCommitTokens;
  const int64_t share = std::max<int64_t>(1, 16 * ds->sms / B);
  const int tiles = static_cast<int>(std::min<int64_t>(std::min<int64_t>(most, cu_seqlens ? share : most), 65535));
  return launched(la_host::launch_pdl(laa::commit_kernel, dim3(B, tiles), laa::kCommitThreads, 0,
                                      static_cast<cudaStream_t>(stream), p));
}

}  // extern "C"
