// la_gated_api.cu -- host side of the C ABI declared in include/la_gated.h: argument validation,
// the workspace layout and the launches.  Nothing here allocates device memory, reads device
// memory or synchronises with the host.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/la_gated.h"
#include "la_gated_kernels.cuh"
#include "la_host_common.h"
#include "la_rows_common.h"

namespace {

using la_host::fail;
using la_host::RowSpan;

la_host::DeviceState g_dev[la_host::kMaxDevices];

// How a scan is cut, and its device workspace: the ticket, each tile's place among the sequences or
// the sequences' order (packed), the published runs and states; for the gradients one row of
// partial sums of dslopes per chain or tile.
struct Plan {
  int tiles = 0, columns = 0, stride = 0, group = 0, groups = 0, spans = 0, per = 0, parts = 0, longest = -1;
  int items = 0;       // tiles or chains, times columns
  bool ticket = false; // a plan kernel runs first
  bool waits = false;  // states pass from block to block
  bool order = false;  // packed, by chains: the sequences of at most `longest` tokens
  bool table = false;  // packed, by tiles of one sequence each: the others
  lag::Mode mode = lag::kMixed;
  size_t order_at = 0, list = 0, runs = 0, words = 0, before = 0, part = 0, bytes = 0;
};

// Blocks the largest part holds at once; a device with fewer SMs runs the same plan.
constexpr int kSlots = 152 * 2;

// Tiles of a group.  A scan is a chain of one step per group (1.4 us each), while a tile composes
// half a group of published runs.  `streams`: the sequences' columns, so kSlots / streams tiles of one
// are computed at once.  Many streams hide the steps, and a run per warp costs nothing; few want whole
// rounds of blocks in one group.  BF16 forward of one sequence, groups of 8, 40, 56, 96, 128 tiles:
// 512 channels 455, 374, 361, 350, 344 us; 1024: 367, 319, 312, 310, 314; 2048: 303, 279, 278, 289,
// 296; 4096: 240, 250, 255, 268, 282.
int group_of(int64_t streams, int warps) {
  const int64_t wide = 4 * kSlots / streams;
  return wide < 24 ? warps : wide < 160 ? static_cast<int>(wide) : 160;
}

// Whether blocks take whole chains (a sequence's channels).  Sequences of one length: for short
// chains, which need no plan kernel, and where the chains fill the device evenly enough.  2 x 8192
// tokens, BF16, by chains and by tiles: 8704 channels, 272 chains, 205 and 215 us (gradients 390 and 403);
// 8192, 256 chains, 195 and 203 (389 and 380); 7168, 224 chains, 205 and 180 (385 and 336); 3 x 4096
// tokens of 8192 channels, 384 chains, 170 and 154 (306 and 288).  FP32 rows gain less by chains (2 x
// 4096 tokens, 8192 channels 172 and 163, 366 and 338).
bool by_chains(int64_t chains, int per) {
  const int64_t waves = (chains + kSlots - 1) / kSlots;
  return per <= 4 || chains * 100 >= waves * kSlots * 80;
}
// Packed: by chains where there are enough of them to fill the device evenly and the sequences are
// not mostly shorter than half a tile.  By chains, in tiles of one sequence each, and in tiles of
// mixed rows, forward, us: 32 sequences of up to 4096 tokens, 4096 channels, 2048 chains: 327, 404,
// 514; 640 chains: 223, 233, 392 (40 sequences of up to 8192 tokens, 1024 channels), uneven ones 415,
// 238, 334 (20 of 50 to 16384 tokens, 2048 channels); 16 of up to 8192 tokens, 1024 channels, 256
// chains: 196, 122, 186.  2048 channels, 38400 tokens (the bytes are 93): 200 sequences 136, 196, 257; 600
// 211, 284, 239; 1200 417, 532, 246 (gradients, 185: 229, 317, 490; 308, 405, 492; 437, 542, 449).  By chains,
// warps past a sequence's end load and compute rows that nobody uses; in mixed tiles every lane searches
// cu_seqlens, for each of the columns anew.
bool packed_by_chains(int64_t tokens, int N, int columns, int stride) {
  return static_cast<int64_t>(N) * columns >= 3 * kSlots && tokens * 2 >= static_cast<int64_t>(N) * stride;
}
// A batch by chains takes sequences much longer than a block's share of the rows by tiles, in a launch
// of its own behind.  One sequence of 32768 tokens among 100 of 330 on average, 4096 channels: 453 us,
// all by chains 800 (gradients 811, 1532); one of 100000, 512 channels: 200 and 2316.  Without such
// sequences the launch costs 3 to 5 us.
int longest_chain(int64_t tokens, int columns, int stride) {
  const int64_t share = tokens * columns / kSlots;
  return static_cast<int>(std::min<int64_t>(std::max<int64_t>(share + share / 4, 4 * stride), INT32_MAX - 1));
}
// Else in tiles of one sequence each, where those are not mostly single tiles.  128 channels, 400
// sequences of up to 128, 256, 384 and 512 tokens, tiles of 128 rows forward and 72 back: in tiles of
// one sequence 51, 51, 57, 70 us, in mixed ones 23, 32, 43, 59; gradients 48, 58, 72, 84 and 35, 56, 82, 108.
bool packed_by_tiles(int64_t tokens, int N, int stride) { return tokens * 2 >= static_cast<int64_t>(N) * stride * 3; }

template <typename E, bool kBack, bool kTma>
Plan plan_for(int B, int T, int N, int C, bool packed) {
  using S = lag::Shape<E, kBack, kTma, lag::kByTiles>;  // and kMixed
  Plan q;
  if (N == 0) return q;
  const int64_t rows = static_cast<int64_t>(B) * T;
  q.stride = S::kTileRows;
  q.columns = (C + lag::kCols - 1) / lag::kCols;
  if (!packed && T > 0 && T <= q.stride) {  // tiles of whole sequences
    q.stride = q.stride / T * T;
  } else if (!packed && T > 0) {
    q.per = (T + q.stride - 1) / q.stride;
    q.waits = !by_chains(static_cast<int64_t>(B) * q.columns, q.per);
  } else if (packed && N <= lag::kMostListed) {
    q.order = packed_by_chains(rows, N, q.columns, q.stride);
    if (q.order) q.longest = longest_chain(rows, q.columns, q.stride);
  }
  // sequences of the table, at most
  const int64_t listed = !packed || N > lag::kMostListed ? 0 : q.order ? std::min<int64_t>(N, rows / (q.longest + 1)) : N;
  q.table = q.order ? listed > 0 : listed > 0 && packed_by_tiles(rows, N, q.stride);
  q.waits = q.waits || q.table || (packed && !q.order);
  q.ticket = q.waits || q.order;
  if (q.order || (q.per && !q.waits)) q.mode = lag::kByChains;
  else if (q.per || q.table) q.mode = lag::kByTiles;
  q.tiles = q.per ? B * q.per : static_cast<int>(q.table ? rows / q.stride + listed : (rows + q.stride - 1) / q.stride);
  if (q.tiles == 0) q.tiles = 1;  // empty sequences alone
  q.parts = (q.mode == lag::kByChains ? N : 0) + (q.mode != lag::kByChains || q.table ? q.tiles : 0);
  q.items = (q.mode == lag::kByChains ? N : q.tiles) * q.columns;
  const int64_t side_by_side = q.order ? 1 : q.mode == lag::kByTiles ? N : 1;
  q.group = group_of(side_by_side * q.columns, S::kWarps);
  q.groups = ((q.per ? q.per : q.tiles) + q.group - 1) / q.group;
  q.spans = q.per ? B * q.groups : q.groups + (q.table ? static_cast<int>(listed) : 0);
  if (q.ticket) {
    q.order_at = 256;
    q.list = q.order_at + (q.order ? la_host::align256(static_cast<size_t>(N) * sizeof(int32_t)) : 0);
    const size_t list = q.table ? q.tiles * sizeof(lag::Tile) : packed ? (static_cast<size_t>(q.tiles) + 1) * sizeof(int2) : 0;
    q.bytes = q.list + la_host::align256(list);
  }
  if (q.waits) {
    const size_t width = static_cast<size_t>(q.columns) * lag::kCols;
    q.runs = q.bytes;
    q.before = q.runs + q.tiles * width * 8;
    q.words = q.tiles * width * 2 + q.spans * width;
    q.bytes = q.runs + la_host::align256(q.words * 4);
  }
  q.part = q.bytes;
  if (kBack) q.bytes += la_host::align256(static_cast<size_t>(q.parts) * C * 4);
  return q;
}

// The workspace a call needs, whether or not its rows can be read by TMA.
template <typename E, bool kBack>
size_t workspace_for(int B, int T, int N, int C, bool packed) {
  const size_t a = plan_for<E, kBack, true>(B, T, N, C, packed).bytes, b = plan_for<E, kBack, false>(B, T, N, C, packed).bytes;
  return a > b ? a : b;
}
size_t workspace_of(int B, int T, int N, int C, bool packed, la_dtype dtype, bool backward) {
  if (dtype == LA_DTYPE_BF16)
    return backward ? workspace_for<__nv_bfloat16, true>(B, T, N, C, packed)
                    : workspace_for<__nv_bfloat16, false>(B, T, N, C, packed);
  return backward ? workspace_for<float, true>(B, T, N, C, packed) : workspace_for<float, false>(B, T, N, C, packed);
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
  // Tiles times columns stay below 2^30 (more than any memory holds), the ticket of a packed batch whose
  // cu_seqlens is refused.  The smallest tiles hold 24 rows (FP32 gradients, unaligned); a packed batch
  // has one more per listed sequence, and a fixed one's hold 12 rows at least on average (T = 25: two).
  if ((static_cast<int64_t>(B) * T / 12 + lag::kMostListed) * ((C + 63) / 64) >= int64_t(1) << 30)
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

template <typename E>
void set_plan(lag::Params<E>* p, const Plan& q, bool backward, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  p->tiles = q.tiles;
  p->columns = q.columns;
  p->stride = q.stride;
  p->group = q.group;
  p->groups = q.groups;
  p->per = q.per;
  if (q.ticket) p->ticket = reinterpret_cast<int*>(ws);
  p->spans = q.spans;
  p->longest = q.longest;
  if (q.order) p->order = reinterpret_cast<int32_t*>(ws + q.order_at);
  if (q.waits) {
    if (q.table) p->table = reinterpret_cast<lag::Tile*>(ws + q.list);
    else if (p->cu_seqlens) p->places = reinterpret_cast<int2*>(ws + q.list);
    p->runs = reinterpret_cast<float4*>(ws + q.runs);
    p->before = reinterpret_cast<float2*>(ws + q.before);
  }
  if (backward) p->part = reinterpret_cast<float*>(ws + q.part);
}

// Whether rows of this stride can be read by TMA boxes / written two channels at a time.
template <typename E>
bool box_rows(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(E) % 16 == 0;
}
template <typename E>
bool pair_rows(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % (2 * sizeof(E)) == 0 && ld % 2 == 0;
}

// Map over a [rows, C] matrix with its row stride: boxes of `box` rows x 64 channels, unswizzled.
template <typename E>
la_status encode_rows_map(CUtensorMap* map, const E* base, int64_t rows, int64_t C, int64_t ld, int box) {
  auto enc = la_host::tensor_map_encoder();
  if (!enc) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the CUDA driver");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * sizeof(E)};
  const cuuint32_t boxes[2] = {lag::kCols, static_cast<cuuint32_t>(box)}, steps[2] = {1, 1};
  const CUresult r = enc(map, sizeof(E) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                         const_cast<E*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(LA_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d", (int)r);
  return LA_OK;
}

template <typename E>
cudaError_t launch_plan(const lag::Params<E>& p, const Plan& q, int sms, cudaStream_t s) {
  size_t want = q.words / 4;
  if (q.order || q.table) want = std::max(want, static_cast<size_t>(std::max(p.N, q.table ? q.tiles : 0)) * 32);
  want = (want + lag::kThreads - 1) / lag::kThreads;
  const unsigned grid = static_cast<unsigned>(want < 1 ? 1 : want < size_t(sms) * 8 ? want : size_t(sms) * 8);
  return la_host::launch_pdl(lag::scan_plan_kernel<E>, grid, lag::kThreads, 0, s, p);
}

template <typename E, bool kBack, bool kTma, lag::Mode kMode>
la_status launch_mode(const lag::Params<E>& p, int64_t items, int sms, cudaStream_t s) {
  using S = lag::Shape<E, kBack, kTma, kMode>;
  lag::Params<E> with = p;
  if (kMode == lag::kByChains) with.stride = S::kTileRows;
  if (kMode == lag::kByTiles && p.table) with.ticket += lag::kTicket;
  lag::Maps maps;
  if constexpr (kTma) {
    for (int i = 0; i < S::kInputs; ++i) {
      const la_status st = encode_rows_map(&maps.of[i], p.in[i], p.rows, p.C, p.ld_in[i], S::kRows);
      if (st != LA_OK) return st;
    }
  }
  const int64_t most = static_cast<int64_t>(sms) * S::kBlocks;
  const cudaError_t ce = la_host::launch_pdl(lag::gated_scan_kernel<E, kBack, kTma, kMode>,
                                             static_cast<unsigned>(items < most ? items : most), S::kThreads,
                                             lag::scan_smem_bytes<E, kBack, kTma, kMode>(), s, with, maps);
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

template <typename E, bool kBack, bool kTma>
la_status launch_scan_as(lag::Params<E> p, int B, void* workspace, float* dslopes, int sms, cudaStream_t s) {
  const bool packed = p.cu_seqlens != nullptr;
  const Plan q = plan_for<E, kBack, kTma>(B, p.T, p.N, p.C, packed);
  set_plan(&p, q, kBack, workspace);
  cudaError_t ce = q.ticket ? launch_plan(p, q, sms, s) : cudaSuccess;
  la_status st = LA_OK;
  if (ce == cudaSuccess && q.tiles > 0) {
    if (q.mode == lag::kByChains) st = launch_mode<E, kBack, kTma, lag::kByChains>(p, q.items, sms, s);
    else if (q.mode == lag::kMixed) st = launch_mode<E, kBack, kTma, lag::kMixed>(p, q.items, sms, s);
    if (st == LA_OK && (q.table || q.mode == lag::kByTiles))
      st = launch_mode<E, kBack, kTma, lag::kByTiles>(p, static_cast<int64_t>(q.tiles) * q.columns, sms, s);
  }
  if (st != LA_OK) return st;
  if (ce == cudaSuccess && kBack)
    ce = la_host::launch_pdl(lag::column_sum_kernel, (p.C + 31) / 32, 1024, 0, s, static_cast<const float*>(p.part),
                             q.parts, p.C, static_cast<const int*>(packed ? p.ticket : nullptr), q.order || q.table, dslopes);
  return ce == cudaSuccess ? LA_OK : fail(LA_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(ce));
}

template <typename E, bool kBack>
la_status launch_scan(const lag::Params<E>& p, int B, void* workspace, float* dslopes, int sms, cudaStream_t s) {
  bool tma = p.rows > 0;
  for (int i = 0; i < (kBack ? 5 : 3); ++i) tma = tma && box_rows<E>(p.in[i], p.ld_in[i]);
  for (int i = 0; i < (kBack ? 3 : 1); ++i) tma = tma && p.C % 2 == 0 && pair_rows<E>(p.out[i], p.ld_out[i]);
  return tma ? launch_scan_as<E, kBack, true>(p, B, workspace, dslopes, sms, s)
             : launch_scan_as<E, kBack, false>(p, B, workspace, dslopes, sms, s);
}

// One-time setup per device: the stages of a scan exceed the default shared memory.
template <typename E, bool kBack, bool kTma, lag::Mode kMode>
cudaError_t setup_kernel() {
  return cudaFuncSetAttribute(lag::gated_scan_kernel<E, kBack, kTma, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              lag::scan_smem_bytes<E, kBack, kTma, kMode>());
}
template <typename E, bool kBack, bool kTma>
cudaError_t setup_modes() {
  cudaError_t e = setup_kernel<E, kBack, kTma, lag::kByChains>();
  if (e == cudaSuccess) e = setup_kernel<E, kBack, kTma, lag::kByTiles>();
  if (e == cudaSuccess) e = setup_kernel<E, kBack, kTma, lag::kMixed>();
  return e;
}
template <typename E>
cudaError_t setup_type() {
  cudaError_t e = setup_modes<E, false, false>();
  if (e == cudaSuccess) e = setup_modes<E, false, true>();
  if (e == cudaSuccess) e = setup_modes<E, true, false>();
  if (e == cudaSuccess) e = setup_modes<E, true, true>();
  return e;
}

la_status device(la_host::DeviceState** ds) {
  return la_host::current_device(g_dev, ds, [] {
    const cudaError_t e = setup_type<__nv_bfloat16>();
    return e == cudaSuccess ? setup_type<float>() : e;
  });
}

template <typename E>
lag::Params<E> params_of(const void* x, const void* r, const void* g, const float* slopes, int64_t ldx, int64_t ldr,
                         int64_t ldg, const int32_t* state_indices, int* dev_error, int T, int N, int C,
                         int pool_size) {
  lag::Params<E> p{};
  p.in[0] = static_cast<const E*>(x);
  p.in[1] = static_cast<const E*>(r);
  p.in[2] = static_cast<const E*>(g);
  p.ld_in[0] = ldx;
  p.ld_in[1] = ldr;
  p.ld_in[2] = ldg;
  p.slopes = slopes;
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
    p.out[0] = static_cast<E*>(o);
    p.ld_out[0] = ldo;
    p.start = state;
    p.finish = state_out;
    p.accepted_len = accepted_len;
    auto quads = [&](const void* ptr, int64_t ld, size_t element) {
      return reinterpret_cast<uintptr_t>(ptr) % (4 * element) == 0 && ld % 4 == 0;
    };
    const bool wide = C % 4 == 0 && quads(x, ldx, es) && quads(r, ldr, es) && quads(g, ldg, es) && quads(o, ldo, es) &&
                      quads(slopes, 0, 4) && quads(state, 0, 4);
    const int span = lag::kThreads * (wide ? 4 : 2);
    const unsigned grid = static_cast<unsigned>(B) * ((C + span - 1) / span);
    cudaError_t ce = la_host::launch_pdl(wide ? lag::gated_decode_kernel<E, 4> : lag::gated_decode_kernel<E, 1>, grid,
                                         lag::kThreads, 0, static_cast<cudaStream_t>(stream), p);
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
  *bytes = workspace_of(B, T, N, C, packed != 0, dtype, backward != 0);
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
  const size_t need = workspace_of(B, T, N, C, cu_seqlens != nullptr, dtype, false);
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  const RowSpan ins[] = {la_host::rows_of(x, ldx, rows, C, es, "x"),
                         la_host::rows_of(r, ldr, rows, C, es, "r"),
                         la_host::rows_of(g, ldg, rows, C, es, "g"),
                         la_host::flat(slopes, static_cast<uint64_t>(C) * 4, "slopes"),
                         pool_span(h0 == h_final ? nullptr : h0, "h0", state_indices, pool_size, N, C),
                         la_host::flat(state_indices, static_cast<uint64_t>(N) * 4, "state_indices"),
                         la_host::flat(cu_seqlens, static_cast<uint64_t>(N) * 4 + 4, "cu_seqlens")};
  const RowSpan outs[] = {la_host::rows_of(o, ldo, rows, C, es, "o"),
                          pool_span(h_final, "h_final", state_indices, pool_size, N, C),
                          la_host::flat(workspace, need, "workspace"),
                          la_host::flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 7, outs, 4)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    auto p = params_of<E>(x, r, g, slopes, ldx, ldr, ldg, state_indices, dev_error, T, N, C,
                          la_host::effective_pool_size(h0, h_final, state_indices, pool_size, N));
    p.out[0] = static_cast<E*>(o);
    p.ld_out[0] = ldo;
    p.start = h0;
    p.finish = h_final;
    p.cu_seqlens = cu_seqlens;
    p.rows = static_cast<int>(rows);
    return launch_scan<E, false>(p, B, workspace, nullptr, ds->sms, static_cast<cudaStream_t>(stream));
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
  const size_t need = workspace_of(B, T, N, C, cu_seqlens != nullptr, dtype, true);
  if ((st = la_host::check_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
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
                          la_host::flat(workspace, need, "workspace"),
                          la_host::flat(dev_error, 4, "dev_error")};
  if ((st = la_host::check_rows(ins, 10, outs, 7)) != LA_OK) return st;
  la_host::DeviceState* ds = nullptr;
  if ((st = device(&ds)) != LA_OK) return st;
  auto run = [&](auto tag) {
    using E = decltype(tag);
    const int pool = states ? pool_size : state_indices ? INT32_MAX : N;
    auto p = params_of<E>(x, r, g, slopes, ldx, ldr, ldg, state_indices, dev_error, T, N, C, pool);
    p.in[3] = static_cast<const E*>(dout);
    p.in[4] = static_cast<const E*>(o);
    p.ld_in[3] = lddout;
    p.ld_in[4] = ldo;
    p.out[0] = static_cast<E*>(dx);
    p.out[1] = static_cast<E*>(dr);
    p.out[2] = static_cast<E*>(dg);
    p.ld_out[0] = lddx;
    p.ld_out[1] = lddr;
    p.ld_out[2] = lddg;
    p.start = dh_final;
    p.finish = dh0;
    p.h0 = h0;
    p.cu_seqlens = cu_seqlens;
    p.rows = static_cast<int>(rows);
    return launch_scan<E, true>(p, B, workspace, dslopes, ds->sms, static_cast<cudaStream_t>(stream));
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
