// attention.cu -- prompt attention and shared-prefix decode attention: the C
// ABI of include/dsa_attention.h. The kernel is in attend.cuh; here are the
// checks of arguments, the tensor maps, the workspace and the launches.
#include "../../include/dsa_attention.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attend.cuh"

namespace dsa {
namespace {

constexpr int kMaxHeadDim = 128;
constexpr int kMaxGroup = 128;
constexpr float kLog2e = 1.4426950408889634f;

int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? dev : -1;
}

// Streaming multiprocessors of the current device, cached per device.
int sm_count() {
  static std::atomic<int> cached[64];
  const int dev = current_device();
  if (dev < 0) return 152;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      return 152;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// The driver's encoder of tensor maps (a host function; looked up once).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn fn = cached.load(std::memory_order_relaxed);
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      return nullptr;
    fn = reinterpret_cast<EncodeFn>(p);
    cached.store(fn, std::memory_order_relaxed);
  }
  return fn;
}

// A map of rank `n` over 16-bit elements; strides (of dimensions 1...) in
// elements; boxes are [64 elements] x box[1...], swizzled by 128 bytes, and
// read zeros outside the tensor.
template <int N>
bool encode(CUtensorMap* map, int32_t dtype, const void* base, const int64_t (&dims)[N],
            const int64_t (&strides)[N - 1], const int (&box)[N]) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  cuuint64_t d[N], st[N - 1];
  cuuint32_t b[N], one[N];
  // Misses fetch aligned pieces of this many bytes: no more than a row of one
  // head is made of. With 256 for every layout a head dimension of 80 read
  // 1070 MB where the rows hold 547 (33 sequences, 8 heads of 160 bytes).
  uint64_t whole = reinterpret_cast<uintptr_t>(base) | static_cast<uint64_t>(dims[0]) * 2 | 256;
  for (int i = 0; i < N; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    one[i] = 1;
    if (i > 0) st[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
    if (i > 0) whole |= st[i - 1];
  }
  const CUtensorMapL2promotion fetch = whole % 256 == 0   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : whole % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                       : whole % 64 == 0  ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                                          : CU_TENSOR_MAP_L2_PROMOTION_NONE;
  return fn(map,
            dtype == DSA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            N, const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, fetch,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q1: boxes of one token (paged calls only).
struct Maps {
  CUtensorMap q, q1, k, v;
};

template <typename T, int DP, bool PAGED>
dsa_status launch(const Maps& m, const AttendArgs& a, int grid, cudaStream_t stream) {
  constexpr size_t kSmem = attend_smem(Layout<DP>::kCtrl);
  static_assert(kSmem <= 232448, "shared memory of one SM");
  static std::atomic<bool> ready[64];  // per device
  const int dev = current_device();
  if (dev < 0) return DSA_ECUDA;
  auto* kernel = attend_kernel<T, DP, PAGED>;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmem)) != cudaSuccess)
      return DSA_ECUDA;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  kernel<<<grid, kAttendThreads, kSmem, stream>>>(m.q, m.q1, m.k, m.v, a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

template <bool PAGED>
dsa_status launch(const Maps& m, const AttendArgs& a, int32_t dtype, int grid,
                  cudaStream_t stream) {
  if (dtype == DSA_DTYPE_BF16)
    return a.dim > 64 ? launch<__nv_bfloat16, 128, PAGED>(m, a, grid, stream)
                      : launch<__nv_bfloat16, 64, PAGED>(m, a, grid, stream);
  return a.dim > 64 ? launch<__half, 128, PAGED>(m, a, grid, stream)
                    : launch<__half, 64, PAGED>(m, a, grid, stream);
}

template <typename T>
dsa_status launch_join(const AttendArgs& a, const JoinArgs& j, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.tokens * a.heads + kJoinWarps - 1) / kJoinWarps));
  const bool ok = a.dim > 64
                      ? launch_after(join_kernel<T, 128>, grid, kJoinWarps * 32, stream, a, j)
                      : launch_after(join_kernel<T, 64>, grid, kJoinWarps * 32, stream, a, j);
  return ok ? DSA_OK : DSA_ECUDA;
}

template <typename T>
bool launch_join_blocks(const AttendArgs& a, unsigned grid, cudaStream_t stream) {
  const dim3 ctas(grid, (a.dim + kJoinCols - 1) / kJoinCols);
  return a.dim > 64 ? launch_after(join_blocks_kernel<T, 128>, ctas, kJoinRows, stream, a)
                    : launch_after(join_blocks_kernel<T, 64>, ctas, kJoinRows, stream, a);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// How a prompt call's work is dealt, and where its partial outputs lie in the
// workspace (each part 256-byte aligned).
struct PromptPlan {
  int32_t tile_tokens;
  int cut, grid;
  bool fits;  // blocks within 32 bits
  size_t cuts, part_o, part_lse, bytes;
};

// Blocks are cut where the batch has more than kCutKeys keys and kCutMean on
// average for a sequence, or more than kCutBatch. Cut / whole, us (32 query
// heads, 8 key/value heads, causal, head dimension 128): 1024 keys 25.0 / 20.0;
// 2048 keys 42.7 / 53.1; one query on 1500 keys 17.2 / 22.3; 8 x 512 keys 41.6
// / 41.3 (8 query heads on 2: 21.4 / 15.0); 4 x 800 41.8 / 40.9; 4 x 1024 54.0 /
// 60.6; 80 x 100 51.7 / 49.0; 2500, 10 and 900 keys 62.9 / 88.8 (8 query heads
// on 2: 29.4 / 34.8). The lengths themselves are on the device: a mean says
// nothing of a batch in which one sequence has most of the keys and the others
// few, and there whole blocks lose (full attention, 128 heads on 8, queries
// 1060, 3357, 175, 2 on keys 2, 173, 2632, 12: 127 / 469).
constexpr int64_t kCutKeys = 1400, kCutMean = 800, kCutBatch = 8192;

PromptPlan plan_prompt(int64_t total_q, int64_t total_k, int32_t heads, int32_t kv_heads,
                       int32_t head_dim, int32_t seqs) {
  PromptPlan p{};
  p.tile_tokens = kTile / (heads / kv_heads);
  // No more blocks than this, whatever the offsets hold.
  const int64_t blocks = (total_q / (2 * p.tile_tokens) + seqs) * kv_heads;
  const int64_t sms = sm_count();
  p.fits = blocks <= INT32_MAX;
  p.cut = (total_k > kCutKeys && total_k > kCutMean * seqs) || total_k > kCutBatch;
  // A block is cut at most into its key tiles.
  const int64_t most = p.cut ? sms : blocks;
  p.grid = static_cast<int>(most < sms ? most : sms);
  if (!p.cut) return p;
  const size_t slots = 2 * static_cast<size_t>(p.grid), dp = head_dim > 64 ? 128 : 64;
  p.cuts = 0;
  p.part_o = up256(p.grid * sizeof(CutBlock));
  p.part_lse = p.part_o + up256(slots * 256 * dp * 4);
  p.bytes = p.part_lse + up256(slots * 256 * 4);
  return p;
}

// How a paged call's work is cut, and where its partial outputs lie in the
// workspace (each part 256-byte aligned).
struct PagedPlan {
  int32_t tile_tokens, prefix_tiles, prefix_blocks, prefix_split;
  int grid;
  bool fits;  // units, slots and CTAs of the join within 32 bits
  size_t starts, prefix_o, prefix_lse, own_o, own_lse, bytes;
};

PagedPlan plan_paged(int64_t batch, int32_t heads, int32_t kv_heads, int32_t head_dim,
                     int64_t prefix_len, int64_t max_pages, int32_t page_size) {
  PagedPlan p{};
  const int32_t group = heads / kv_heads;
  const size_t dp = head_dim > 64 ? 128 : 64;
  p.tile_tokens = kTile / group;
  // One row tile holds the batch: its stream would be alone with the prefix,
  // so two streams take alternate key tiles instead.
  p.prefix_split = batch <= p.tile_tokens;
  const int64_t block = (p.prefix_split ? 1 : 2) * static_cast<int64_t>(p.tile_tokens);
  p.prefix_tiles = static_cast<int32_t>((prefix_len + kTile - 1) / kTile);
  p.prefix_blocks = static_cast<int32_t>((batch + block - 1) / block);
  const int64_t groups = static_cast<int64_t>(kv_heads) * p.prefix_blocks;
  const int64_t own_tiles = (max_pages * page_size - prefix_len + kTile - 1) / kTile;
  const int64_t most = groups * p.prefix_tiles + batch * kv_heads * own_tiles;
  p.fits = most <= INT32_MAX / (kTwoTileCost + kSegCost) - 1024 &&
           batch * heads <= static_cast<int64_t>(kJoinWarps) * INT32_MAX;
  const int64_t sms = sm_count();
  p.grid = static_cast<int>(most < 1 ? 1 : (most < sms ? most : sms));
  const size_t pslots = p.prefix_tiles > 0 ? groups + p.grid : 0;
  const size_t oslots = own_tiles > 0 ? batch * kv_heads + p.grid : 0;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t was = at;
    at += up256(n);
    return was;
  };
  p.starts = take((batch + 1) * 4);
  p.prefix_o = take(pslots * 256 * dp * 4);
  p.prefix_lse = take(pslots * 256 * 4);
  p.own_o = take(oslots * 2 * group * dp * 4);
  p.own_lse = take(oslots * 2 * group * 4);
  p.bytes = at;
  return p;
}

// Sizes and scale that both operators share.
dsa_status check_common(int32_t dtype, int64_t tokens, int32_t heads, int32_t kv_heads,
                        int32_t head_dim, float scale) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (tokens < 0 || heads < 0 || kv_heads < 1 || heads % kv_heads != 0 || head_dim < 1)
    return DSA_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale * kLog2e)) return DSA_EINVAL;
  if (dtype == DSA_DTYPE_F32 || head_dim > kMaxHeadDim || head_dim % 8 != 0 ||
      heads / kv_heads > kMaxGroup || tokens > INT32_MAX)
    return DSA_EUNSUPPORTED;
  return DSA_OK;
}

dsa_status check_pages(int64_t num_pages, int32_t page_size, int64_t max_pages,
                       int64_t prefix_len) {
  if (num_pages < 0 || page_size < 1 || max_pages < 0 || prefix_len < 0) return DSA_EINVAL;
  if (num_pages > INT32_MAX || max_pages > INT32_MAX || page_size < 16 ||
      (page_size & (page_size - 1)) != 0 || max_pages * page_size > INT32_MAX)
    return DSA_EUNSUPPORTED;
  return prefix_len % page_size != 0 || prefix_len > max_pages * page_size ? DSA_EINVAL : DSA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool by8(int64_t a, int64_t b = 0, int64_t c = 0) {
  return a % 8 == 0 && b % 8 == 0 && c % 8 == 0 && a >= 0 && b >= 0 && c >= 0;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_prompt_attention(
    const void* q, const void* k, const void* v, int32_t dtype, int64_t total_q, int64_t total_k,
    int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t q_st, int64_t q_sh, int64_t k_st,
    int64_t k_sh, int64_t v_st, int64_t v_sh, const int32_t* cu_q, const int32_t* cu_k,
    int32_t seqs, int32_t causal, float scale, void* out, int64_t o_st, int64_t o_sh, float* lse,
    int64_t l_st, int64_t l_sh, void* workspace, size_t workspace_bytes, void* stream) {
  if (total_k < 0 || seqs < 0) return DSA_EINVAL;
  const dsa_status st = dsa::check_common(dtype, total_q, heads, kv_heads, head_dim, scale);
  if (st != DSA_OK) return st;
  if (total_k > INT32_MAX - 4096) return DSA_EUNSUPPORTED;
  if (total_q == 0 || heads == 0 || seqs == 0) return DSA_OK;
  if (!q || !out || !cu_q || !cu_k || (total_k > 0 && (!k || !v))) return DSA_EINVAL;
  if (!dsa::aligned16(q) || !dsa::aligned16(k) || !dsa::aligned16(v) || !dsa::aligned16(out) ||
      !dsa::by8(q_st, q_sh) || !dsa::by8(k_st, k_sh) || !dsa::by8(v_st, v_sh) ||
      !dsa::by8(o_st, o_sh))
    return DSA_EUNSUPPORTED;
  const dsa::PromptPlan p = dsa::plan_prompt(total_q, total_k, heads, kv_heads, head_dim, seqs);
  if (!p.fits) return DSA_EUNSUPPORTED;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes ||
                      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return DSA_EINVAL;
  dsa::AttendArgs a{};
  a.cut = p.cut;
  if (p.cut) {
    char* ws = static_cast<char*>(workspace);
    a.cuts = reinterpret_cast<dsa::CutBlock*>(ws + p.cuts);
    a.prefix_o = reinterpret_cast<float*>(ws + p.part_o);
    a.prefix_lse = reinterpret_cast<float*>(ws + p.part_lse);
  }
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_st = q_st;
  a.q_sh = q_sh;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.dim = head_dim;
  a.tile_tokens = p.tile_tokens;
  a.c = scale * dsa::kLog2e;
  a.tokens = total_q;
  a.total_k = total_k;
  a.k_st = k_st;
  a.k_sh = k_sh;
  a.v_st = v_st;
  a.v_sh = v_sh;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.seqs = seqs;
  a.causal = causal != 0;
  a.out = out;
  a.o_st = o_st;
  a.o_sh = o_sh;
  a.lse = lse;
  a.l_st = l_st;
  a.l_sh = l_sh;
  dsa::Maps m;
  if (!dsa::encode<3>(&m.q, dtype, q, {head_dim, heads, total_q}, {q_sh, q_st},
                      {64, a.group, a.tile_tokens}))
    return DSA_EUNSUPPORTED;
  m.q1 = m.k = m.v = m.q;  // without keys nothing is loaded through these
  if (total_k > 0 &&
      (!dsa::encode<3>(&m.k, dtype, k, {head_dim, kv_heads, total_k}, {k_sh, k_st},
                       {64, 1, dsa::kTile}) ||
       !dsa::encode<3>(&m.v, dtype, v, {head_dim, kv_heads, total_k}, {v_sh, v_st},
                       {64, 1, dsa::kTile})))
    return DSA_EUNSUPPORTED;
  cudaStream_t strm = static_cast<cudaStream_t>(stream);
  const dsa_status done = dsa::launch<false>(m, a, dtype, p.grid, strm);
  if (done != DSA_OK || !p.cut) return done;
  const bool ok = dtype == DSA_DTYPE_BF16
                      ? dsa::launch_join_blocks<__nv_bfloat16>(a, p.grid, strm)
                      : dsa::launch_join_blocks<__half>(a, p.grid, strm);
  return ok ? DSA_OK : DSA_ECUDA;
}

extern "C" size_t dsa_prompt_workspace_bytes(int64_t total_q, int64_t total_k, int32_t heads,
                                             int32_t kv_heads, int32_t head_dim, int32_t seqs) {
  if (dsa::check_common(DSA_DTYPE_BF16, total_q, heads, kv_heads, head_dim, 1.f) != DSA_OK ||
      total_k < 0 || total_k > INT32_MAX || seqs < 0 || total_q == 0 || heads == 0 || seqs == 0)
    return 0;
  return dsa::plan_prompt(total_q, total_k, heads, kv_heads, head_dim, seqs).bytes;
}

extern "C" size_t dsa_shared_prefix_workspace_bytes(int64_t batch, int32_t heads,
                                                    int32_t kv_heads, int32_t head_dim,
                                                    int64_t prefix_len, int64_t max_pages,
                                                    int32_t page_size) {
  if (dsa::check_common(DSA_DTYPE_BF16, batch, heads, kv_heads, head_dim, 1.f) != DSA_OK ||
      dsa::check_pages(0, page_size, max_pages, prefix_len) != DSA_OK || batch == 0 || heads == 0)
    return 0;
  return dsa::plan_paged(batch, heads, kv_heads, head_dim, prefix_len, max_pages, page_size).bytes;
}

extern "C" dsa_status dsa_shared_prefix_attention(
    const void* q, const void* k_pages, const void* v_pages, int32_t dtype, int64_t batch,
    int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t num_pages, int32_t page_size,
    int64_t q_sb, int64_t q_sh, int64_t k_sn, int64_t k_st, int64_t k_sh, int64_t v_sn,
    int64_t v_st, int64_t v_sh, const int32_t* prefix_pages, int64_t prefix_len,
    const int32_t* tables, int64_t max_pages, int64_t ld_tables, const int32_t* lens, float scale,
    void* out, int64_t o_sb, int64_t o_sh, float* lse, int64_t l_sb, int64_t l_sh,
    void* workspace, size_t workspace_bytes, void* stream) {
  if (ld_tables < max_pages) return DSA_EINVAL;
  dsa_status st = dsa::check_common(dtype, batch, heads, kv_heads, head_dim, scale);
  if (st != DSA_OK) return st;
  st = dsa::check_pages(num_pages, page_size, max_pages, prefix_len);
  if (st != DSA_OK) return st;
  if (batch == 0 || heads == 0) return DSA_OK;
  if (!q || !out || !lens || (max_pages > 0 && !tables) || (prefix_len > 0 && !prefix_pages) ||
      (num_pages > 0 && (!k_pages || !v_pages)))
    return DSA_EINVAL;
  if (!dsa::aligned16(q) || !dsa::aligned16(k_pages) || !dsa::aligned16(v_pages) ||
      !dsa::aligned16(out) || !dsa::by8(q_sb, q_sh) || !dsa::by8(k_sn, k_st, k_sh) ||
      !dsa::by8(v_sn, v_st, v_sh) || !dsa::by8(o_sb, o_sh))
    return DSA_EUNSUPPORTED;
  const dsa::PagedPlan p =
      dsa::plan_paged(batch, heads, kv_heads, head_dim, prefix_len, max_pages, page_size);
  if (!p.fits) return DSA_EUNSUPPORTED;
  if (!workspace || workspace_bytes < p.bytes ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return DSA_EINVAL;
  char* ws = static_cast<char*>(workspace);
  dsa::AttendArgs a{};
  a.q = q;
  a.k = k_pages;
  a.v = v_pages;
  a.q_st = q_sb;
  a.q_sh = q_sh;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.dim = head_dim;
  a.tile_tokens = p.tile_tokens;
  a.c = scale * dsa::kLog2e;
  a.tokens = batch;
  a.k_st = k_st;
  a.k_sh = k_sh;
  a.v_st = v_st;
  a.v_sh = v_sh;
  a.k_sn = k_sn;
  a.v_sn = v_sn;
  a.num_pages = num_pages;
  a.max_pages = num_pages > 0 ? max_pages : 0;  // without pages nothing is seen
  a.ld_tables = ld_tables;
  a.page_size = page_size;
  while ((1 << a.page_log2) < page_size) ++a.page_log2;
  a.prefix_pages = prefix_pages;
  a.tables = tables;
  a.lens = lens;
  a.prefix_len = prefix_len;
  a.prefix_tiles = num_pages > 0 ? p.prefix_tiles : 0;
  a.prefix_blocks = p.prefix_blocks;
  a.prefix_split = p.prefix_split;
  a.starts = reinterpret_cast<int32_t*>(ws + p.starts);
  a.prefix_o = reinterpret_cast<float*>(ws + p.prefix_o);
  a.prefix_lse = reinterpret_cast<float*>(ws + p.prefix_lse);
  a.own_o = reinterpret_cast<float*>(ws + p.own_o);
  a.own_lse = reinterpret_cast<float*>(ws + p.own_lse);
  dsa::Maps m;
  if (!dsa::encode<3>(&m.q, dtype, q, {head_dim, heads, batch}, {q_sh, q_sb},
                      {64, a.group, a.tile_tokens}) ||
      !dsa::encode<3>(&m.q1, dtype, q, {head_dim, heads, batch}, {q_sh, q_sb}, {64, a.group, 1}))
    return DSA_EUNSUPPORTED;
  m.k = m.v = m.q;
  const int rows = page_size < dsa::kTile ? page_size : dsa::kTile;
  if (num_pages > 0 &&
      (!dsa::encode<4>(&m.k, dtype, k_pages, {head_dim, kv_heads, page_size, num_pages},
                       {k_sh, k_st, k_sn}, {64, 1, rows, 1}) ||
       !dsa::encode<4>(&m.v, dtype, v_pages, {head_dim, kv_heads, page_size, num_pages},
                       {v_sh, v_st, v_sn}, {64, 1, rows, 1})))
    return DSA_EUNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = dsa::launch<true>(m, a, dtype, p.grid, s);
  if (st != DSA_OK) return st;
  const dsa::JoinArgs j{out, o_sb, o_sh, lse, l_sb, l_sh, p.grid};
  return dtype == DSA_DTYPE_BF16 ? dsa::launch_join<__nv_bfloat16>(a, j, s)
                                 : dsa::launch_join<__half>(a, j, s);
}

extern "C" int dsa_attention_error(int clear) {
  unsigned int code = 0;
  // the copies below wait for the default stream alone
  if (cudaDeviceSynchronize() != cudaSuccess) return -1;
  if (cudaMemcpyFromSymbol(&code, dsa::g_pipe_error, sizeof(code)) != cudaSuccess) return -1;
  if (clear && code != 0) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(dsa::g_pipe_error, &zero, sizeof(zero)) != cudaSuccess) return -1;
  }
  return static_cast<int>(code);
}
