// quant_attention.cu -- attention of single tokens over pages of e4m3 codes:
// dsa_quant_attention of include/dsa_quant.h. The kernels are in quant_attend.cuh;
// here are the checks of arguments, the workspace and the launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "quant_attend.cuh"

namespace dsa {
namespace {

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
  return n < 1024 ? n : 1024;  // as many shares as the kernels take
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// How a call's work is cut, and where its partial outputs lie in the workspace
// (each part 256-byte aligned).
struct QuantPlan {
  int32_t dp, columns, splits, split_heads;
  bool whole;
  int64_t grid;
  bool fits;
  size_t spans, part_o, part_lse, bytes;
};

// Warps of a CTA of the attention kernel.
int32_t quant_warps(int columns) {
  return columns == 1 ? QuantLayout<128, 1>::kWarps : QuantLayout<128, 2>::kWarps;
}

// Tiles of all heads; those of the sequences and their starts then stay within 31 bits.
constexpr int64_t kMaxUnits = 250000000;
// Tiles of a row that a CTA of its own still takes, if there is an SM for each row: one
// launch instead of two. Lengths are on the device, so that the room of the table's
// rows decides. 3 sequences with 2 heads of 64, 16 with 2 of 128 and 18 with 8 of 128,
// us, in one launch and in two:
//    4 tiles   5.0 10.9    5.3 9.7    5.4 10.2
//   16         8.1 11.2    8.6 9.7    8.6 11.4
//   32        10.9 11.5   10.4 9.9   12.4 15.4
//   64        18.4 11.6   16.2 12.4  19.6 21.9
// Short sequences in a wide table pay for that: three of about 200 tokens, 2 heads of
// 64, take 4.9 us with room for 1024 tokens, 7.7 for 2048 and 8.3 for 8192.
constexpr int64_t kWholeTiles = 16;

QuantPlan plan_attention(int64_t batch, int32_t heads, int32_t kv_heads, int32_t head_dim,
                         int64_t max_pages, int32_t page_size) {
  QuantPlan p{};
  const int32_t group = heads / kv_heads;
  p.dp = head_dim > 64 ? 128 : 64;
  p.splits = (group + 15) / 16;
  p.split_heads = (group + p.splits - 1) / p.splits;
  p.columns = p.split_heads > 8 ? 2 : 1;
  const int64_t tile = kQuantTileBytes / p.dp;
  const int64_t tiles = (max_pages * page_size + tile - 1) / tile;
  const int64_t rows = batch * kv_heads * p.splits, units = rows * tiles;
  p.fits = batch * kv_heads * ((max_pages * page_size + 31) / 32) <= kMaxUnits;
  const int64_t sms = sm_count();
  p.whole = rows <= sms && tiles <= kWholeTiles;
  if (p.whole) {
    p.grid = rows;
    return p;
  }
  const int64_t warps = quant_warps(p.columns), most = (units + warps - 1) / warps;
  p.grid = most < 1 ? 1 : (most < sms ? most : sms);
  const size_t columns = 2 * static_cast<size_t>(p.grid) * warps * 8 * p.columns;
  p.spans = 0;
  p.part_o = up256(batch * sizeof(int2));
  p.part_lse = p.part_o + up256(columns * p.dp * 4);
  p.bytes = p.part_lse + up256(columns * 4);
  return p;
}

template <int DP, int NT, int TEAM>
bool launch_join(const QuantAttnArgs& a, cudaStream_t stream) {
  const int64_t items = a.batch * a.pool.kv_heads * a.group, each = JoinShape<TEAM>::kWarps / TEAM;
  return launch_after(quant_join_kernel<DP, NT, TEAM>,
                      dim3(static_cast<unsigned>((items + each - 1) / each)),
                      JoinShape<TEAM>::kThreads, stream, a);
}

template <int DP, int NT, int KD>
dsa_status launch(const QuantAttnArgs& a, const QuantPlan& p, cudaStream_t stream) {
  constexpr int kSmem = QuantLayout<DP, NT>::kSmem;
  static_assert(kSmem + 8192 <= 232448, "shared memory of one SM");
  static std::atomic<bool> ready[2][64];  // per device
  const int dev = current_device();
  if (dev < 0) return DSA_ECUDA;
  auto* kernel = p.whole ? quant_attend_row_kernel<DP, NT, KD> : quant_attend_kernel<DP, NT, KD>;
  if (!ready[p.whole][dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
        cudaSuccess)
      return DSA_ECUDA;
    ready[p.whole][dev].store(true, std::memory_order_relaxed);
  }
  kernel<<<static_cast<unsigned>(p.grid), QuantLayout<DP, NT>::kThreads, kSmem, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return DSA_ECUDA;
  if (p.whole) return DSA_OK;
  // A warp has eight pieces of a row under way at once, so that it joins rows of
  // about as many; where there are more, 8 or 32 warps do.
  const int64_t rows = a.batch * a.rows;
  const bool ok = 8 * rows >= a.warps    ? launch_join<DP, NT, 1>(a, stream)
                  : 64 * rows >= a.warps ? launch_join<DP, NT, 8>(a, stream)
                                         : launch_join<DP, NT, 32>(a, stream);
  return ok ? DSA_OK : DSA_ECUDA;
}

// Heads of 80 and 96 multiply no more than they have, which is faster than going
// through products of 128: 33 sequences, 136,000 tokens of 8 heads of 80, take 49.6 us
// instead of 53.2 (5 query heads each) and 60.5 instead of 72.1 (9); of 96, 48.3
// instead of 49.6 (4) and 61.7 instead of 70.0 (16). Heads of 112 go through products
// of 128 (54.9 us; 4).
template <int NT>
dsa_status launch_heads(const QuantAttnArgs& a, const QuantPlan& p, cudaStream_t s) {
  if (p.dp == 64) return launch<64, NT, 64>(a, p, s);
  if (a.pool.dim == 80) return launch<128, NT, 80>(a, p, s);
  if (a.pool.dim == 96) return launch<128, NT, 96>(a, p, s);
  return launch<128, NT, 128>(a, p, s);
}

constexpr int64_t kMaxRows = 1000000000;

dsa_status check_sizes(int64_t batch, int32_t heads, int32_t kv_heads) {
  if (batch < 0 || heads < 0 || kv_heads < 1 || heads % kv_heads != 0) return DSA_EINVAL;
  if (heads / kv_heads > 128 || batch > INT32_MAX || batch * heads > kMaxRows)
    return DSA_EUNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_quant_attention_workspace_bytes(int64_t batch, int32_t heads,
                                                      int32_t kv_heads, int32_t head_dim,
                                                      int64_t max_pages, int32_t page_size) {
  if (dsa::check_sizes(batch, heads, kv_heads) != DSA_OK || batch == 0 || heads == 0 ||
      head_dim < 1 || head_dim > 128 || head_dim % 16 != 0 || max_pages < 0 ||
      max_pages > INT32_MAX || page_size < 16 || (page_size & (page_size - 1)) != 0 ||
      max_pages * page_size > INT32_MAX)
    return 0;
  const dsa::QuantPlan p =
      dsa::plan_attention(batch, heads, kv_heads, head_dim, max_pages, page_size);
  return p.fits ? p.bytes : 0;
}

extern "C" dsa_status dsa_quant_attention(const dsa_quant_pages* pages, const void* q,
                                          int32_t dtype, int64_t batch, int32_t heads,
                                          int64_t q_sb, int64_t q_sh, const int32_t* lens,
                                          float scale, void* out, int64_t o_sb, int64_t o_sh,
                                          float* lse, int64_t l_sb, int64_t l_sh, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (!(scale > 0.f) || !std::isfinite(scale * dsa::kLog2e)) return DSA_EINVAL;
  dsa::QuantAttnArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, pages, batch);
  if (st != DSA_OK) return st;
  const int32_t kv_heads = a.pool.kv_heads;
  st = dsa::check_sizes(batch, heads, kv_heads);
  if (st != DSA_OK) return st;
  if (dtype == DSA_DTYPE_F32) return DSA_EUNSUPPORTED;
  if (batch == 0 || heads == 0) return DSA_OK;
  if (!q || !out || !lens) return DSA_EINVAL;
  if (!dsa::quant_aligned16(q) || !dsa::quant_aligned16(out)) return DSA_EUNSUPPORTED;
  for (int64_t s : {q_sb, q_sh, o_sb, o_sh})
    if (s < 0 || s % 8 != 0) return DSA_EUNSUPPORTED;
  const dsa::QuantPlan p =
      dsa::plan_attention(batch, heads, kv_heads, a.pool.dim, a.pool.max_pages, pages->page_size);
  if (!p.fits) return DSA_EUNSUPPORTED;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes ||
                      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return DSA_EINVAL;
  if (a.pool.num_pages == 0) a.pool.max_pages = 0;  // nothing is seen
  a.q = q;
  a.q_sb = q_sb;
  a.q_sh = q_sh;
  a.batch = batch;
  a.group = heads / kv_heads;
  a.splits = p.splits;
  a.split_heads = p.split_heads;
  a.rows = kv_heads * p.splits;
  a.lens = lens;
  a.c = scale * dsa::kLog2e;
  a.out = out;
  a.o_sb = o_sb;
  a.o_sh = o_sh;
  a.lse = lse;
  a.l_sb = l_sb;
  a.l_sh = l_sh;
  a.bf16 = dtype == DSA_DTYPE_BF16;
  a.warps = static_cast<int32_t>(p.grid) * dsa::quant_warps(p.columns);
  char* ws = static_cast<char*>(workspace);
  a.spans = reinterpret_cast<int2*>(ws + p.spans);
  a.part_o = reinterpret_cast<float*>(ws + p.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + p.part_lse);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto run = p.columns == 1 ? dsa::launch_heads<1> : dsa::launch_heads<2>;
  return run(a, p, s);
}
